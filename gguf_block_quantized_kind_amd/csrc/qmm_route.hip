// qmm_route.hip -- the choice of experts: scores, groups, the topk largest, and
// their weights.
//
// One wave takes one token.  The values that decide are held in 64 bits: a
// score plus a bias, and sums of scores, lie closer together than f32 tells
// apart in every few thousand tokens.
#include <math.h>

#include "qmm_internal.h"

namespace qmm {
namespace route {

__device__ __forceinline__ double shfl_xor(double v, int m) {
  const int2 a = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, int2{__shfl_xor(a.x, m), __shfl_xor(a.y, m)});
}

__device__ __forceinline__ float logit(const Route &r, int64_t row, int e) {
  return r.f16 ? (float)static_cast<const _Float16 *>(r.logits)[row * r.stride + e]
               : static_cast<const float *>(r.logits)[row * r.stride + e];
}

// e^(l - m), also where both are infinite.
__device__ __forceinline__ double above(float l, float m) { return l == m ? 1.0 : exp((double)l - (double)m); }

__global__ __launch_bounds__(64) void route_kernel(const Route r) {
  extern __shared__ double pick[];  // [E]
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int E = (int)r.E, k = (int)r.topk;
  int id = -1;  // lane i: the expert of slot i
  double total = 0.0;
  float top = -INFINITY;
  if (!r.slots || r.slots[row] >= 0) {
    // The largest logit and the sum of the exponentials.
    if (!r.sigmoid) {
      for (int e = lane; e < E; e += 64) top = fmaxf(top, logit(r, row, e));  // fmaxf passes a NaN by
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
      for (int e = lane; e < E; e += 64) {
        const float l = logit(r, row, e);
        if (l > -INFINITY) total += above(l, top);
      }
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) total += shfl_xor(total, m);
    }
    // Without a bias or sums the logits decide as their scores would.
    const bool plain = !r.bias && (r.n_group == 1 || r.group_top == 1);
    for (int e = lane; e < E; e += 64) {
      const float l = logit(r, row, e);
      double c = -INFINITY;
      if (l > -INFINITY) {
        if (plain) c = l;
        else c = (r.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : above(l, top) / total) + (r.bias ? (double)r.bias[e] : 0.0);
        if (c != c) c = -INFINITY;
      }
      pick[e] = c;
    }
    __syncthreads();
    if (r.n_group > 1) {
      const int size = E / (int)r.n_group;
      double best = -INFINITY;  // lane g: its group's value
      if (lane < r.n_group) {
        double a = -INFINITY, b = -INFINITY;
        for (int i = 0; i < size; ++i) {
          const double c = pick[lane * size + i];
          if (c > a) b = a, a = c;
          else if (c > b) b = c;
        }
        best = r.group_top == 2 && b > -INFINITY ? a + b : a;
      }
      int before = 0;
      for (int g = 0; g < (int)r.n_group; ++g) {
        const int2 v = __builtin_bit_cast(int2, best);
        const double other = __builtin_bit_cast(double, int2{__shfl(v.x, g), __shfl(v.y, g)});
        if (other > best || (other == best && g < lane)) ++before;
      }
      if (lane < r.n_group && before >= r.topk_group)
        for (int i = 0; i < size; ++i) pick[lane * size + i] = -INFINITY;
      __syncthreads();
    }
    for (int j = 0; j < k; ++j) {
      double c = -INFINITY;
      int at = INT32_MAX;
      for (int e = lane; e < E; e += 64)
        if (pick[e] > c) c = pick[e], at = e;
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) {
        const double oc = shfl_xor(c, m);
        const int oa = __shfl_xor(at, m);
        if (oc > c || (oc == c && oa < at)) c = oc, at = oa;
      }
      if (c == -INFINITY) break;
      if (lane == j) id = at;
      if (lane == 0) pick[at] = -INFINITY;
      __syncthreads();
    }
  }
  // Weights of the chosen, normalized relative to the largest chosen logit, so
  // that they stay right where the scores themselves vanish.
  double w = 0.0;
  const float l = id >= 0 ? logit(r, row, id) : -INFINITY;
  if (r.normalize) {
    float lead = l;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) lead = fmaxf(lead, __shfl_xor(lead, m));
    if (id >= 0) {
      if (!r.sigmoid) w = above(l, lead);
      else if (l >= 0.f) w = 1.0 / (1.0 + exp(-(double)l));
      else w = (lead < 0.f ? above(l, lead) : exp((double)l)) / (1.0 + exp((double)l));
    }
    double sum = w;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) sum += shfl_xor(sum, m);
    if (id >= 0) w /= sum;
  } else if (id >= 0) {
    w = r.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : above(l, top) / total;
  }
  if (lane < k) {
    r.ids[row * k + lane] = id;
    r.weights[row * k + lane] = (float)(w * (double)r.scale);
  }
}

}  // namespace route

hipError_t launch_moe_route(const Route &r, hipStream_t s) {
  hipLaunchKernelGGL(route::route_kernel, dim3((unsigned)r.M), dim3(64), (size_t)r.E * sizeof(double), s, r);
  return hipGetLastError();
}

}  // namespace qmm
