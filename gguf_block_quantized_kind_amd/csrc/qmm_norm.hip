// qmm_norm.hip -- root-mean-square norm with the residual's addition:
//   h = x + residual (rounded to f32),  y = h / sqrt(mean(h^2) + eps) * weight
// to f32 or f16, or per 32 elements to 8 bits with a scale, which is the
// quantization of qmm_gemv_i8 applied to the f32 y (codes in the lane order of
// the weights they meet, with each block's scale and code sum).
//
// A row belongs to R threads (a part of a wave, a wave, or a workgroup) that
// keep it in registers as pieces of 8 elements, thread r the pieces r, r + R,
// ...: x, residual and weight are read once, with every load of a thread
// issued before the first is used, and sum and y are written once.  The rows'
// places need no alignment beyond their elements'.
//
// Squares are summed, and the factor applied, in 64 bits: squares of f32 leave
// f32's range both ways, and a code beside a border would fall on either side
// by the order of an f32 sum.
//
// Bound: memory, 5.1 TB/s of reads and writes (8192 rows of 4096, f32 with a residual
// to f16: 470 MB, 84 us; a large copy's rate); few rows by the launch and one
// workgroup's chain of load, sum, factor and store (3.4 us, 4.0 to 8 bits).
#include "qmm_internal.h"
#include "qmm_lanes.h"

namespace qmm {
namespace norm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

constexpr int V = 8;  // elements of a piece
// Workgroups along x (HIP: fewer than 2^32 threads); the others follow along y.
constexpr int64_t kGridX = 1 << 20;

// Elements [at, at + 8) of a row of D (those past its end read as 0).
// full: the same on all lanes, and then left is not looked at.
__device__ __forceinline__ void load8(const void *p, int f16, int64_t at, bool full, int left, float (&v)[V]) {
  if (full || left >= V) {
    if (f16) {
      half8 h;
      __builtin_memcpy(&h, static_cast<const _Float16 *>(p) + at, sizeof h);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = (float)h[i];
    } else {
      __builtin_memcpy(v, static_cast<const float *>(p) + at, sizeof v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = i >= left ? 0.f : f16 ? (float)static_cast<const _Float16 *>(p)[at + i] : static_cast<const float *>(p)[at + i];
  }
}

__device__ __forceinline__ void store8(void *p, int f16, int64_t at, bool full, int left, const float (&v)[V]) {
  if (full || left >= V) {
    if (f16) {
      half8 h;
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = (_Float16)v[i];
      __builtin_memcpy(static_cast<_Float16 *>(p) + at, &h, sizeof h);
    } else {
      __builtin_memcpy(static_cast<float *>(p) + at, v, sizeof v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) {
        if (f16) static_cast<_Float16 *>(p)[at + i] = (_Float16)v[i];
        else static_cast<float *>(p)[at + i] = v[i];
      }
  }
}

// A call and what divides a row's number into a token and a head.
struct Split : Norm {
  uint32_t by;
  int shift;
};

// R threads a row (8 to 64: 256 / R rows a workgroup; above: the workgroup's
// one row), NP pieces a thread, Q8: to 8 bits.
template <int R, int NP, bool Q8>
__global__ __launch_bounds__(R > 256 ? R : 256) void rmsnorm_kernel(const Split n) {
  constexpr int kThreads = R > 256 ? R : 256;
  const int r = threadIdx.x % R;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / R) + threadIdx.x / R;
  const int D = (int)n.D;
  const bool live = row < n.T * n.H;
  const int64_t at = live ? row : 0;
  const int64_t t = (int64_t)((uint64_t)(uint32_t)at * n.by >> n.shift);
  const int64_t head = (at - t * n.H) * D;

  const bool full = D == V * R * NP;
  float h[NP][V], w[NP][V];
#pragma unroll
  for (int i = 0; i < NP; ++i) load8(n.x, n.x_f16, t * n.x_stride + head + V * (r + i * R), full, D - V * (r + i * R), h[i]);
  // (Four pieces a thread leave no registers for residual and weight beside
  // them: a piece's residual is added as it comes, the weight is loaded with the
  // factor known.)
  constexpr bool kLate = NP >= 4;
  if (n.residual) {
    float a[kLate ? 1 : NP][V];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float(&b)[V] = a[kLate ? 0 : i];
      load8(n.residual, n.residual_f16, t * n.residual_stride + head + V * (r + i * R), full, D - V * (r + i * R), b);
      if constexpr (kLate) {
#pragma unroll
        for (int e = 0; e < V; ++e) h[i][e] += b[e];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (!kLate) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) h[i][e] += a[i][e];
    }
  }
  auto weights = [&]() {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (n.weight) {
        load8(n.weight, 0, V * (r + i * R), full, D - V * (r + i * R), w[i]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) w[i][e] = 1.f;
      }
    }
  };
  if constexpr (!kLate) weights();
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) ss = fma((double)h[i][e], (double)h[i][e], ss);
  ss = reduce<(R < 64 ? R : 64)>(ss, [](double a, double b) { return a + b; });
  if constexpr (R > 64) {
    __shared__ double part[R / 64];
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = ss;
    __syncthreads();
    ss = part[0];
#pragma unroll
    for (int i = 1; i < R / 64; ++i) ss += part[i];
  }
  const double m = ss / (double)D + (double)n.eps;
  const double f = m > 0.0 ? rsqrt(m) : m == 0.0 ? 0.0 : m;  // a row of zeros without eps stays one; NaN stays
  if constexpr (kLate) weights();
  if (!live) return;
  if (n.sum) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      store8(n.sum, n.residual_f16, t * n.sum_stride + head + V * (r + i * R), full, D - V * (r + i * R), h[i]);
  }
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) h[i][e] = (float)((double)h[i][e] * f * (double)w[i][e]);
  if constexpr (!Q8) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      store8(n.y, n.y_f16, t * n.y_stride + head + V * (r + i * R), full, D - V * (r + i * R), h[i]);
  } else {
    // A block is the pieces of four neighbouring threads (D is a multiple of
    // 32, so they are all there or none is).
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int p = r + i * R;
      // Magnitudes by their bits, so that a NaN or infinity is the largest: its
      // block gets a NaN for a scale and codes of 0.
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(h[i][e]) & 0x7FFFFFFFu);
      top = max(top, dpp<0xB1>(top));
      top = max(top, dpp<0x4E>(top));
      const float amax = top >= 0x7F800000u ? __builtin_nanf("") : __uint_as_float(top);
      const float d = amax / 127.0f;
      int c[V], sum = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float q = d > 0.f ? h[i][e] / d : 0.f;
        c[e] = max(-127, min(127, (int)__builtin_rintf(q)));  // beyond it only where d is subnormal
        sum += c[e];
      }
      sum += (int)dpp<0xB1>((uint32_t)sum);
      sum += (int)dpp<0x4E>((uint32_t)sum);
      if (V * p >= D) continue;
      uint32_t b[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        b[k] = (uint32_t)(c[4 * k] & 255) | (uint32_t)(c[4 * k + 1] & 255) << 8 | (uint32_t)(c[4 * k + 2] & 255) << 16 |
               (uint32_t)(c[4 * k + 3] & 255) << 24;
      const int64_t block = row * (D / 32) + p / 4;
      uint32_t *q = reinterpret_cast<uint32_t *>(n.codes + block * 32);
      const int u = p & 3;
      // Elements 8u + 4k .. + 3: in order, or at the place of qmm_gemv_i8's
      // nibble order (element 16h + s at 8 (s / 4) + 4h + s % 4).
      if (n.q8 == 1) {
        q[2 * u] = b[0];
        q[2 * u + 1] = b[1];
      } else {
        q[4 * (u & 1) + (u >> 1)] = b[0];
        q[4 * (u & 1) + 2 + (u >> 1)] = b[1];
      }
      if (u == 0) {
        n.scales[block] = d;
        n.code_sums[block] = sum;
      }
    }
  }
}

template <int R, int NP>
hipError_t run(const Norm &call, hipStream_t s) {
  constexpr int kThreads = R > 256 ? R : 256;
  const int64_t rows = call.T * call.H, per = kThreads / R;
  // row / H = row * by >> shift for rows below 2^31 (there are no more), with by =
  // 2^shift / H rounded up, beyond an exact one too: by H is at most 2^shift + 2^(shift -
  // 31), as H is at most 2^(shift - 31).
  Split n;
  static_cast<Norm &>(n) = call;
  n.shift = 31;
  while ((int64_t)1 << (n.shift - 31) < n.H) ++n.shift;
  n.by = (uint32_t)(((uint64_t)1 << n.shift) / (uint64_t)n.H + 1);
  const int64_t groups = (rows + per - 1) / per, wide = groups < kGridX ? groups : kGridX;
  const dim3 grid((unsigned)wide, (unsigned)((groups + wide - 1) / wide)), block(kThreads);
  if (n.q8) hipLaunchKernelGGL((rmsnorm_kernel<R, NP, true>), grid, block, 0, s, n);
  else hipLaunchKernelGGL((rmsnorm_kernel<R, NP, false>), grid, block, 0, s, n);
  return hipGetLastError();
}

}  // namespace norm

hipError_t launch_rmsnorm(const Norm &n, hipStream_t s) {
  const int64_t pieces = (n.D + norm::V - 1) / norm::V;
  if (pieces <= 8) return norm::run<8, 1>(n, s);
  if (pieces <= 16) return norm::run<16, 1>(n, s);
  if (pieces <= 32) return norm::run<32, 1>(n, s);
  if (pieces <= 64) return norm::run<64, 1>(n, s);
  if (pieces <= 256) return norm::run<256, 1>(n, s);
  // A piece a thread while a workgroup has enough of them.  Rows of 4096, one with
  // 8-bit codes 4.0 us (256 threads with two pieces 4.6), 8192 to f16 84.4 (88.6); rows
  // of 8192, one 5.1 (512 with two 5.2), 8192 170 (175).
  if (pieces <= 512) return norm::run<512, 1>(n, s);
  if (pieces <= 1024) return norm::run<1024, 1>(n, s);
  if (pieces <= 2048) return norm::run<1024, 2>(n, s);
  return norm::run<1024, 4>(n, s);
}

}  // namespace qmm
