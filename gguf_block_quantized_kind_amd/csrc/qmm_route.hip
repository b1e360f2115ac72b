// qmm_route.hip -- the choice of experts: scores, groups, the topk largest, and
// their weights.
//
// The choice is that of 64-bit scores, since a score plus a bias, or two sums
// of scores, lie closer together than f32 tells apart in every few thousand
// tokens.  Nearly all of the work is done in f32 all the same: f32 values
// bring out topk + 2 candidates, whose scores are computed in 64 bits (their
// weights need those anyway), and whose order is corrected where neighbours lie
// within the f32 values' error.  Groups whose f32 sums lie within 2^-19 are told
// apart by the 64-bit scores of their largest experts.  Where a doubt is left about
// which experts belong among the candidates (rows of many equal scores), the row is
// done again in 64 bits throughout.
//
// Candidates.  L = 16 or 64 lanes take a row, each up to EPL experts in
// registers.  An expert's key is a 32-bit whole number: its value's bits, made
// to order as the values do, with the lowest BITS replaced by the complement of
// its number, so keys differ, equal values go by the lowest number, and the
// key names its expert.  The next smaller key after x is x + max over keys of
// (key - x) in 32-bit wrap-around arithmetic (keys below x wrap to the top of the
// range, the nearest one highest): one subtraction and half a max3 an expert and
// a round, no compares, no removal.
//
// Bound.  16384 tokens of 256 experts (eight groups, a bias) are 17.9 MB, 3.5 us of
// memory time; the kernel takes 11.2 us, 5 of them the launch and one wave's chain
// of dependent steps (2049 tokens take 6.7), the rest the arithmetic: 950 instructions
// a wave of four rows, a third of them the selection's rounds.
#include <math.h>

#include "qmm_internal.h"
#include "qmm_lanes.h"

namespace qmm {
namespace route {

__device__ __forceinline__ double shfl(double v, int lane) {
  const int2 a = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, int2{__shfl(a.x, lane), __shfl(a.y, lane)});
}

template <bool F16>
__device__ __forceinline__ float logit_of(const Route &r, int64_t at) {
  if constexpr (F16) return (float)static_cast<const _Float16 *>(r.logits)[at];
  else return static_cast<const float *>(r.logits)[at];
}
__device__ __forceinline__ float logit(const Route &r, int64_t row, int e) {
  return r.f16 ? (float)static_cast<const _Float16 *>(r.logits)[row * r.stride + e]
               : static_cast<const float *>(r.logits)[row * r.stride + e];
}

// e^(l - m), also where both are infinite.
__device__ __forceinline__ double above(float l, float m) { return l == m ? 1.0 : exp((double)l - (double)m); }
__device__ __forceinline__ double sigmoid(float l) {
  const double t = exp(-fabs((double)l));
  return (l >= 0.f ? 1.0 : t) / (1.0 + t);
}

// Orders this wave's LDS accesses.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int L>
__device__ __forceinline__ float row_max(float v) { return reduce<L>(v, [](float a, float b) { return fmaxf(a, b); }); }
template <int L>
__device__ __forceinline__ float row_min(float v) { return reduce<L>(v, [](float a, float b) { return fminf(a, b); }); }
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v) { return reduce<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); }); }
template <int L>
__device__ __forceinline__ double row_sum(double v) { return reduce<L>(v, [](double a, double b) { return a + b; }); }

// Weight of a chosen expert with logit l (id < 0: none) on each of the L lanes
// of a row: normalized relative to the largest chosen logit, so that it stays
// right where the scores themselves vanish.  The exponentials are in 64 bits (a
// difference of logits has no rounding there), the quotients in f32.
template <int L>
__device__ __forceinline__ float weight_of(const Route &r, int id, float l, float top, double total) {
  double w = 0.0, below = 1.0;  // numerator, denominator
  float sum = 1.f;
  if (r.sigmoid) {
    const double t = exp(-fabs((double)l));
    below = 1.0 + t;
    w = l >= 0.f ? 1.0 : t;
    if (r.normalize) {
      const float lead = row_max<L>(id >= 0 ? l : -INFINITY);
      if (lead < 0.f) w = above(l, lead);
    }
  } else {
    if (r.normalize) top = row_max<L>(id >= 0 ? l : -INFINITY);
    else below = total;
    w = above(l, top);
  }
  const float share = id >= 0 ? (float)w / (float)below : 0.f;
  if (r.normalize) sum = (float)row_sum<L>((double)share);
  return id >= 0 ? share / sum : 0.f;
}

// A row by one wave, in 64 bits throughout; pick: this wave's LDS [E].
__device__ __forceinline__ void route_row(const Route &r, int64_t row, double *pick) {
  const int lane = threadIdx.x & 63;
  const int E = (int)r.E, k = (int)r.topk;
  int id = -1;  // lane i: the expert of slot i
  double total = 0.0;
  float top = -INFINITY;
  if (!r.slots || r.slots[row] >= 0) {
    // The largest logit and the sum of the exponentials.
    if (!r.sigmoid) {
      for (int e = lane; e < E; e += 64) top = fmaxf(top, logit(r, row, e));  // fmaxf passes a NaN by
      top = row_max<64>(top);
      for (int e = lane; e < E; e += 64) {
        const float l = logit(r, row, e);
        if (l > -INFINITY) total += above(l, top);
      }
      total = row_sum<64>(total);
    }
    // Without a bias or sums the logits decide as their scores would.
    const bool plain = !r.bias && (r.n_group == 1 || r.group_top == 1);
    wave_sync();  // an earlier row's reads
    for (int e = lane; e < E; e += 64) {
      const float l = logit(r, row, e);
      double c = -INFINITY;
      if (l > -INFINITY) {
        if (plain) c = l;
        else c = (r.sigmoid ? sigmoid(l) : above(l, top) / total) + (r.bias ? (double)r.bias[e] : 0.0);
        if (c != c) c = -INFINITY;
      }
      pick[e] = c;
    }
    wave_sync();
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
        const double other = shfl(best, g);
        if (other > best || (other == best && g < lane)) ++before;
      }
      if (lane < r.n_group && before >= r.topk_group)
        for (int i = 0; i < size; ++i) pick[lane * size + i] = -INFINITY;
      wave_sync();
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
      wave_sync();
    }
  }
  const float w = weight_of<64>(r, id, id >= 0 ? logit(r, row, id) : -INFINITY, top, total);
  if (lane < k) {
    r.ids[row * k + lane] = id;
    r.weights[row * k + lane] = w * r.scale;
  }
}

// Any number of experts and groups.
__global__ __launch_bounds__(64) void route_any_kernel(const Route r) {
  extern __shared__ double lds[];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row < r.M) route_row(r, row, lds);
}

// What a row's experts are ranked by, and whether the sum of the exponentials
// is needed: the logits (no bias, no sums of two), without or with that sum
// (for weights that are not normalized); the sigmoid + bias; the softmax + bias.
enum Mode { kLogit, kLogitSum, kSigmoid, kSoftmax };

// Bits of a float made to order as the floats (neither NaN nor -0).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

constexpr uint32_t kNone = 0x00800000u;  // ordered(the lowest finite float)

constexpr int log2_of(int v) { return v <= 1 ? 0 : 1 + log2_of(v / 2); }
constexpr int kWaves = 4;

// What f32 values may be off by beside their truncation in the keys: sigmoids
// and softmax shares are within 2^-22, the sum with a bias half a step more.
__device__ __forceinline__ float slack(int mode, float v) {
  return mode == kSigmoid || mode == kSoftmax ? 0x1p-21f + 0x1p-23f * fabsf(v) : 0.f;
}

// L lanes a row, EPL experts a lane.  The lanes are dealt out to the groups
// evenly (n_group divides L), and within a group's lanes its experts go in
// units of UNIT neighbours (one load), the lanes side by side.
// A call with its groups dealt out: experts of a group, and the logarithm of the
// lanes that share it.
struct Split : Route {
  int size, log_per;
};

// An expert's score with its bias, in 64 bits.
template <int MODE>
__device__ __forceinline__ double score(const Route &r, float l, int e, float top, double total) {
  return (MODE == kSigmoid ? sigmoid(l) : above(l, top) / total) + (r.bias ? (double)r.bias[e] : 0.0);
}

// The two largest values over the `per` lanes of a group, from each lane's.
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return a > b ? b : a; }
template <int L, typename T>
__device__ __forceinline__ void join_groups(int per, T &a, T &b) {
  auto join = [&](T oa, T ob) {
    b = larger(smaller(a, oa), larger(b, ob));
    a = larger(a, oa);
  };
  if (per >= 2) join(dpp<0xB1>(a), dpp<0xB1>(b));
  if (per >= 4) join(dpp<0x4E>(a), dpp<0x4E>(b));
  if (per >= 8) join(dpp<0x141>(a), dpp<0x141>(b));
  if (per >= 16) join(dpp<0x140>(a), dpp<0x140>(b));
  if (L == 64 && per >= 32) join(shfl_xor(a, 16), shfl_xor(b, 16));
}

// Groups of larger values than this lane's, or of equal ones and before it.
template <int L, typename T>
__device__ __forceinline__ int groups_before(T value, int q, int g, int log_per, int G) {
  int before = 0;
  if constexpr (L == 16) {
    // The same lane of every other group, by turns of the row.
    const int per = 1 << log_per, mine = g << log_per;  // lanes below belong to earlier groups
    auto seen = [&](T other, int n) {
      const bool earlier = ((q - n) & 15) < mine;
      before += (int)(other > value) | ((int)(other == value) & (int)earlier);
    };
#define QMM_TURN(n) \
  if ((n & (per - 1)) == 0) seen(dpp<0x120 + n>(value), n);
    QMM_TURN(1) QMM_TURN(2) QMM_TURN(3) QMM_TURN(4) QMM_TURN(5) QMM_TURN(6) QMM_TURN(7) QMM_TURN(8) QMM_TURN(9)
    QMM_TURN(10) QMM_TURN(11) QMM_TURN(12) QMM_TURN(13) QMM_TURN(14) QMM_TURN(15)
#undef QMM_TURN
  } else {
    for (int h = 0; h < G; ++h) {
      const T other = lane_of(value, h << log_per);
      before += other > value || (other == value && h < g);
    }
  }
  return before;
}

template <int L, int EPL, int MODE, bool F16>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const Split r) {
  constexpr int BITS = log2_of(L * EPL);
  constexpr uint32_t kLow = (1u << BITS) - 1;
  constexpr int UNIT = EPL < 4 ? EPL : 4, NU = EPL / UNIT;
  extern __shared__ double lds[];
  const int lane = threadIdx.x & 63, q = lane % L;
  const int64_t first = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWaves + (threadIdx.x >> 6)) * (64 / L);
  if (first >= r.M) return;  // the whole wave
  const int64_t row = first + lane / L;
  const bool there = row < r.M;
  const int k = (int)r.topk, G = (int)r.n_group;
  const bool live = there && (!r.slots || r.slots[row] >= 0);
  const int size = r.size, log_per = r.log_per, per = 1 << log_per;  // experts and lanes of a group
  const int g = q >> log_per, sub = q & (per - 1);

  // Logits and biases; experts that are not there read as -inf.  Where the
  // experts fill every lane (the same for all rows) the loads go out together
  // under no lane's condition, rows that are skipped reading the last row's.
  float l[EPL], b[EPL];
  constexpr bool kBias = MODE == kSigmoid || MODE == kSoftmax;
#pragma unroll
  for (int i = 0; i < EPL; ++i) b[i] = 0.f;
  if (size == NU * UNIT * per) {
    const int64_t base = min(row, r.M - 1) * r.stride + g * size + sub * UNIT;
    if constexpr (F16) {
      _Float16 h[NU][UNIT];
#pragma unroll
      for (int u = 0; u < NU; ++u)
        __builtin_memcpy(h[u], static_cast<const _Float16 *>(r.logits) + base + u * per * UNIT, sizeof h[u]);
#pragma unroll
      for (int i = 0; i < EPL; ++i) l[i] = (float)h[i / UNIT][i % UNIT];
    } else {
#pragma unroll
      for (int u = 0; u < NU; ++u)
        __builtin_memcpy(&l[u * UNIT], static_cast<const float *>(r.logits) + base + u * per * UNIT, UNIT * sizeof(float));
    }
    if (kBias && r.bias) {
#pragma unroll
      for (int u = 0; u < NU; ++u)
        __builtin_memcpy(&b[u * UNIT], r.bias + g * size + (u * per + sub) * UNIT, UNIT * sizeof(float));
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = live ? l[i] : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int at = (i / UNIT * per + sub) * UNIT + i % UNIT;  // within the group
      const bool is = live && at < size;
      const int e = is ? g * size + at : 0;
      const int64_t from = (is ? row : 0) * r.stride + e;
      l[i] = logit_of<F16>(r, from);
      if (kBias && r.bias) b[i] = r.bias[e];
      l[i] = is ? l[i] : -INFINITY;
    }
  }

  // The largest logit and the sum of the exponentials.
  float top = -INFINITY;
  double total = 0.0;
  if constexpr (MODE == kLogitSum || MODE == kSoftmax) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = fmaxf(top, l[i]);
    top = row_max<L>(top);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (!(l[i] > -INFINITY)) continue;
      if constexpr (MODE == kSoftmax) total += above(l[i], top);  // decides: 64 bits
      else total += l[i] == top ? 1.0 : (double)expf(l[i] - top);
    }
    total = row_sum<L>(total);
  }

  // Values in f32.
  float c[EPL];
  const float share = MODE == kSoftmax ? (float)(1.0 / total) : 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float v = l[i];
    float s;
    if constexpr (MODE == kSigmoid) s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504f)) + b[i];
    else if constexpr (MODE == kSoftmax) s = (v == top ? 1.0f : __builtin_amdgcn_exp2f((v - top) * 1.44269504f)) * share + b[i];
    else s = v + 0.0f;  // -0 ranks as 0
    c[i] = v > -INFINITY && s > -INFINITY ? s : -INFINITY;  // NaN of either: never chosen
  }

  if (G > 1) {
    // The group's value, on each of its lanes.
    float a = -INFINITY, b2 = -INFINITY;  // the two largest
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      b2 = __builtin_amdgcn_fmed3f(a, b2, c[i]);
      a = __builtin_amdgcn_fmed3f(a, c[i], INFINITY);
    }
    join_groups<L>(per, a, b2);
    const float value = r.group_top == 2 && b2 > -INFINITY ? a + b2 : a;
    bool kept = groups_before<L>(value, q, g, log_per, G) < (int)r.topk_group;
    if constexpr (MODE == kSigmoid || MODE == kSoftmax) {
      // How far the kept ones are above the others.
      const float in = row_min<L>(kept ? value : INFINITY), out = row_max<L>(kept ? -INFINITY : value);
      // What the sums round off goes by their terms.
      const float terms = row_max<L>(a > -INFINITY ? fabsf(a) + (b2 > -INFINITY ? fabsf(b2) : 0.f) : 0.f);
      const bool near = out > -INFINITY && !(in - out > 0x1p-19f + 0x1p-21f * terms);
      if (__any(near)) {
        // The groups by 64-bit values, of the experts that may be among their two
        // (or one) largest.  One row of every few thousand, but the call waits for it:
        // 16384 tokens of 256 experts 11.2 us, 20 with such rows done again as a whole.
        const float least = r.group_top == 2 ? b2 : a;
        uint32_t in_question = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (c[i] > -INFINITY && !(c[i] < least - slack(MODE, least) - slack(MODE, c[i]))) in_question |= 1u << i;
        double da = -INFINITY, db = -INFINITY;
        while (__any(in_question != 0)) {
          if (in_question) {
            const int i = __builtin_ctz(in_question);
            in_question &= in_question - 1;
            const int e = g * size + (i / UNIT * per + sub) * UNIT + i % UNIT;
            const double v = score<MODE>(r, logit_of<F16>(r, row * r.stride + e), e, top, total);
            if (v > da) db = da, da = v;
            else if (v > db) db = v;
          }
        }
        join_groups<L>(per, da, db);
        kept = groups_before<L>(r.group_top == 2 && db > -INFINITY ? da + db : da, q, g, log_per, G) < (int)r.topk_group;
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = kept ? c[i] : -INFINITY;
  }

  // (Experts that are out have the keys of -inf, below kNone.)
  uint32_t key[EPL], best = 0;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const uint32_t low = kLow - (uint32_t)(g * size + (u * per + sub) * UNIT);
#pragma unroll
    for (int x = 0; x < UNIT; ++x) {
      const int i = u * UNIT + x;
      key[i] = (ordered(c[i]) & ~kLow) | ((low - x) & kLow);
      best = max(best, key[i]);
    }
  }
  // Candidates: lane j gets the j-th largest key.
  uint32_t x = row_max<L>(best), mine = q == 0 ? x : 0u;
  for (int j = 1; j < k + 2; ++j) {
    uint32_t d = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) d = max(d, key[i] - x);
    d = row_max<L>(d);
    x = x + d < x ? x + d : 0u;  // none below: 0, and it stays
    mine = q == j ? x : mine;
  }

  // Order and completeness within the values' error.
  const int id0 = mine >= kNone ? (int)(kLow - (mine & kLow)) : -1;
  const uint32_t cell = mine & ~kLow;
  const uint32_t next = __shfl_down(mine, 1), over = __shfl_down(mine, 2);
  const float v = unordered(cell);
  bool close = false, open = false;
  // f16 logits fill no more bits than the keys keep.
  if constexpr (!((MODE == kLogit || MODE == kLogitSum) && F16)) {
    auto near = [&](uint32_t other) {
      if (other < kNone) return false;
      const float w = unordered(other | kLow);  // its cell's upper end
      return !(v - w > 2.0f * slack(MODE, v));
    };
    if (id0 >= 0 && q < k) close = near(next);
    if (id0 >= 0 && q == k - 1) open = near(over);
  }

  // The candidates' scores in 64 bits.
  const float cl = id0 >= 0 ? logit_of<F16>(r, row * r.stride + id0) : -INFINITY;
  int slot = q;
  if (__any(close)) {
    double exact = -INFINITY;
    if (id0 >= 0) {
      if constexpr (kBias) exact = score<MODE>(r, cl, id0, top, total);
      else exact = cl;
    }
    int before = 0;
    for (int j = 0; j < k + 2; ++j) {
      const double o = shfl(exact, lane - q + j);
      const int oi = __shfl(id0, lane - q + j);
      before += oi >= 0 && (o > exact || (o == exact && oi < id0));
    }
    if (id0 >= 0) slot = before;
  }
  const int id = slot < k ? id0 : -1;
  const float w = weight_of<L>(r, id, cl, top, total);
  if (there && q < k + 2 && slot < k) {
    r.ids[row * k + slot] = id;
    r.weights[row * k + slot] = w * r.scale;
  }
  // Rows in doubt again, one at a time.
  uint64_t again = __ballot(open && live);
  while (again) {
    const int at = __builtin_ctzll(again);
    again &= L == 64 ? 0ull : ~(((1ull << (L % 64)) - 1) << (at / L * L));
    route_row(r, first + at / L, lds + (threadIdx.x >> 6) * r.E);
  }
}

constexpr int64_t kGridX = 1 << 20;

template <int L, int EPL, int MODE>
void launch(const Split &r, dim3 grid, size_t lds, hipStream_t s) {
  if (r.f16) hipLaunchKernelGGL((route_kernel<L, EPL, MODE, true>), grid, dim3(64 * kWaves), lds, s, r);
  else hipLaunchKernelGGL((route_kernel<L, EPL, MODE, false>), grid, dim3(64 * kWaves), lds, s, r);
}

template <int L, int EPL>
hipError_t run(const Route &call, int mode, hipStream_t s) {
  Split r;
  static_cast<Route &>(r) = call;
  r.size = (int)(r.E / r.n_group), r.log_per = __builtin_ctz((unsigned)(L / r.n_group));
  const int64_t per = kWaves * (64 / L), groups = (r.M + per - 1) / per, wide = groups < kGridX ? groups : kGridX;
  const dim3 grid((unsigned)wide, (unsigned)((groups + wide - 1) / wide));
  const size_t lds = (size_t)kWaves * r.E * sizeof(double);
  switch (mode) {
    case kLogit: launch<L, EPL, kLogit>(r, grid, lds, s); break;
    case kLogitSum: launch<L, EPL, kLogitSum>(r, grid, lds, s); break;
    case kSigmoid: launch<L, EPL, kSigmoid>(r, grid, lds, s); break;
    default: launch<L, EPL, kSoftmax>(r, grid, lds, s); break;
  }
  return hipGetLastError();
}

}  // namespace route

hipError_t launch_moe_route(const Route &r, hipStream_t s) {
  using namespace route;
  const bool plain = !r.bias && (r.n_group == 1 || r.group_top == 1);
  const int mode = plain ? (r.sigmoid || r.normalize ? kLogit : kLogitSum) : r.sigmoid ? kSigmoid : kSoftmax;
  // Experts of a lane, in whole units, where L lanes share a row (0: they cannot:
  // groups that do not divide them, more candidates than lanes).
  auto fit = [&](int64_t L, int64_t unit) -> int64_t {
    if (L % r.n_group != 0 || r.topk + 2 > L) return 0;
    const int64_t size = r.E / r.n_group, step = L / r.n_group * unit;
    return (size + step - 1) / step * unit;
  };
  // Many rows: 16 lanes each, four rows a wave.  Few: a wave each, whose
  // selection takes fewer steps in a row.
  if (const int64_t n = fit(16, 4); n && r.M > 2048) {
    if (n <= 4) return run<16, 4>(r, mode, s);
    if (n <= 8) return run<16, 8>(r, mode, s);
    if (n <= 16) return run<16, 16>(r, mode, s);
  }
  if (const int64_t n = fit(64, 4)) {
    if (fit(64, 1) == 1) return run<64, 1>(r, mode, s);
    if (fit(64, 2) == 2) return run<64, 2>(r, mode, s);
    if (n <= 4) return run<64, 4>(r, mode, s);
    if (n <= 8) return run<64, 8>(r, mode, s);
    if (n <= 16) return run<64, 16>(r, mode, s);
  }
  const int64_t wide = r.M < kGridX ? r.M : kGridX;
  hipLaunchKernelGGL(route_any_kernel, dim3((unsigned)wide, (unsigned)((r.M + wide - 1) / wide)), dim3(64),
                     (size_t)r.E * sizeof(double), s, r);
  return hipGetLastError();
}

}  // namespace qmm
