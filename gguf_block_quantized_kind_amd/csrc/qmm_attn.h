// qmm_attn.h -- attention of one new token per sequence over the paged cache
// of qmm_kv.h: the matrix-core kernel, by key kind, value kind, head size and
// query type.
//
//   s_t = scale * q . k_t,   out = sum_t e^{s_t} v_t / (sum_t e^{s_t} + e^sink)
//
// over the tokens lo <= t < len of a sequence, lo = max(0, len - window).
//
// Work.  The tokens of a (sequence, key head) are cut into splits of whole
// 32-token groups; a workgroup of four waves takes one split, its waves every
// fourth group.  The G = n_q / n_kv query heads that share the key head are
// the columns of the matrix-core products (16 at a time), so the cache is
// read once per key head.  The number of groups per split follows from the
// lengths themselves, which every workgroup reads: the host need not know
// them, and the call can be captured.
//
// Products, per group (layouts in qmm_kv.h):
//   scores   D[token][head] = K . Q^T.  F16 keys are the operand as they are.
//            Codes enter as f16 subnormals, u * 2^-24 with u the stored
//            unsigned code (one v_perm or AND per two codes; a high nibble
//            stays in place as 16 u, its query element divided by 16), the
//            offset as the accumulator's start value -offset * sum q (Q4_0
//            beside f32 queries: signed integers, as the values); each
//            block's product is scaled by the token's f32 block scale.
//   values   D[element][head] += V^T . P^T; the block scale goes into the
//            weight, p * d.  Beside f16 queries weights are rounded once to
//            f16 and codes enter as exact signed integers in f16.  Beside f32
//            queries weights are f32: with codes as three bf16 terms of eight
//            bits each, which have f32's range (codes are exact in bf16 too);
//            with F16 values in f32 products, v_mfma_f32_16x16x4_f32, or up to
//            four heads v_mfma_f32_4x4x1_16b_f32, which takes the same 64 values
//            against 4 columns instead of 16 in a quarter of the time (the heads
//            then fill the 16 score columns four times over).
// f32 queries are split into two f16 terms (exact to about 2^-22 of an element, or
// 2^-39 of the head's largest).
//
// The softmax keeps a running reference R per head.  Beside f32 queries it is
// the running maximum - 40, so that the last terms of a weight 2^-100 of the
// largest, times the smallest scale 2^-24, are still normal.  Beside f16 queries it is the maximum of (maximum of s
// over eight tokens + exponent of their largest value scale) - 14, so that p * d =
// 2^(s - R) * d reaches 2^14..2^15 for the strongest token and block: weights
// down to 2^-28 of it are normal f16 numbers, below that they lose bits, each
// at most 2^-39 of it (2^-25 against 2^14).  One term so loses what a weak
// token or a small block contributes to an element that the strong ones leave
// empty; two f16 terms share the exponent range and lose it too (all of it from
// e^-30 down), which f32 results do not bear.  f16 results do: the wider terms
// would bring them from 2.3e-4 to 2.0e-4 of the exact norm, of which the result's
// own rounding is 2.0e-4, for 95 -> 102 us (64 ragged sequences) and 32 -> 38 (48
// windows).  What they cost f32 queries against two f16 terms, 64 sequences of 0
// to 8192 tokens, 8 key heads: 32 heads of 128, Q8_0 119 -> 121 us, Q4_0 95 -> 101,
// F16 197 -> 197; 64 heads of 128, 123 -> 127, 96 -> 106, 202 -> 211; 32 heads of
// 256, 240 -> 268, 208 -> 271, 386 -> 388.  The f32 forms against each other: f32
// products of 16 columns for codes, 64 heads of 128, Q8_0 158 us, Q4_0 141; of four
// columns for 32 heads of 128 120 and 101, of 256 278 and 292; F16 values with 32
// heads of 128 in 16 columns 203.
//
// Sums.  A split may hold any number of tokens, and a running f32 sum of
// like terms rounds the same way each time.  The weights' sum takes eight at a
// time and carries what each addition rounds off; the accumulators take at most
// kAdds groups before they are added to the wave's part in LDS, and keep what that
// addition rounds off.  So the error does not grow with the length (plain running
// sums: 1e-3 at a million tokens of a split; no difference in time measured).
//
// What bounds it: the cache's bytes, read once at the rate of a large read (5.5
// TB/s here) as soon as there are enough of them.  Measured, the attention
// kernel alone: one sequence of 131071 tokens, 32 / 8 heads of 128, Q8_0 keys
// and values (285 MB) 53 us, 5.3 TB/s; 64 sequences of 0 to 8192 tokens, Q8_0
// and Q4_0 (437 MB) 91 us, 4.8 TB/s, in Q8_0 with heads of 96 (429 MB) 83 us, of
// 192 (857 MB) 160 us, of 256 (1.14 GB) 218 us, 5.2 to 5.3 TB/s; 16 of 0 to 4001,
// 32 / 32 heads, F16, f32 queries (474 MB) 86 us, 5.5 TB/s; 48 windows of 4096,
// 64 / 8 heads of 64, Q4_0 (99 MB) 29 us, 3.4 TB/s, of which about 8 are starts and
// ends; 1024 sequences of 0 to 600, Q8_0 (683 MB) 144 us, 4.8 TB/s, after a plan of
// 5.  Choices that were measured against another:
//   accumulators in vector registers instead of accumulation registers (which
//     cost 112 moves a group at heads of 128), one fused multiply-convert per
//     weight: 64 ragged sequences 120 -> 92 us.  Heads of 256 spill into
//     accumulation registers in most kinds and leave one wave per SIMD; a bound
//     of two waves spills to memory instead (f32 queries, Q8_0: 282 -> 816 us);
//   keys of the next group loaded as soon as this one's are used, values
//     likewise: 92 us there against 113 with two or three whole groups in flight
//     at once, whose registers cost a wave per SIMD;
//   one equal range of the batch's groups per workgroup, in one round, instead
//     of splits: 92 -> 119 us (all workgroups start and end together, and a
//     range covers two pairs' ends);
//   joining the splits in the attention kernel (the last to arrive) instead of
//     by a second launch: its release fences alone, which write the L2 back,
//     cost 30 to 70 us; the launch costs 5.
#pragma once

#include <algorithm>
#include <atomic>

#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {
namespace attn {

using kv::C_F16;
using kv::C_Q4_0;
using kv::C_Q8_0;

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kFloor = -3e38f;  // R of no tokens
constexpr float kFar = 0x1p20f;  // scores whose products are rounded by more than 2^-5
constexpr int kWaves = 4;
constexpr int kMinGroups = 4;  // groups per split at least: one per wave
constexpr int kMaxSlots = 1280;  // most workgroups counted on at once (five on each of 256 compute units)
// A workgroup's start and end, in groups' time, for the choice between one round
// of splits and two.  With 2, 8 and 32: 48 windows of 4096, 8 heads of 64 in Q4_0
// (groups of 2 KB) 39, 33, 33 us; 64 ragged sequences, heads of 128 in Q8_0 and
// Q4_0 96.4, 95.8, 102.4; heads of 256 in F16 (32 KB) no difference.
constexpr float kOverhead = 8.0f;

struct Args {
  const uint8_t *kp, *vp;
  int64_t k_page_bytes, v_page_bytes, n_pages;
  int page_groups;  // 32-token groups per page
  int n_kv, n_q, G, tiles, heads;  // tiles of `heads` = min(G, 16) query heads
  const void *q;
  int64_t q_stride;
  const int32_t *table;
  int64_t max_pages;
  const int32_t *lens;
  int B;
  float scale2;  // scale * log2(e)
  int64_t window;
  const float *sinks;
  void *out;
  float *part;    // [item][heads][D], then [item][heads][2]: reference and sum
  int32_t *plan;   // [B][2]: a sequence's first split and number of splits, for the join
  int32_t *units;  // more than 64 sequences: number of splits, then each split's sequence
  int64_t items;  // workgroups launched
  int slots;      // workgroups the GPU holds at once
};

// The groups [g0, g0 + n) of sequence b that hold attended tokens [lo, len).
struct Span {
  int lo, len, g0, n;
};
__device__ __forceinline__ int length_of(const Args &a, int b) {
  const int64_t most = a.max_pages * a.page_groups * kv::kGroup;
  const int len = b < a.B ? max(a.lens[b], 0) : 0;
  return len > most ? (int)most : len;
}
__device__ __forceinline__ Span span_at(const Args &a, int len) {
  const int lo = a.window > 0 && len > a.window ? len - (int)a.window : 0;
  const int g0 = lo / kv::kGroup;
  return Span{lo, len, g0, len > 0 ? (int)(((int64_t)len + kv::kGroup - 1) / kv::kGroup) - g0 : 0};
}
__device__ __forceinline__ Span span_of(const Args &a, int b) { return span_at(a, length_of(a, b)); }

// Reductions over the four lane groups G of a column (lanes j, 16 + j, 32 + j,
// 48 + j), every lane receiving the result: each swap exchanges rows of 16 or
// 32 lanes between two copies of the value.
__device__ __forceinline__ float max_over_groups(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  v = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float sum_over_groups(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  v = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

// Sums of two values over pairs of lane groups, one swap for both: over groups
// 2i and 2i + 1, a's in group 2i and b's in 2i + 1; over groups i and i + 2, a's in
// groups 0 and 1 and b's in 2 and 3.
__device__ __forceinline__ float sum_of_rows(float u, float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, u), __builtin_bit_cast(uint32_t, v), false, false);
  return __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
}
__device__ __forceinline__ float sum_of_halves(float u, float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, u), __builtin_bit_cast(uint32_t, v), false, false);
  return __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
}

// Inclusive sum over the lanes of a wave, without LDS: within rows of 16, then
// each row's last lane into the rows after it.
__device__ __forceinline__ uint32_t scan(uint32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2, 3
  return v;
}

// Splits are numbered through the batch (at least one per sequence, so that
// every output row is written).  find_split: the sequence (-1: past the last)
// that split `unit` belongs to, its first split and their number.
//
// Groups per split, c.  Either all splits run at once: the smallest c whose
// splits fit the slots, costing c + overhead; or there are two rounds of them
// (of which the second overlaps the first's ends, by half a split on
// average), c = total / (2 slots), costing total / slots + 2 overheads + c / 2.
// Equal lengths take the first, very unequal ones the second.
//
// Up to 64 sequences every wave works this out by itself, one lane each; more
// are planned by plan_kernel, once, before.
constexpr int kLanes = 64;
struct Found {
  int b, first, splits, len;
};
// At least groups / splits (in f32, rounded up past its errors).
__device__ __forceinline__ int per_split(float groups, float splits) {
  return (int)fminf(fmaxf(groups / splits * (1.0f + 0x1p-20f) + 1.0f, (float)kMinGroups), 0x1p26f);
}
// ceil(n / c) for 0 <= n <= 2^26, c >= 4: a quotient in f32 is within two of it.
__device__ __forceinline__ int splits_of(int n, int c, float inv) {
  int q = (int)((float)n * inv);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int r = q * c - n;  // (within a few c of 0: no overflow)
    q += r < 0 ? 1 : r >= c ? -1 : 0;
  }
  return max(q, 1);
}
// Two rounds of splits, or `once`, where all run at once: the cheaper.
__device__ __forceinline__ int choose(int once, int twice, float groups, float slots) {
  return (float)once <= groups / slots + kOverhead + 0.5f * (float)twice ? once : twice;
}
__device__ __forceinline__ int fewer(int c, float items, float slots) { return (int)((float)c * (items / slots)) + 1; }

__device__ __forceinline__ Found find_split(const Args &a, int lane, uint32_t unit) {
  const int nh = a.n_kv * a.tiles, len = length_of(a, lane);
  int n = span_at(a, len).n;
  if (a.B == 1) {
    n = __builtin_amdgcn_readfirstlane(n);
    const int most = max(a.slots / nh, 1), c = max((n + most - 1) / most, kMinGroups);
    const int splits = splits_of(n, c, 1.0f / (float)c);
    return Found{unit < (uint32_t)splits ? 0 : -1, 0, splits, __builtin_amdgcn_readfirstlane(len)};
  }
  // (At most 2^26 groups a sequence: one less keeps 64 of them below 2^32.)
  const uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)scan((uint32_t)min(n, (1 << 26) - 1)), 63);
  const float groups = (float)total * (float)nh, slots = (float)a.slots;
  int c = per_split(groups, 2.0f * slots);
  if (a.B * nh <= a.slots) {
    int once = per_split(groups, slots);
#pragma unroll 1
    for (int i = 0; i < 3; ++i) {
      const uint32_t splits = lane < a.B ? (uint32_t)splits_of(n, once, 1.0f / (float)once) : 0;
      const int items = __builtin_amdgcn_readlane((int)scan(splits), 63) * nh;
      if (items <= a.slots) break;
      once = fewer(once, (float)items, slots);
    }
    c = choose(once, c, groups, slots);  // (if they still do not all fit, the cost is near enough)
  }
  c = __builtin_amdgcn_readfirstlane(c);
  const uint32_t splits = lane < a.B ? (uint32_t)splits_of(n, c, 1.0f / (float)c) : 0;
  const uint32_t incl = scan(splits);
  const uint64_t mask = __ballot(unit < incl);
  if (!mask) return Found{-1, 0, 0, 0};
  const int l = __ffsll((unsigned long long)mask) - 1;
  return Found{l, __builtin_amdgcn_readlane((int)(incl - splits), l), __builtin_amdgcn_readlane((int)splits, l),
               __builtin_amdgcn_readlane(len, l)};
}

__device__ __forceinline__ ushort2v as_us2(uint32_t v) { return __builtin_bit_cast(ushort2v, v); }
__device__ __forceinline__ uint32_t as_u(ushort2v v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ half2v as_h2(uint32_t v) { return __builtin_bit_cast(half2v, v); }
__device__ __forceinline__ half8 as_h8(u32x4 v) { return __builtin_bit_cast(half8, v); }
__device__ __forceinline__ uint32_t pk_add(uint32_t a, _Float16 b) {
  const half2v v = __builtin_bit_cast(half2v, a) + half2v{b, b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint32_t pk_fma(uint32_t a, _Float16 m, _Float16 b) {
  const half2v v = __builtin_elementwise_fma(__builtin_bit_cast(half2v, a), half2v{m, m}, half2v{b, b});
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {  // a's in the low half
  return __builtin_amdgcn_perm(bits_of(b), bits_of(a), 0x07060302);
}

// Bytes of one block as a lane reads them.
template <int KIND> struct Raw { u32x4 w; };  // Q8_0
template <> struct Raw<C_F16> { u32x4 w[2]; };
template <> struct Raw<C_Q4_0> { u32x2 w; };

template <int KIND>
__device__ __forceinline__ void load_block(const uint8_t *block, int lane, Raw<KIND> &r) {
  if constexpr (KIND == C_F16) {
    r.w[0] = *(const u32x4 *)(block + lane * 16);
    r.w[1] = *(const u32x4 *)(block + 1024 + lane * 16);
  } else if constexpr (KIND == C_Q8_0) {
    r.w = *(const u32x4 *)(block + lane * 16);
  } else {
    r.w = *(const u32x2 *)(block + lane * 8);
  }
}

// Eight bytes of Q8_0, or the nibbles of pairs of Q4_0 bytes, as exact signed
// integers in f16: the code under the mantissa of 1024 (a high nibble 16 times
// too high), the offset taken off by one packed operation.
__device__ __forceinline__ half8 signed_bytes(uint32_t a, uint32_t b) {
  const uint32_t k = 0x64646464;  // 1024 + u
  return as_h8(u32x4{pk_add(__builtin_amdgcn_perm(k, a, 0x04010400), -1152.0f16),
                     pk_add(__builtin_amdgcn_perm(k, a, 0x04030402), -1152.0f16),
                     pk_add(__builtin_amdgcn_perm(k, b, 0x04010400), -1152.0f16),
                     pk_add(__builtin_amdgcn_perm(k, b, 0x04030402), -1152.0f16)});
}
// The constants sit in registers so that mask and exponent are one v_and_or
// (an instruction takes one scalar operand, and these literals need two).
struct Nibbles {
  uint32_t k, low, high;
  __device__ __forceinline__ Nibbles() : k(0x64006400), low(0x000f000f), high(0x00f000f0) {
    asm("" : "+v"(k), "+s"(low), "+s"(high));
  }
  __device__ __forceinline__ uint32_t signed_low(uint32_t a) const { return pk_add((a & low) | k, -1032.0f16); }
  __device__ __forceinline__ uint32_t signed_high(uint32_t a) const {  // (1024 + 16 u) / 16 - 72
    return pk_fma((a & high) | k, 0.0625f16, -72.0f16);
  }
};

// Whether codes of keys enter as f16 subnormals.  The matrix cores align the
// products of one step by the operands' exponent fields, so a subnormal code u
// keeps only about 24 - 10 + log2(u) bits: fine beside f16 queries, too few
// for Q4_0 beside f32 ones (measured: outputs off by 5e-6 instead of 3e-7).
template <int KK, bool SPLIT>
constexpr bool kSubnormalKeys = KK == C_Q8_0 || (KK == C_Q4_0 && !SPLIT);

// Key operand of tile m: halves, codes * 2^-24 (Q4_0 high nibbles 2^-20), or
// signed codes.
template <int KK, bool SPLIT>
__device__ __forceinline__ half8 key_operand(const Raw<KK> &r, int m, const Nibbles &nb) {
  if constexpr (KK == C_F16) return as_h8(r.w[m]);
  if constexpr (KK == C_Q4_0 && SPLIT) {
    const uint32_t a = r.w[m], b = a >> 8;
    return as_h8(u32x4{nb.signed_low(a), nb.signed_high(a), nb.signed_low(b), nb.signed_high(b)});
  }
  if constexpr (KK == C_Q8_0) {
    const uint32_t a = r.w[2 * m], b = r.w[2 * m + 1];
    return as_h8(u32x4{__builtin_amdgcn_perm(0, a, 0x0c010c00), __builtin_amdgcn_perm(0, a, 0x0c030c02),
                       __builtin_amdgcn_perm(0, b, 0x0c010c00), __builtin_amdgcn_perm(0, b, 0x0c030c02)});
  } else if constexpr (KK == C_Q4_0) {
    const uint32_t a = r.w[m], b = a >> 8;
    return as_h8(u32x4{a & 0x000f000f, a & 0x00f000f0, b & 0x000f000f, b & 0x00f000f0});
  }
}

// Value operand of tile x: halves, or exact signed codes.  Token order of the
// eight K entries: natural, for Q4_0 0 2 1 3 4 6 5 7.
template <int VK>
__device__ __forceinline__ half8 value_operand(const Raw<VK> &r, int x, const Nibbles &nb) {
  if constexpr (VK == C_F16) return as_h8(r.w[x]);
  if constexpr (VK == C_Q8_0) return signed_bytes(r.w[2 * x], r.w[2 * x + 1]);
  if constexpr (VK == C_Q4_0) {
    const uint32_t a = r.w[0], b = r.w[1];
    if (x == 0) return as_h8(u32x4{nb.signed_low(a), nb.signed_low(a >> 8), nb.signed_low(b), nb.signed_low(b >> 8)});
    return as_h8(u32x4{nb.signed_high(a), nb.signed_high(a >> 8), nb.signed_high(b), nb.signed_high(b >> 8)});
  }
}
template <int VK>
__device__ __forceinline__ constexpr int v_token(int k) {
  if (VK != C_Q4_0) return k;
  const int p = k & 3;
  return (k & 4) + (p == 1 ? 2 : p == 2 ? 1 : p);
}

// Value operand of tile x beside f32 queries: codes (Q4_0's times 16) in bf16, in
// natural order.  A signed byte (Q4_0: the nibble in the upper half, its top bit
// turned) becomes f32, whose upper half holds it.
template <int VK>
__device__ __forceinline__ bf16x8 value_bf16(const Raw<VK> &r, int x) {
  u32x4 u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t c;
    if constexpr (VK == C_Q8_0) c = r.w[2 * x + i] ^ 0x80808080u;
    else c = ((x == 0 ? r.w[i] << 4 : r.w[i]) & 0xf0f0f0f0u) ^ 0x80808080u;
    u[2 * i] = upper_halves((float)(int8_t)c, (float)(int8_t)(c >> 8));
    u[2 * i + 1] = upper_halves((float)(int8_t)(c >> 16), (float)(int8_t)(c >> 24));
  }
  return __builtin_bit_cast(bf16x8, u);
}

// The query elements of the eight K entries of lane group G, of a block of 32
// (qmm_kv.h; Q4_0 bytes are taken in the order 0, 2, 1, 3, low and high nibbles
// of a pair of bytes side by side), as floats.
template <int KK, typename QT>
__device__ __forceinline__ void load_q(const QT *q, int G, float (&v)[8]) {
  typedef QT q4 __attribute__((ext_vector_type(4)));
  q4 a, b;
  __builtin_memcpy(&a, q + (KK == C_Q4_0 ? 4 * G : 8 * G), sizeof a);
  __builtin_memcpy(&b, q + (KK == C_Q4_0 ? 16 + 4 * G : 8 * G + 4), sizeof b);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int y = (k & 1) * 2 + (k >> 2);
    v[k] = KK == C_Q4_0 ? (float)(k & 2 ? b[y] : a[y]) : (float)(k < 4 ? a[k] : b[k - 4]);
  }
}

// Four elements of the result: the sums o over the weights' sum l (both on
// reference R), with the sink's share on the larger of the two references;
// zeros where nothing was attended.
template <typename QT>
__device__ __forceinline__ void store_out(QT *out, floatx4 o, float l, float R, const float *sinks, int head) {
  float root = 1.0f;  // of the sums' factor, which may lie below f32's range
  if (sinks) {
    // (Cut where it would overflow: an infinite sink takes all the weight, like
    // any other far above the scores.  A NaN stays.)
    float sink = sinks[head] * 1.44269504f;
    sink = sink > 3e38f ? 3e38f : sink;
    const float Rn = fmaxf(R, sink);
    root = __builtin_amdgcn_exp2f(0.5f * (R - Rn));
    l = __builtin_fmaf(l * root, root, __builtin_amdgcn_exp2f(sink - Rn));
  }
  const float inv = l > 0.0f || l != l ? root / l : 0.0f;
  o *= root;
  typedef QT q4 __attribute__((ext_vector_type(4)));
  *(q4 *)out = q4{(QT)(o[0] * inv), (QT)(o[1] * inv), (QT)(o[2] * inv), (QT)(o[3] * inv)};
}

// COLS: 16, or 4 for f32 queries of up to four heads over F16 values.
template <int KK, int VK, int NB, typename QT, int COLS>
__global__ __launch_bounds__(64 * kWaves) void attn_kernel(Args a) {
  constexpr int D = NB * 32;
  constexpr bool SPLIT = sizeof(QT) == 4;  // two terms of the query, f32 weights
  constexpr float kUnit = SPLIT && VK == C_Q4_0 ? 0.0625f : 1.0f;  // of the accumulators
  constexpr bool SUB = kSubnormalKeys<KK, SPLIT>;
  constexpr int kPitch = D + 4;
  extern __shared__ __attribute__((aligned(16))) float lds[];  // [part][heads][kPitch], then [part][heads][2]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane & 15, G = lane >> 4;

  // Which split this workgroup has.
  const uint32_t nh = (uint32_t)(a.n_kv * a.tiles), unit = blockIdx.x / nh;
  const int hh = (int)(blockIdx.x - unit * nh), kvh = hh % a.n_kv, tile = hh / a.n_kv;
  Found f;
  if (a.B <= kLanes) {
    f = find_split(a, lane, unit);
    if (f.b < 0) return;
    if ((int)unit == f.first && hh == 0 && threadIdx.x == 0) {
      a.plan[2 * f.b] = f.first;
      a.plan[2 * f.b + 1] = f.splits;
    }
  } else {
    if (unit >= (uint32_t)a.units[0]) return;
    f.b = a.units[1 + unit];
    f.first = a.plan[2 * f.b], f.splits = a.plan[2 * f.b + 1], f.len = length_of(a, f.b);
  }
  const int b = __builtin_amdgcn_readfirstlane(f.b), splits = __builtin_amdgcn_readfirstlane(f.splits);
  const Span sp = span_at(a, __builtin_amdgcn_readfirstlane(f.len));
  const int each = (sp.n + splits - 1) / splits, mine = (int)unit - f.first;
  const int gs = __builtin_amdgcn_readfirstlane(sp.g0 + min(mine * each, sp.n));
  const int ge = __builtin_amdgcn_readfirstlane(sp.g0 + min((mine + 1) * each, sp.n));

  // This tile's query heads: column j is head kvh * G + tile * 16 + j.
  const int heads = min(a.heads, a.G - tile * 16);
  const int head0 = kvh * a.G + tile * 16;

  // Group g's bytes.  A page outside the cache stands for absent tokens: page
  // 0 is read in its place and given no weight.
  constexpr int kKG = kv::group_bytes(KK, NB), kVG = kv::group_bytes(VK, NB);
  constexpr int kKB = kv::block_code_bytes(KK), kVB = kv::block_code_bytes(VK);
  // (Page numbers come through scalar loads: a vector load of one would wait
  // for every key and value load before it.)
  const auto *table = (const __attribute__((address_space(4))) int32_t *)(a.table + (int64_t)b * a.max_pages);
  Raw<KK> kr[NB];
  Raw<VK> vr[NB];
  half8 kd[KK == C_F16 ? 1 : NB], vd[VK == C_F16 ? 1 : NB];
  auto load_keys = [&](int page, int in_page) {
    const uint8_t *p = a.kp + page * a.k_page_bytes + (int64_t)in_page * kKG;
#pragma unroll
    for (int n = 0; n < NB; ++n) load_block<KK>(p + n * kKB, lane, kr[n]);
    if constexpr (KK != C_F16) {
#pragma unroll
      for (int n = 0; n < NB; ++n) kd[n] = *(const half8 *)(p + NB * kKB + n * 64 + G * 16);
    }
  };
  auto load_values = [&](int page, int in_page) {
    const uint8_t *p = a.vp + page * a.v_page_bytes + (int64_t)in_page * kVG;
    if constexpr (VK != C_F16) {
#pragma unroll
      for (int n = 0; n < NB; ++n) vd[n] = *(const half8 *)(p + NB * kVB + n * 64 + G * 16);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) load_block<VK>(p + n * kVB, lane, vr[n]);
  };
  auto usable = [&](int page) { return page >= 0 && page < a.n_pages; };
  // This wave's groups: g, then every fourth.  (pi, gi) is the page table's
  // entry and the group in its page of the group two steps ahead (past the end
  // the last one again), whose page number is read that early.
  int g = gs + wave, page = 0, in_page = 0, pi = 0, gi = 0, gn = g, page_next = 0, in_next = 0;
  bool there = false;
  auto advance = [&] {
    if (gn + kWaves < ge) {
      gn += kWaves;
      gi += kWaves;
      while (gi >= a.page_groups) gi -= a.page_groups, ++pi;
    }
  };
  if (g < ge) {
    pi = g / a.page_groups, gi = g - pi * a.page_groups;
    page = table[pi], in_page = kvh * a.page_groups + gi;
    advance();
    page_next = table[pi], in_next = kvh * a.page_groups + gi;
    there = usable(page);
    page = there ? page : 0;
    load_keys(page, in_page);
    load_values(page, in_page);
  }

  // The query scaled by a power of two to 2^14 .. 2^15, in one or two terms,
  // and what undoes it; the sign of the scale goes into the query, so that
  // the largest product is the largest score.  (f16 queries beside f16 keys
  // need no scaling: their products are exact.)
  half8 qh[NB], ql[SPLIT ? NB : 1];
  floatx4 qoff[SUB ? NB : 1];
  float qscale = a.scale2 == 0.0f ? 1.0f : fabsf(a.scale2);
  {
    const QT *q = (const QT *)a.q + (int64_t)b * a.q_stride + (int64_t)(head0 + min(j % COLS, heads - 1)) * D;
    const float sign = a.scale2 > 0.0f ? 1.0f : a.scale2 < 0.0f ? -1.0f : 0.0f;
    float up = sign;
    float v[NB][8];
#pragma unroll
    for (int n = 0; n < NB; ++n) load_q<KK>(q + n * 32, G, v[n]);
    if constexpr (KK != C_F16 || SPLIT) {
      float big = 0.0f;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(v[n][k]));
      big = max_over_groups(big);
      // 2^e brings big to [2^14, 2^15); the exponents kept where 2^e and 2^-e are normal.
      int e = 14 + 127 - (int)(__builtin_bit_cast(uint32_t, big) >> 23);
      e = big > 0.0f && big < __builtin_inff() ? min(max(e, -113), 125) : 0;
      up *= __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
      qscale *= __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
      if constexpr (SUB) qscale *= 0x1p24f;
      // Products lie below 2^42 and differ by 2^-32 or more: past these limits
      // all scores are 0, or all but the largest far below it, as without
      // them, and none overflows.
      qscale = fminf(fmaxf(qscale, 0x1p-126f), 0x1p80f);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool high = KK == C_Q4_0 && SUB && (k & 2);
        const float w = v[n][k] * (high ? up * 0.0625f : up);
        const _Float16 h = (_Float16)w;
        qh[n][k] = h;
        float got = (float)h;
        if constexpr (SPLIT) {
          const _Float16 l = (_Float16)(w - got);
          ql[n][k] = l;
          got += (float)l;
        }
        sum += high ? 16.0f * got : got;
      }
      if constexpr (SUB) {
        const float off = sum_over_groups(sum) * (KK == C_Q8_0 ? -128.0f : -8.0f) * 0x1p-24f;
        qoff[n] = floatx4{off, off, off, off};
      }
    }
  }

  // Of 16 columns a lane's accumulators are elements 4G .. 4G + 3 of column j, of
  // four the elements 4 (j / 4) .. + 3 of column j % 4, over the tokens of the
  // lane group alone.
  floatx4 acc[NB][2];
#pragma unroll
  for (int n = 0; n < NB; ++n) acc[n][0] = acc[n][1] = floatx4{0, 0, 0, 0};
  float R = kFloor, sum = 0.0f, rest = 0.0f;  // weights' sum: sum + rest
  const Nibbles nb;

  // This wave's part in LDS, to which the accumulators are added every kAdds
  // groups; they keep what that addition rounds off.  Of four columns a lane
  // stores, of the sums over the lane groups, elements 2 (G / 2) and 1 more of its
  // four, of tile G % 2.
  constexpr int kAdds = SPLIT ? 32 : 64;
  constexpr int kOwn = COLS == 16 ? 4 : 2;
  typedef float own_t __attribute__((ext_vector_type(kOwn)));
  float *ml = lds + kWaves * a.heads * kPitch;  // [part][heads][2]: reference and sum
  float *own = lds + (wave * a.heads + j % COLS) * kPitch + (COLS == 16 ? 4 * G : j / 4 * 4 + G / 2 * 2 + G % 2 * 16);
  const bool stores = j % COLS < heads;
  float R_part = kFloor;
  bool started = false;
  auto add_part = [&] {
    const float f = __builtin_amdgcn_exp2f(R_part - R);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      own_t add[COLS == 16 ? 2 : 1];
      if constexpr (COLS == 16) {
        add[0] = acc[n][0] * kUnit, add[1] = acc[n][1] * kUnit;
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float low = sum_of_rows(acc[n][0][r], acc[n][1][r]), high = sum_of_rows(acc[n][0][r + 2], acc[n][1][r + 2]);
          add[0][r] = sum_of_halves(low, high) * kUnit;
        }
      }
#pragma unroll
      for (int x = 0; x < (COLS == 16 ? 2 : 1); ++x) {
        own_t *o = (own_t *)(own + n * 32 + x * 16);
        own_t left = {};
        if (!started) {
          if (stores) *o = add[x];
        } else if (stores) {
          const own_t old = *o * f, now = old + add[x];
          *o = now;
          left = (add[x] - (now - old)) * (1.0f / kUnit);
        }
        if constexpr (COLS == 16) {
          acc[n][x] = left;
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[n][k >> 2][k & 3] = G == ((k & 2) | k >> 2) ? left[k & 1] : 0.0f;
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // (few blocks at a time: registers)
    }
    R_part = R;
    started = true;
  };

  do {
    const int stop = min(ge, g + kAdds * kWaves);
    while (g < stop) {
      // The next group's keys load as soon as this one's are used, its values
      // likewise (after the last group once more the last: the loads are issued
      // whatever follows, so that no wait is widened by a branch).
      advance();
      const int page_after = table[pi], in_after = kvh * a.page_groups + gi;

      // Products of tokens 8G + k with head j, without the query's scale.
      float s[8];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        floatx4 t = {0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const half8 k = key_operand<KK, SPLIT>(kr[n], m, nb);
          floatx4 u;
          if constexpr (KK == C_F16) u = t;
          else if constexpr (SUB) u = qoff[n];
          else u = floatx4{0, 0, 0, 0};
          u = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qh[n], u, 0, 0, 0);
          if constexpr (SPLIT) u = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, ql[n], u, 0, 0, 0);
          if constexpr (KK == C_F16) t = u;
          else
#pragma unroll
            for (int r = 0; r < 4; ++r) t[r] = __builtin_fmaf((float)kd[n][4 * m + r], u[r], t[r]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) s[4 * m + r] = t[r];
      }
      const bool there_next = usable(page_next);
      const int next = there_next ? page_next : 0;
      load_keys(next, in_next);

      // Tokens outside [lo, len) of the first and last group: whatever their
      // bytes hold, they weigh nothing.
      const int t0 = g * kv::kGroup;
      if (t0 < sp.lo || t0 > sp.len - kv::kGroup || !there) {
        bool in[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int t = t0 + 8 * G + k;
          in[k] = there && t >= sp.lo && t < sp.len;
          if (!in[k]) s[k] = -__builtin_inff();
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if constexpr (VK == C_F16) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                vr[n].w[x][k] &= (in[2 * k] ? 0xffffu : 0u) | (in[2 * k + 1] ? 0xffff0000u : 0u);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) vd[n][k] = in[k] ? vd[n][k] : (_Float16)0.0f;
          }
        }
      }

      // The reference: per lane (its eight tokens) the largest score and (f16
      // weights) the exponent of the largest value scale, then over the lanes of
      // the column.
      float top = s[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) top = fmaxf(top, s[k]);
      top *= qscale;
      float below = SPLIT ? 40.0f : 14.0f;  // f16 weights: 14 - the exponent of the largest value scale
      if constexpr (VK != C_F16 && !SPLIT) {
        // Magnitudes of halves compare as integers (Q8_0 scales have no sign).
        ushort2v part[4] = {{0, 0}, {0, 0}, {0, 0}, {0, 0}};
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const u32x4 w = __builtin_bit_cast(u32x4, vd[n]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            part[k] = __builtin_elementwise_max(part[k], as_us2(VK == C_Q4_0 ? w[k] & 0x7fff7fffu : w[k]));
        }
        ushort2v most = __builtin_elementwise_max(__builtin_elementwise_max(part[0], part[1]),
                                                  __builtin_elementwise_max(part[2], part[3]));
        // A NaN scale (a block that held an infinity or NaN) leaves the other
        // blocks' reference alone.
        if (__any(max(most[0], most[1]) >= 0x7c00)) {
          most = ushort2v{0, 0};
          for (int n = 0; n < NB; ++n)
            for (int k = 0; k < 8; ++k) {
              const uint16_t m = __builtin_bit_cast(uint16_t, (_Float16)vd[n][k]) & 0x7fff;
              if (m < 0x7c00) most[0] = max(most[0], m);
            }
        }
        const half2v big = as_h2(as_u(most));
        // 2^e <= scale < 2^(e + 1); f16 scales are 0 or at least 2^-24.
        const float bf = fmaxf(fmaxf((float)big[0], (float)big[1]), 0x1p-24f);
        below = (float)(127 + 14 - (int)(__builtin_bit_cast(uint32_t, bf) >> 23));
      }
      // (Among scores whose f32 neighbours lie further apart than `below` means,
      // the reference is the score itself: weights up to 1, not 2^14 or 2^40.)
      top = fabsf(top) < kFar ? top - below : top;
      top = max_over_groups(top);
      if (__any(top > R)) {  // rare after the first groups
        const float Rn = fmaxf(R, top), alpha = __builtin_amdgcn_exp2f(R - Rn);
        R = Rn;
        sum *= alpha;
        rest *= alpha;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) acc[n][x] *= alpha;
      }
      float p[8];
      if (__any(fabsf(R) >= kFar)) {
        // The score rounded as the reference was: what the product's rounding
        // leaves, itself large here, must not become a weight.
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = __builtin_amdgcn_exp2f(kv::in_f32(s[k] * qscale) - R);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k], qscale, -R));
      }
      const float eight = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7])), before = sum;
      sum += eight;
      rest += eight - (sum - before);

      if constexpr (SPLIT && VK == C_F16) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float v = (float)as_h8(vr[n].w[x])[k];
              if constexpr (COLS == 16)  // K entries: token k of each lane group
                acc[n][x] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, p[k], acc[n][x], 0, 0, 0);
              else  // sixteen products of the four lanes that share j / 4 and G
                acc[n][x] = __builtin_amdgcn_mfma_f32_4x4x1f32(v, p[k], acc[n][x], 0, 0, 0);
            }
          }
        }
      } else if constexpr (SPLIT) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          float w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = __builtin_fmaf(p[k], (float)vd[n][k], 0.0f);  // one v_fma_mix
          // The weight's 24 bits, eight to a term: each cut off, the rest exact.
          bf16x8 term[3];
#pragma unroll
          for (int t = 0; t < 3; ++t) {
            u32x4 u;
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = upper_halves(w[2 * k], w[2 * k + 1]);
            term[t] = __builtin_bit_cast(bf16x8, u);
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] -= __builtin_bit_cast(float, bits_of(w[k]) & 0xffff0000u);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const bf16x8 v = value_bf16<VK>(vr[n], x);
#pragma unroll
            for (int t = 2; t >= 0; --t) acc[n][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, term[t], acc[n][x], 0, 0, 0);
          }
        }
      } else {
        half8 ph;
        if constexpr (VK == C_F16) {
#pragma unroll
          for (int k = 0; k < 8; ++k) ph[k] = (_Float16)p[k];
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if constexpr (VK != C_F16) {
#pragma unroll
            for (int k = 0; k < 8; ++k)  // one v_fma_mix each
              ph[k] = (_Float16)__builtin_fmaf(p[v_token<VK>(k)], (float)vd[n][v_token<VK>(k)], 0.0f);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
            acc[n][x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value_operand<VK>(vr[n], x, nb), ph, acc[n][x], 0, 0, 0);
        }
      }
      load_values(next, in_next);
      there = there_next;
      page_next = page_after, in_next = in_after;
      g += kWaves;
    }
    add_part();
  } while (g < ge);
  sum = sum_over_groups(sum + rest);

  // The four waves' parts, joined through LDS with their references.
  if (G == 0 && j < heads) {
    ml[(wave * a.heads + j) * 2] = R;
    ml[(wave * a.heads + j) * 2 + 1] = sum;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < heads * (D / 4); i += 64 * kWaves) {
    const int h = i / (D / 4), d = i % (D / 4) * 4;
    float Rm = kFloor, l = 0.0f;
    for (int w = 0; w < kWaves; ++w) Rm = fmaxf(Rm, ml[(w * a.heads + h) * 2]);
    floatx4 o = {0, 0, 0, 0};
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(ml[(w * a.heads + h) * 2] - Rm);
      l = __builtin_fmaf(f, ml[(w * a.heads + h) * 2 + 1], l);
      o += *(const floatx4 *)(lds + (w * a.heads + h) * kPitch + d) * f;
    }
    if (splits == 1) {
      store_out((QT *)a.out + ((int64_t)b * a.n_q + head0 + h) * D + d, o, l, Rm, a.sinks, head0 + h);
    } else {
      const int64_t part = (int64_t)blockIdx.x * a.heads + h;
      *(floatx4 *)(a.part + part * D + d) = o;
      if (d == 0) {
        float *m = a.part + a.items * a.heads * D + part * 2;
        m[0] = Rm;
        m[1] = l;
      }
    }
  }
}

hipError_t launch_plan(const Args &a, hipStream_t s);

// How many workgroups the GPU holds is looked up once per instantiation and
// device (with the most LDS a call uses).
template <int KK, int VK, int NB, typename QT, int COLS>
static hipError_t run_cols(Args &a, hipStream_t s) {
  static std::atomic<int> slots[64];
  auto *kernel = attn_kernel<KK, VK, NB, QT, COLS>;
  auto lds = [](int heads) { return (unsigned)(kWaves * (NB * 32 + 4 + 2) * heads * sizeof(float)); };  // <= 66 KiB
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
  a.slots = slots[dev].load(std::memory_order_relaxed);
  if (a.slots == 0) {
    int n = 0;
    e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds(COLS));
    if (e != hipSuccess) return e;
    e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 64 * kWaves, lds(COLS));
    if (e != hipSuccess) return e;
    a.slots = std::min(std::max(n, 1) * device_cus(), kMaxSlots);
    slots[dev].store(a.slots, std::memory_order_relaxed);
  }
  // Splits of the longest sequences the page table can hold, and of any batch.
  const int64_t nh = a.n_kv * a.tiles, most = a.max_pages * a.page_groups;
  a.items = std::min(2 * a.slots + a.B * nh, a.B * nh * ((most + kMinGroups - 1) / kMinGroups));
  if (a.B > kLanes) {
    e = launch_plan(a, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)a.items), dim3(64 * kWaves), lds(a.heads), s, a);
  return hipGetLastError();
}

template <int KK, int VK, int NB, typename QT>
static hipError_t run(Args &a, hipStream_t s) {
  if constexpr (sizeof(QT) == 4 && VK == C_F16) {
    if (a.heads <= 4) return run_cols<KK, VK, NB, QT, 4>(a, s);
  }
  return run_cols<KK, VK, NB, QT, 16>(a, s);
}

template <int KK, int VK, typename QT>
static hipError_t run_nb(Args &a, int NB, hipStream_t s) {
  switch (NB) {
    case 2: return run<KK, VK, 2, QT>(a, s);
    case 3: return run<KK, VK, 3, QT>(a, s);
    case 4: return run<KK, VK, 4, QT>(a, s);
    case 6: return run<KK, VK, 6, QT>(a, s);
    case 8: return run<KK, VK, 8, QT>(a, s);
  }
  return hipErrorInvalidValue;
}

template <int KK, int VK>
static hipError_t run_kinds(Args &a, int NB, int f16, hipStream_t s) {
  return f16 ? run_nb<KK, VK, _Float16>(a, NB, s) : run_nb<KK, VK, float>(a, NB, s);
}

hipError_t launch_f16_f16(Args &, int NB, int f16, hipStream_t);
hipError_t launch_f16_q8(Args &, int NB, int f16, hipStream_t);
hipError_t launch_f16_q4(Args &, int NB, int f16, hipStream_t);
hipError_t launch_q8_f16(Args &, int NB, int f16, hipStream_t);
hipError_t launch_q8_q8(Args &, int NB, int f16, hipStream_t);
hipError_t launch_q8_q4(Args &, int NB, int f16, hipStream_t);
hipError_t launch_q4_f16(Args &, int NB, int f16, hipStream_t);
hipError_t launch_q4_q8(Args &, int NB, int f16, hipStream_t);
hipError_t launch_q4_q4(Args &, int NB, int f16, hipStream_t);

}  // namespace attn
}  // namespace qmm
