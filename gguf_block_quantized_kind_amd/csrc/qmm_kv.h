// qmm_kv.h -- the paged key/value cache: where its bytes lie, and the block
// quantizer and rotation shared by the kernels that write it.
//
// A page holds page_size tokens of n_kv heads; page_size is a multiple of 32
// and the unit is a group of 32 consecutive tokens of one head:
//
//   page = [head][page_size / 32 groups], group = codes, then scales
//   codes  NB = head_dim / 32 blocks of 32 elements x 32 tokens, each laid
//          out as the lanes of v_mfma_f32_16x16x32_f16 read it (below)
//   scales (Q8_0, Q4_0) f16 [NB][32 tokens]
//
// so a group is 32 * qmm_row_bytes-like bytes (2, 34/32 or 18/32 bytes per
// element) and every byte of it is read by whole 8- or 16-byte lane loads.
//
// In a key block the matrix-core rows are tokens and its K dimension the
// elements; in a value block the rows are elements and K the tokens.  Lane
// (i, G) of a wave (i = lane % 16, G = lane / 16) holds, of row i, the K
// entries 8G .. 8G + 7 (Q4_0 keys: the elements 4G .. 4G + 3 and 16 + those,
// two to a byte).  There are two row tiles per block:
//   keys    tile m, row i = token 8 (i / 4) + 4 m + i % 4, so that the rows
//           4G + r of a lane's score registers are tokens 8G + 4m + r: the
//           eight tokens whose weights the same lane supplies as the K
//           entries of the value product, with no movement between lanes;
//   values  tile x, row j = element 16 x + j.
//   F16     [tile][G][row][8] halves           1024 bytes per tile
//   Q8_0    [G][row][tile][8] bytes, code + 128
//   Q4_0    keys [G][row][tile][4] bytes, byte y = elements 4G + y (low
//           nibble) and 16 + 4G + y (high); values [G][row][8 tokens] bytes,
//           elements row (low) and 16 + row (high); codes 0 .. 15 = value / d + 8
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm_internal.h"

namespace qmm {
namespace kv {

// Cache kinds by GGUF type id.
enum CacheKind : int { C_F16 = 1, C_Q4_0 = 2, C_Q8_0 = 8 };

constexpr int kGroup = 32;  // tokens per group

// Bytes of one block (32 elements x 32 tokens) without its scales, and of a
// group of NB blocks with them.
__host__ __device__ constexpr int block_code_bytes(int kind) {
  return kind == C_F16 ? 2048 : kind == C_Q8_0 ? 1024 : 512;
}
__host__ __device__ constexpr int group_bytes(int kind, int NB) {
  return NB * (block_code_bytes(kind) + (kind == C_F16 ? 0 : 64));
}

// Byte of (block b, token r of the group, element c of the block) in a group;
// Q4_0: the byte holding it (nibble c / 16).
template <int KIND, bool IS_V>
__device__ __forceinline__ int code_offset(int b, int r, int c) {
  const int base = b * block_code_bytes(KIND);
  if constexpr (!IS_V) {
    const int i = 4 * (r >> 3) + (r & 3), m = (r >> 2) & 1;
    if constexpr (KIND == C_F16) return base + ((m * 4 + (c >> 3)) * 16 + i) * 16 + (c & 7) * 2;
    if constexpr (KIND == C_Q8_0) return base + (((c >> 3) * 16 + i) * 2 + m) * 8 + (c & 7);
    return base + ((((c & 15) >> 2) * 16 + i) * 2 + m) * 4 + (c & 3);
  } else {
    const int G = r >> 3, e = r & 7;
    if constexpr (KIND == C_F16) return base + (((c >> 4) * 4 + G) * 16 + (c & 15)) * 16 + e * 2;
    if constexpr (KIND == C_Q8_0) return base + ((G * 16 + (c & 15)) * 2 + (c >> 4)) * 8 + e;
    return base + (G * 16 + (c & 15)) * 8 + e;
  }
}
__device__ __forceinline__ int scale_offset(int kind, int NB, int b, int r) {
  return NB * block_code_bytes(kind) + (b * kGroup + r) * 2;
}

// The smallest f16 not below d >= 0, at most 65504 (rounding the step up keeps
// every code in its range, so the error of a code is at most half a step).
__device__ __forceinline__ _Float16 f16_up(float d) {
  _Float16 h = (_Float16)fminf(d, 65504.0f);
  if ((float)h < d && (float)h < 65504.0f)
    h = __builtin_bit_cast(_Float16, (uint16_t)(__builtin_bit_cast(uint16_t, h) + 1));
  return h;
}

// The scale of a block from the bits of its largest |x| and (Q4_0) its largest
// x.  An infinity or NaN shows in the bits: such a block gets a NaN scale and
// reads back as NaN throughout.
template <int KIND>
__device__ __forceinline__ _Float16 block_scale(float hi, uint32_t bits) {
  if (bits >= 0x7f800000u) return __builtin_bit_cast(_Float16, (uint16_t)0x7e00);
  const float big = __builtin_bit_cast(float, bits);
  if constexpr (KIND == C_Q8_0) {  // big / 127, correctly rounded as in encode
    const float inv = 1.0f / 127.0f, q = big * inv;
    return f16_up(__builtin_fmaf(__builtin_fmaf(-127.0f, q, big), inv, q));
  }
  const _Float16 h = f16_up(big * 0.125f);
  return hi == big && big != 0.0f ? -h : h;  // the extreme element becomes code 0: -8 d
}

// The bits of |x|: above 0x7f7fffff for an infinity or NaN.  (A function: a bit
// cast of a vector's element in place reads the vector's first element.)
__device__ __forceinline__ uint32_t magnitude_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// A block's step and its reciprocal, each correctly rounded (both 0 where
// every code is that of zero: a zero or NaN scale, whose elements are taken as
// zeros).
struct Step {
  float d, inv;
};
__device__ __forceinline__ Step step_of(_Float16 h) {
  const float d = (float)h;
  const bool none = d == 0.0f || d != d;
  return Step{none ? 0.0f : d, none ? 0.0f : 1.0f / d};
}

// The stored code of x (an integer in f32; the caller's conversion to a byte
// cuts it at 0 and 255): the nearest integer to the correctly rounded x / d,
// ties to even.  With inv the correctly rounded 1 / d, one residual step makes
// the quotient correctly rounded (Markstein, IBM J. Res. Dev. 34, 1990): three
// operations an element instead of a division's dozen.
template <int KIND>
__device__ __forceinline__ float encode(float x, Step st) {
  const float q0 = x * st.inv;
  const float q = rintf(__builtin_fmaf(__builtin_fmaf(-st.d, q0, x), st.inv, q0));
  return KIND == C_Q8_0 ? fmaxf(q, -127.0f) + 128.0f : fminf(q + 8.0f, 15.0f);
}

// A constant in scalar registers (in a loop the compiler would keep it in vector
// registers, and so waves off the GPU).
__device__ __forceinline__ double uniform(double v) {
  asm("" : "+s"(v));
  return v;
}

// m cos and m sin of pos * freq (radians per position), computed in 64 bits and
// rounded once.  (A 32-bit angle at position 10^6 would already be off by 0.06, and
// a 64-bit product costs what a 32-bit one does here.)  The angle is reduced to an
// eighth of a turn; there the Taylor series' first omitted terms are below 1e-11.
__device__ __forceinline__ void rotation(int pos, double freq, float m, float &c, float &s) {
  double t = (double)pos * freq * 0.15915494309189533577;  // turns
  t -= rint(t);
  const double q = rint(4.0 * t);
  const double x = (t - 0.25 * q) * 6.283185307179586477, z = x * x;
  double sp = __builtin_fma(z, uniform(-1.0 / 39916800), 1.0 / 362880);
  sp = __builtin_fma(z, sp, uniform(-1.0 / 5040));
  sp = __builtin_fma(z, sp, uniform(1.0 / 120));
  sp = __builtin_fma(z, sp, uniform(-1.0 / 6));
  sp = __builtin_fma(z * x, sp, x);
  double cp = __builtin_fma(z, uniform(1.0 / 479001600), -1.0 / 3628800);
  cp = __builtin_fma(z, cp, uniform(1.0 / 40320));
  cp = __builtin_fma(z, cp, uniform(-1.0 / 720));
  cp = __builtin_fma(z, cp, uniform(1.0 / 24));
  cp = __builtin_fma(z, cp, -0.5);
  cp = __builtin_fma(z, cp, 1.0);
  const int k = (int)q & 3;
  const float a = (float)((k & 1 ? sp : cp) * m), b = (float)((k & 1 ? cp : sp) * m);
  c = (k == 1 || k == 2) ? -a : a;
  s = (k & 2) ? -b : b;
}

// The members of a rotated pair, by the same operations wherever they are
// computed, rounded to f32 before any narrower type: a result does not depend
// on the alignment of its row.  (Without the barrier the compiler rounds some
// of them from the exact sum to f16.)
__device__ __forceinline__ float in_f32(float x) {
  asm("" : "+v"(x));
  return x;
}
__device__ __forceinline__ float turned_a(float u, float v, float c, float s) {
  return in_f32(__builtin_fmaf(u, c, -(v * s)));
}
__device__ __forceinline__ float turned_b(float u, float v, float c, float s) {
  return in_f32(__builtin_fmaf(u, s, v * c));
}

struct Rope {
  const double *freqs;  // n_rot / 2 radians per position
  int n_rot;
  int interleaved;
  float mscale;
};

struct Cache {
  uint8_t *k_pages, *v_pages;
  int64_t n_slots;  // n_pages * page_size
  int page_size, page_shift;  // shift: log2 of a power of two, else -1
  int n_kv, NB;
};

// Rotation of whole rows, V pairs of every head of a range per thread: the
// angle costs about sixty operations (half of them 64-bit), so each is used
// for as many heads as leave the grid full.
struct Rotate {
  const void *x;
  void *y;
  int64_t x_stride, y_stride;
  const int32_t *pos;
  int64_t T;
  int H, D, per;       // heads per thread
  int chunks, ranges;  // D / 2 / V, ceil(H / per)
  Rope rope;
};
template <typename T, int V>
struct Vec {
  typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T>
struct Vec<T, 1> {
  struct type {
    T v;
    __device__ __forceinline__ T &operator[](int) { return v; }
  };
};
template <typename T, typename O, int V>
__device__ __forceinline__ void rotate_rows(const Rotate &r, int64_t i) {
  using X = typename Vec<T, V>::type;
  using Y = typename Vec<O, V>::type;
  const uint32_t per_token = (uint32_t)(r.chunks * r.ranges), t32 = (uint32_t)i / per_token;  // (fewer than 2^32 threads)
  const int64_t t = t32;
  if (t >= r.T) return;
  const int rest = (int)((uint32_t)i - t32 * per_token), range = rest / r.chunks, p = (rest - range * r.chunks) * V;
  const int half = r.rope.n_rot >> 1;
  const bool turned = p < half, split = turned && !r.rope.interleaved;
  // Elements [da, da + V) and [db, db + V): the two members of V pairs, or (interleaved, passing) 2 V neighbours.
  const int da = split ? p : 2 * p, db = split ? p + half : 2 * p + V;
  float c[V], s[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    c[k] = 1.0f;
    s[k] = 0.0f;
    if (turned) rotation(r.pos[t], r.rope.freqs[p + k], r.rope.mscale, c[k], s[k]);
  }
  const int h1 = min(r.H, (range + 1) * r.per);
  const T *x = (const T *)r.x + t * r.x_stride;
  O *y = (O *)r.y + t * r.y_stride;
  for (int h = range * r.per; h < h1; ++h) {
    X a, b;
    __builtin_memcpy(&a, __builtin_assume_aligned(x + (int64_t)h * r.D + da, sizeof(X)), sizeof(X));
    __builtin_memcpy(&b, __builtin_assume_aligned(x + (int64_t)h * r.D + db, sizeof(X)), sizeof(X));
    Y u, v;
    if (!turned) {
#pragma unroll
      for (int k = 0; k < V; ++k) u[k] = (O)(float)a[k], v[k] = (O)(float)b[k];
    } else if (split) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        u[k] = (O)turned_a((float)a[k], (float)b[k], c[k], s[k]);
        v[k] = (O)turned_b((float)a[k], (float)b[k], c[k], s[k]);
      }
    } else if constexpr (V == 1) {
      u[0] = (O)turned_a((float)a[0], (float)b[0], c[0], s[0]);
      v[0] = (O)turned_b((float)a[0], (float)b[0], c[0], s[0]);
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        u[k] = (O)turned_a((float)a[k], (float)a[k + 1], c[k / 2], s[k / 2]);
        u[k + 1] = (O)turned_b((float)a[k], (float)a[k + 1], c[k / 2], s[k / 2]);
        v[k] = (O)turned_a((float)b[k], (float)b[k + 1], c[(V + k) / 2], s[(V + k) / 2]);
        v[k + 1] = (O)turned_b((float)b[k], (float)b[k + 1], c[(V + k) / 2], s[(V + k) / 2]);
      }
    }
    __builtin_memcpy(__builtin_assume_aligned(y + (int64_t)h * r.D + da, sizeof(Y)), &u, sizeof(Y));
    __builtin_memcpy(__builtin_assume_aligned(y + (int64_t)h * r.D + db, sizeof(Y)), &v, sizeof(Y));
  }
}

// The same by q_out's type and the width, known at run time.
template <typename T>
__device__ __forceinline__ void rotate_any(const Rotate &r, int out_f16, int wide, int64_t i) {
  if (out_f16) wide ? rotate_rows<T, _Float16, 4>(r, i) : rotate_rows<T, _Float16, 1>(r, i);
  else wide ? rotate_rows<T, float, 4>(r, i) : rotate_rows<T, float, 1>(r, i);
}

// Fills in the split of T rows of H heads; four pairs a thread where every
// vector they make is aligned, else one.
inline bool plan_rotate(Rotate &r, int x_bytes, int y_bytes, int64_t &threads) {
  const int v = 4;
  const bool wide = r.D % (2 * v) == 0 && r.rope.n_rot % (2 * v) == 0 && r.x_stride % v == 0 && r.y_stride % v == 0 &&
                    (uintptr_t)r.x % (v * x_bytes) == 0 && (uintptr_t)r.y % (v * y_bytes) == 0;
  r.chunks = r.D / 2 / (wide ? v : 1);
  // Heads per thread: one until the grid holds eight waves per SIMD.
  const int64_t one = r.T * r.chunks * r.H, full = (int64_t)device_cus() * 4 * 8 * 64;
  r.per = (int)(one / full < 1 ? 1 : one / full > r.H ? r.H : one / full);
  r.ranges = (r.H + r.per - 1) / r.per;
  threads = r.T * r.chunks * r.ranges;
  return wide;
}

}  // namespace kv
}  // namespace qmm
