// qmm_kv.hip -- writing new tokens into the paged key/value cache (quantized
// to its kind, with or without the rotation of the keys and queries) and
// reading tokens back.  Layout and quantizer: qmm_kv.h.
//
// A wave works by itself on eight tokens of one head's keys or values, through
// its own rows of LDS (rows lie along the elements, cache units across
// tokens), and goes on to further heads while the next head's rows load:
//   write  rows -> LDS (f32; rotated there), block scales, then every lane
//          encodes the elements of one cache unit and stores it: 16, 8 or 4
//          bytes of one key token, or eight tokens of an element pair of the
//          values.
//   read   the reverse; keys need no LDS, a unit of theirs being a run of one
//          row's elements.
// A value unit holds eight tokens whose slots are consecutive from a multiple
// of eight.  Such octets are found wherever they start among the call's
// tokens: a wave takes the octet that starts within its eight tokens, and then
// those of its tokens that no octet covers (other sequences' single tokens,
// the ends of a prompt), byte by byte.  A prompt's tokens so fill whole units
// from any start.
//
// What bounds it: memory traffic when there is much of it, and a wave's chain of
// loads and LDS rounds when there is not.  Measured, 32768 tokens of 8 heads of
// 128 in Q4_0: f32 rows written (306 MB) in 74 us, 4.2 TB/s, read back as f16
// (172 MB) in 38 us, 4.5 TB/s; 5003 tokens, Q8_0 keys and Q4_0 values, written
// from f16 (29 MB) in 15 us and read as f32 (49 MB) in 12; with 32 query heads
// rotated, one token of 8 heads appended in 5.5 us, 8192 from f32 to Q8_0 (353 MB)
// in 90, 3.9 TB/s, from f16 to Q4_0 (177 MB) in 67, 2.7 TB/s (each head's keys
// compute their angles anew).  A half wave per block of a token with
// byte stores took 420 and 230 us for the first two; windows of 32 tokens per
// workgroup, synchronized three times, 82 and 51.
#include <algorithm>
#include <type_traits>

#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {
namespace kv {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;

// Where the tokens [8 w - 8, 8 w + 16) lie: lane L has token 8 w - 8 + L.
struct Places {
  int slot;      // -1: skipped, or not a token of the call
  int r;         // token of its group
  int64_t base;  // first byte of head 0's group of the token
  // Lanes of the octet that starts at one of the wave's own tokens (0: none),
  // and of its own tokens that no octet covers.
  int octet;
  uint32_t rest;
};

__device__ __forceinline__ Places find_places(const Cache &c, int kind, const int32_t *slots, int64_t w, int64_t T) {
  Places p;
  const int lane = threadIdx.x & 63;
  const int64_t t = 8 * w - 8 + lane;
  const bool token = lane < 24 && t >= 0 && t < T;
  int slot = token ? slots[t] : -1;
  slot = slot < c.n_slots ? max(slot, -1) : -1;
  const int page = c.page_shift >= 0 ? max(slot, 0) >> c.page_shift : max(slot, 0) / c.page_size;
  const int at = max(slot, 0) - page * c.page_size;
  p.slot = slot;
  p.r = at % kGroup;
  p.base = ((int64_t)page * c.n_kv * (c.page_size / kGroup) + at / kGroup) * group_bytes(kind, c.NB);
  // Octets: a slot at a multiple of eight followed by its seven neighbours
  // (pages are whole groups, so an octet never leaves its group).  Two cannot
  // start within eight tokens.
  const uint32_t next = (uint32_t)__ballot(slot >= 0 && __shfl_down(slot, 1, 64) == slot + 1);
  const uint32_t two = next & next >> 1, four = two & two >> 2;
  const uint32_t start = (uint32_t)__ballot(slot >= 0 && slot % 8 == 0) & four & four >> 3 & 0xffff;
  const uint32_t before = start & 0xff, own = start & 0xff00;
  uint32_t covered = before ? 0xffu << (__ffs(before) - 1) : 0;
  if (own) covered |= 0xffu << (__ffs(own) - 1);
  p.octet = own ? __ffs(own) - 1 : 0;
  p.rest = (uint32_t)__ballot(token) & 0xff00 & ~covered;
  return p;
}
__device__ __forceinline__ int64_t lane_of(int64_t v, int lane) {
  return (int64_t)(uint32_t)__shfl((int)v, lane, 64) | (int64_t)__shfl((int)(v >> 32), lane, 64) << 32;
}

// The lane number, whose uses the compiler does not move out of the loop over
// the heads: kept addresses of every kind's path would cost registers, and so
// waves.
__device__ __forceinline__ int fresh_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// LDS written by some lanes of the wave is read by others after this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename T>
__device__ __forceinline__ floatx4 load4(const T *x, bool vec) {
  if (vec) {
    typename Vec<T, 4>::type v;
    __builtin_memcpy(&v, __builtin_assume_aligned(x, 4 * sizeof(T)), sizeof v);
    return floatx4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
  }
  return floatx4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
}

__device__ __forceinline__ uint32_t pack_h(float a, float b) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
}

// One byte of a code at place k of w.
__device__ __forceinline__ uint32_t put(uint32_t w, int k, float code) {
  return __builtin_amdgcn_cvt_pk_u8_f32(code, k, w);
}

// Eight tokens being written or read: lanes first .. first + 7 of the places,
// those in `mask`.
struct Eight {
  int first;
  uint32_t mask;
  bool whole;  // an octet
};

// A token's group and place in it, as offsets from head 0's first group.
struct Spot {
  int64_t base;
  int r;
};
__device__ __forceinline__ Spot spot_of(const Places &p, int lane) {
  return Spot{lane_of(p.base, lane), __shfl(p.r, lane, 64)};
}

// Block scales, four lanes per (token (lane / 4) % 8, block) with eight
// elements each: stored in the cache, and as steps for the encoding.
template <int KIND, int NB>
__device__ __forceinline__ void write_scales(uint8_t *head, const Spot &at, const Eight &g, float *rows, Step *steps) {
  constexpr int pitch = NB * 32 + 4;
  const int lane = fresh_lane(), t = (lane >> 2) & 7;
  if (!(g.mask >> t & 1)) return;  // (all four lanes)
#pragma unroll 1
  for (int b0 = 0; b0 < NB; b0 += 2) {
    const int b = b0 + (lane >> 5);
    if (b >= NB) continue;
    float *e = rows + t * pitch + b * 32 + (lane & 3) * 8;
    const floatx4 u = *(const floatx4 *)e, v = *(const floatx4 *)(e + 4);
    float hi = u[0];
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (KIND == C_Q4_0) hi = fmaxf(hi, fmaxf(u[k], v[k]));
      bits = max(bits, max(magnitude_bits(u[k]), magnitude_bits(v[k])));
    }
#pragma unroll
    for (int k = 1; k < 4; k <<= 1) {
      if constexpr (KIND == C_Q4_0) hi = fmaxf(hi, __shfl_xor(hi, k, 4));
      bits = max(bits, (uint32_t)__shfl_xor((int)bits, k, 4));
    }
    const _Float16 h = block_scale<KIND>(hi, bits);
    if (bits >= 0x7f800000u) *(floatx4 *)e = *(floatx4 *)(e + 4) = floatx4{0, 0, 0, 0};
    if ((lane & 3) == 0) {
      steps[b * 8 + t] = step_of(h);
      *(_Float16 *)(head + at.base + scale_offset(KIND, NB, b, at.r)) = h;
    }
  }
}

template <int KIND, int NB>
__device__ __forceinline__ void write_keys(uint8_t *head, const Spot &at, const Eight &g, const float *rows,
                                           const Step *steps) {
  constexpr int pitch = NB * 32 + 4;
  const int lane = fresh_lane(), t = lane & 7, r = at.r;  // `at`: of token lane % 8
  uint8_t *token = head + at.base;
  if (!(g.mask >> t & 1)) return;
#pragma unroll 1
  for (int i0 = 0; i0 < NB * 32; i0 += 64) {
    const int i = i0 + lane, G = (i >> 3) & 3, b = i >> 5;
    if (b >= NB) continue;
    const float *e = rows + t * pitch + b * 32;
    uint8_t *o = token + code_offset<KIND, false>(b, r, KIND == C_Q4_0 ? 4 * G : 8 * G);
    const floatx4 u = *(const floatx4 *)(e + (KIND == C_Q4_0 ? 4 * G : 8 * G));
    const floatx4 v = *(const floatx4 *)(e + (KIND == C_Q4_0 ? 16 + 4 * G : 8 * G + 4));
    if constexpr (KIND == C_F16) {
      *(u32x4 *)o = u32x4{pack_h(u[0], u[1]), pack_h(u[2], u[3]), pack_h(v[0], v[1]), pack_h(v[2], v[3])};
    } else {
      const Step st = steps[b * 8 + t];
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lo = put(lo, k, encode<KIND>(u[k], st));
        hi = put(hi, k, encode<KIND>(v[k], st));
      }
      if constexpr (KIND == C_Q8_0) *(u32x2 *)o = u32x2{lo, hi};
      else *(uint32_t *)o = lo | hi << 4;
    }
  }
}

template <int KIND, int NB>
__device__ __forceinline__ void write_values(uint8_t *head, const Places &p, const Spot &first, const Eight &g,
                                             const float *rows, const Step *steps) {
  constexpr int pitch = NB * 32 + 4;
  const int lane = fresh_lane(), j = lane & 15;
  if (g.whole) {
    const int r = first.r;
    uint8_t *octet = head + first.base;
#pragma unroll 1
    for (int i0 = 0; i0 < NB * 16; i0 += 64) {
      const int b = (i0 + lane) >> 4;
      if (b >= NB) continue;
      const float *e = rows + b * 32 + j;
      uint8_t *o = octet + code_offset<KIND, true>(b, r, j);
      if constexpr (KIND == C_F16) {
        u32x4 a, v;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = pack_h(e[2 * k * pitch], e[(2 * k + 1) * pitch]);
          v[k] = pack_h(e[2 * k * pitch + 16], e[(2 * k + 1) * pitch + 16]);
        }
        *(u32x4 *)o = a;
        *(u32x4 *)(o + 1024) = v;
      } else {
        uint32_t q[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const Step st = steps[b * 8 + k];
          q[k >> 2] = put(q[k >> 2], k & 3, encode<KIND>(e[k * pitch], st));
          q[2 + (k >> 2)] = put(q[2 + (k >> 2)], k & 3, encode<KIND>(e[k * pitch + 16], st));
        }
        if constexpr (KIND == C_Q8_0) *(u32x4 *)o = u32x4{q[0], q[1], q[2], q[3]};
        else *(u32x2 *)o = u32x2{q[0] | q[2] << 4, q[1] | q[3] << 4};
      }
    }
  } else {
    for (uint32_t m = g.mask; m; m &= m - 1) {
      const int t = __ffs(m) - 1, r = __builtin_amdgcn_readlane(p.r, g.first + t);
      uint8_t *token = head + lane_of(p.base, g.first + t);
#pragma unroll
      for (int i0 = 0; i0 < NB * 16; i0 += 64) {
        const int b = (i0 + lane) >> 4;
        if (b >= NB) continue;
        const float *e = rows + t * pitch + b * 32 + j;
        uint8_t *o = token + code_offset<KIND, true>(b, r, j);
        if constexpr (KIND == C_F16) {
          *(_Float16 *)o = (_Float16)e[0];
          *(_Float16 *)(o + 1024) = (_Float16)e[16];
        } else {
          const Step st = steps[b * 8 + t];
          const uint32_t q = put(put(0, 0, encode<KIND>(e[0], st)), 1, encode<KIND>(e[16], st));
          if constexpr (KIND == C_Q8_0) {
            o[0] = (uint8_t)q;
            o[8] = (uint8_t)(q >> 8);
          } else {
            o[0] = (uint8_t)(q | q >> 4);
          }
        }
      }
    }
  }
}

struct WriteArgs {
  Cache cache;
  int k_kind, v_kind;
  const void *k, *v;
  int64_t k_stride, v_stride;
  int k_vec, v_vec;
  const int32_t *pos, *slots;
  int64_t T;
  int64_t kv_wgs;   // workgroups of the cache part; the rest rotate q
  int per, ranges;  // heads per wave, ceil(n_kv / per)
  Rope rope;
  Rotate q;
  int q_out_f16, q_wide;
};

// Eight rows from token t0 on, those in `mask`, as NB vectors of four a lane.
template <typename T, int NB>
__device__ __forceinline__ void load_rows(floatx4 (&v)[NB], const T *x, int64_t stride, bool vec, uint32_t mask) {
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int i = k * 64 + (threadIdx.x & 63), t = i / (NB * 8), d = i % (NB * 8) * 4;
    if (mask >> t & 1) v[k] = load4(x + t * stride + d, vec);
  }
}

template <typename T, int NB, bool ROPE>
__global__ __launch_bounds__(64 * kWaves) void kv_write_kernel(WriteArgs a) {
  if ((int64_t)blockIdx.x >= a.kv_wgs) {
    if constexpr (ROPE) rotate_any<T>(a.q, a.q_out_f16, a.q_wide, ((int64_t)blockIdx.x - a.kv_wgs) * 256 + threadIdx.x);
    return;
  }
  constexpr int D = NB * 32, pitch = D + 4;
  __shared__ __attribute__((aligned(16))) float lds_rows[kWaves][8 * pitch];
  __shared__ Step lds_steps[kWaves][NB * 8];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  float *rows = lds_rows[wave];
  Step *steps = lds_steps[wave];
  // The four waves of a workgroup take neighbouring tokens: a group of 32 fills
  // whole cache lines only together, and workgroups lie on different L2s.
  const uint32_t four = blockIdx.x / (uint32_t)(2 * a.ranges), w = four * kWaves + wave;
  if (8 * (int64_t)w >= a.T) return;
  const int rest = (int)(blockIdx.x - four * 2 * a.ranges), is_v = rest >= a.ranges;
  const int h0 = (is_v ? rest - a.ranges : rest) * a.per, h1 = min(h0 + a.per, a.cache.n_kv);
  const int kind = is_v ? a.v_kind : a.k_kind;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const bool vec = is_v ? a.v_vec : a.k_vec;
  const int64_t own = 8 * (int64_t)w;
  const uint32_t tokens = a.T - own >= 8 ? 0xff : (1u << (a.T - own)) - 1;

  // The wave's own rows load beside their slots: right unless an octet starts
  // inside them (a prompt that begins off a multiple of eight).
  const T *x = (const T *)(is_v ? a.v : a.k) + h0 * D;
  floatx4 next[NB];
  load_rows<T, NB>(next, x + own * stride, stride, vec, tokens);
  const Places p = find_places(a.cache, kind, a.slots, w, a.T);
  const int64_t head_bytes = (int64_t)(a.cache.page_size / kGroup) * group_bytes(kind, NB);
  const uint32_t valid = (uint32_t)__ballot(p.slot >= 0);
  const int half = ROPE ? a.rope.n_rot >> 1 : 0;
  const uint32_t per_half = ROPE ? (1u << 20) / (uint32_t)half + 1 : 0;
  const bool shifted = p.octet > 8;

  for (int pass = 0; pass < 2; ++pass) {
    Eight g = pass == 0 ? Eight{p.octet, 0xff, true} : Eight{8, (p.rest & valid) >> 8, false};
    if (pass == 0 ? p.octet == 0 : g.mask == 0) continue;
    const T *xp = x + (own - 8 + g.first) * stride;
    if (pass == 0 ? shifted : p.octet != 0) load_rows<T, NB>(next, xp, stride, vec, g.mask);
    uint8_t *head = (is_v ? a.cache.v_pages : a.cache.k_pages) + h0 * head_bytes;
    const Spot scales_at = spot_of(p, g.first + ((lane >> 2) & 7)), codes_at = spot_of(p, g.first + (is_v ? 0 : lane & 7));
    for (int h = h0; h < h1; ++h, xp += D, head += head_bytes) {
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = k * 64 + lane, t = i / (NB * 8), d = i % (NB * 8) * 4;
        *(floatx4 *)(rows + t * pitch + d) = next[k];
      }
      if (h + 1 < h1) load_rows<T, NB>(next, xp + D, stride, vec, g.mask);
      wave_sync();
      if (ROPE && !is_v) {
#pragma unroll 1
        for (int i = lane; i < 8 * half; i += 64) {
          const int t = (int)(i * per_half >> 20), q = i - t * half;  // i / half: i < 1024
          if (!(g.mask >> t & 1)) continue;
          float c, s;
          rotation(a.pos[own - 8 + g.first + t], a.rope.freqs[q], a.rope.mscale, c, s);
          float *u = rows + t * pitch + (a.rope.interleaved ? 2 * q : q), *v = u + (a.rope.interleaved ? 1 : half);
          const float xa = *u, xb = *v;
          *u = turned_a(xa, xb, c, s);
          *v = turned_b(xa, xb, c, s);
        }
        wave_sync();
      }
      auto go = [&](auto k) {
        constexpr int KIND = decltype(k)::value;
        if constexpr (KIND != C_F16) {
          write_scales<KIND, NB>(head, scales_at, g, rows, steps);
          wave_sync();
        }
        if (is_v) write_values<KIND, NB>(head, p, codes_at, g, rows, steps);
        else write_keys<KIND, NB>(head, codes_at, g, rows, steps);
      };
      if (kind == C_Q8_0) go(std::integral_constant<int, C_Q8_0>{});
      else if (kind == C_Q4_0) go(std::integral_constant<int, C_Q4_0>{});
      else go(std::integral_constant<int, C_F16>{});
      wave_sync();  // before the next rows
    }
  }
}

struct ReadArgs {
  Cache cache;
  int k_kind, v_kind;
  const int32_t *slots;
  void *k_out, *v_out;
  int64_t T;
  int per, ranges;  // heads per wave, ceil(n_kv / per)
};

template <typename O>
__device__ __forceinline__ void store4(O *p, floatx4 v) {
  if constexpr (sizeof(O) == 2) *(half4 *)p = half4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
  else *(floatx4 *)p = v;
}

// d * (code - offset), exactly: the value fits f32 and the offset's product
// comes in by the same rounding.  Byte k of w, `zero` = -offset * d.
__device__ __forceinline__ float value(uint32_t w, int k, float d, float zero) {
  return __builtin_fmaf((float)(w >> (8 * k) & 255u), d, zero);
}
template <int KIND>
constexpr float kOffset = KIND == C_Q8_0 ? -128.0f : -8.0f;

// `valid`: bit t of token t of the eight (the others read as zeros).
template <int KIND, int NB, typename O>
__device__ __forceinline__ void read_keys(const uint8_t *head, const Places &p, const Eight &g, uint32_t valid, O *out,
                                          int64_t out_stride) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i0 = 0; i0 < NB * 32; i0 += 64) {
    const int i = i0 + lane, t = i / (NB * 4), c = i % (NB * 4), b = c >> 2, G = c & 3;
    const int r = __shfl(p.r, g.first + (t & 7), 64);
    const int64_t base = lane_of(p.base, g.first + (t & 7));
    if (t >= 8 || !(g.mask >> t & 1)) continue;
    O *o = out + t * out_stride + b * 32 + (KIND == C_Q4_0 ? 4 * G : 8 * G);
    floatx4 u = {0, 0, 0, 0}, v = u;
    if (valid >> t & 1) {
      const uint8_t *group = head + base;
      const uint8_t *at = group + code_offset<KIND, false>(b, r, KIND == C_Q4_0 ? 4 * G : 8 * G);
      if constexpr (KIND == C_F16) {
        const half8 h = *(const half8 *)at;
        u = floatx4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
        v = floatx4{(float)h[4], (float)h[5], (float)h[6], (float)h[7]};
      } else {
        const float d = (float)*(const _Float16 *)(group + scale_offset(KIND, NB, b, r)), z = kOffset<KIND> * d;
        uint32_t lo, hi;
        if constexpr (KIND == C_Q8_0) {
          const u32x2 q = *(const u32x2 *)at;
          lo = q[0], hi = q[1];
        } else {
          const uint32_t q = *(const uint32_t *)at;
          lo = q & 0x0f0f0f0f, hi = q >> 4 & 0x0f0f0f0f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u[k] = value(lo, k, d, z);
          v[k] = value(hi, k, d, z);
        }
      }
    }
    store4(o, u);
    store4(o + (KIND == C_Q4_0 ? 16 : 4), v);
  }
}

template <int KIND, int NB, typename O>
__device__ __forceinline__ void read_values(const uint8_t *head, const Places &p, const Eight &g, uint32_t valid, O *out,
                                            int64_t out_stride, O *rows) {
  constexpr int D = NB * 32, pitch = D + 16 / (int)sizeof(O);
  const int lane = threadIdx.x & 63, j = lane & 15;
  if (g.whole) {
    const int r = __builtin_amdgcn_readlane(p.r, g.first);
    const uint8_t *octet = head + lane_of(p.base, g.first);
#pragma unroll
    for (int i0 = 0; i0 < NB * 16; i0 += 64) {
      const int b = (i0 + lane) >> 4;
      if (b >= NB) continue;
      const uint8_t *at = octet + code_offset<KIND, true>(b, r, j);
      O *e = rows + b * 32 + j;
      if constexpr (KIND == C_F16) {
        const half8 u = *(const half8 *)at, v = *(const half8 *)(at + 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k * pitch] = (O)(float)u[k], e[k * pitch + 16] = (O)(float)v[k];
      } else {
        const half8 h = *(const half8 *)(octet + scale_offset(KIND, NB, b, r));
        u32x4 q;
        if constexpr (KIND == C_Q8_0) {
          q = *(const u32x4 *)at;
        } else {
          const u32x2 n = *(const u32x2 *)at;
          q = u32x4{n[0] & 0x0f0f0f0f, n[1] & 0x0f0f0f0f, n[0] >> 4 & 0x0f0f0f0f, n[1] >> 4 & 0x0f0f0f0f};
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float d = (float)h[k], z = kOffset<KIND> * d;
          e[k * pitch] = (O)value(q[k >> 2], k & 3, d, z);
          e[k * pitch + 16] = (O)value(q[2 + (k >> 2)], k & 3, d, z);
        }
      }
    }
  } else {
    for (uint32_t m = g.mask; m; m &= m - 1) {
      const int t = __ffs(m) - 1, r = __builtin_amdgcn_readlane(p.r, g.first + t);
      const uint8_t *group = head + lane_of(p.base, g.first + t);
#pragma unroll
      for (int i0 = 0; i0 < NB * 16; i0 += 64) {
        const int b = (i0 + lane) >> 4;
        if (b >= NB) continue;
        float u = 0.0f, v = 0.0f;
        if (valid >> t & 1) {
          const uint8_t *at = group + code_offset<KIND, true>(b, r, j);
          if constexpr (KIND == C_F16) {
            u = (float)*(const _Float16 *)at, v = (float)*(const _Float16 *)(at + 1024);
          } else {
            const float d = (float)*(const _Float16 *)(group + scale_offset(KIND, NB, b, r)), z = kOffset<KIND> * d;
            if constexpr (KIND == C_Q8_0) u = value(at[0], 0, d, z), v = value(at[8], 0, d, z);
            else u = value(at[0] & 15, 0, d, z), v = value(at[0] >> 4, 0, d, z);
          }
        }
        rows[t * pitch + b * 32 + j] = (O)u;
        rows[t * pitch + b * 32 + j + 16] = (O)v;
      }
    }
  }
  wave_sync();
  constexpr int per = 16 / sizeof(O);
#pragma unroll
  for (int i0 = 0; i0 < 8 * (D / per); i0 += 64) {
    const int i = i0 + lane, t = i / (D / per), d = (i % (D / per)) * per;
    if (t < 8 && (g.mask >> t & 1)) *(u32x4 *)(out + t * out_stride + d) = *(const u32x4 *)(rows + t * pitch + d);
  }
  wave_sync();  // before the next rows
}

template <typename O, int NB>
__global__ __launch_bounds__(64 * kWaves) void kv_read_kernel(ReadArgs a) {
  constexpr int D = NB * 32;
  __shared__ u32x4 tile[kWaves][8 * (D * sizeof(O) + 16) / 16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // The four waves of a workgroup take neighbouring tokens: a group of 32 fills
  // whole cache lines only together, and workgroups lie on different L2s.
  const uint32_t four = blockIdx.x / (uint32_t)(2 * a.ranges), w = four * kWaves + wave;
  if (8 * (int64_t)w >= a.T) return;
  const int rest = (int)(blockIdx.x - four * 2 * a.ranges), is_v = rest >= a.ranges, n = a.cache.n_kv;
  const int h0 = (is_v ? rest - a.ranges : rest) * a.per, h1 = min(h0 + a.per, n);
  const int kind = is_v ? a.v_kind : a.k_kind;
  const Places p = find_places(a.cache, kind, a.slots, w, a.T);
  const int64_t head_bytes = (int64_t)(a.cache.page_size / kGroup) * group_bytes(kind, NB);
  const uint32_t valid = (uint32_t)__ballot(p.slot >= 0);
  for (int pass = 0; pass < 2; ++pass) {
    const Eight g = pass == 0 ? Eight{p.octet, 0xff, true} : Eight{8, p.rest >> 8, false};
    if (pass == 0 ? p.octet == 0 : g.mask == 0) continue;
    const int64_t t0 = 8 * (int64_t)w - 8 + g.first;
    for (int h = h0; h < h1; ++h) {
      O *out = (O *)(is_v ? a.v_out : a.k_out) + (t0 * n + h) * D;
      const uint8_t *head = (is_v ? a.cache.v_pages : a.cache.k_pages) + h * head_bytes;
      auto go = [&](auto k) {
        constexpr int KIND = decltype(k)::value;
        if (is_v) read_values<KIND, NB, O>(head, p, g, valid >> g.first, out, (int64_t)n * D, (O *)tile[wave]);
        else read_keys<KIND, NB, O>(head, p, g, valid >> g.first, out, (int64_t)n * D);
      };
      if (kind == C_Q8_0) go(std::integral_constant<int, C_Q8_0>{});
      else if (kind == C_Q4_0) go(std::integral_constant<int, C_Q4_0>{});
      else go(std::integral_constant<int, C_F16>{});
    }
  }
}

// Heads per wave: one until the grid holds four rounds of eight waves per SIMD
// (32768 tokens of 8 x 128 in Q4_0: two heads a wave write in 72 us and read
// in 37, one in 82 and 41, four in 77 and 41, all eight in 90 and 47).
static void split_heads(int64_t T, int64_t n_kv, int &per, int &ranges, int64_t &wgs) {
  const int64_t one = (T + 7) / 8 * 2 * n_kv, full = (int64_t)4 * device_cus() * 4 * 8;
  per = (int)std::min(std::max(one / full, (int64_t)1), n_kv);
  ranges = (int)((n_kv + per - 1) / per);
  wgs = (T + 8 * kWaves - 1) / (8 * kWaves) * 2 * ranges;
}

static Cache make_cache(const KvCache &k) {
  const int P = (int)k.page_size;
  return Cache{(uint8_t *)k.k_pages, (uint8_t *)k.v_pages, k.n_pages * k.page_size, P, P & (P - 1) ? -1 : __builtin_ctz(P),
               (int)k.n_kv, (int)(k.head_dim / 32)};
}

template <typename T, int NB>
static hipError_t run_write(const KvCache &kc, const KvWrite &w, hipStream_t s) {
  WriteArgs a{};
  a.cache = make_cache(kc);
  a.k_kind = kc.k_kind, a.v_kind = kc.v_kind;
  a.k = w.k, a.v = w.v;
  a.k_stride = w.k_stride, a.v_stride = w.v_stride;
  a.k_vec = w.k_stride % 4 == 0 && (uintptr_t)w.k % (4 * sizeof(T)) == 0;
  a.v_vec = w.v_stride % 4 == 0 && (uintptr_t)w.v % (4 * sizeof(T)) == 0;
  a.pos = w.pos, a.slots = w.slots, a.T = w.T;
  split_heads(w.T, kc.n_kv, a.per, a.ranges, a.kv_wgs);
  int64_t threads = 0;
  if (w.rope) {
    a.rope = Rope{w.freqs, (int)w.n_rot, w.interleaved, w.mscale};
    a.q.x = w.q, a.q.y = w.q_out, a.q.x_stride = w.q_stride, a.q.y_stride = w.q_out_stride;
    a.q.pos = w.pos, a.q.T = w.T, a.q.H = (int)w.n_q, a.q.D = (int)kc.head_dim, a.q.rope = a.rope;
    a.q_out_f16 = w.q_out_f16;
    a.q_wide = plan_rotate(a.q, sizeof(T), w.q_out_f16 ? 2 : 4, threads);
  }
  const dim3 grid((unsigned)(a.kv_wgs + (threads + 255) / 256));
  if (w.rope) hipLaunchKernelGGL((kv_write_kernel<T, NB, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((kv_write_kernel<T, NB, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int NB>
static hipError_t run_read(const KvCache &kc, const int32_t *slots, int64_t T, void *k_out, void *v_out, int f16,
                           hipStream_t s) {
  ReadArgs a{make_cache(kc), kc.k_kind, kc.v_kind, slots, k_out, v_out, T, 0, 0};
  int64_t wgs;
  split_heads(T, kc.n_kv, a.per, a.ranges, wgs);
  const dim3 grid((unsigned)wgs);
  if (f16) hipLaunchKernelGGL((kv_read_kernel<_Float16, NB>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((kv_read_kernel<float, NB>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace kv

hipError_t launch_kv_write(const KvCache &c, const KvWrite &w, hipStream_t s) {
  switch (c.head_dim / 32) {
#define QMM_CASE(NB) \
  case NB:           \
    return w.f16 ? kv::run_write<_Float16, NB>(c, w, s) : kv::run_write<float, NB>(c, w, s);
    QMM_CASE(2) QMM_CASE(3) QMM_CASE(4) QMM_CASE(6) QMM_CASE(8)
#undef QMM_CASE
  }
  return hipErrorInvalidValue;
}

hipError_t launch_kv_read(const KvCache &c, const int32_t *slots, int64_t T, void *k_out, void *v_out, int f16,
                          hipStream_t s) {
  switch (c.head_dim / 32) {
#define QMM_CASE(NB) \
  case NB:           \
    return kv::run_read<NB>(c, slots, T, k_out, v_out, f16, s);
    QMM_CASE(2) QMM_CASE(3) QMM_CASE(4) QMM_CASE(6) QMM_CASE(8)
#undef QMM_CASE
  }
  return hipErrorInvalidValue;
}

int64_t kv_page_bytes(int kind, int64_t page_size, int64_t n_kv, int64_t head_dim) {
  return page_size / kv::kGroup * n_kv * kv::group_bytes(kind, (int)(head_dim / 32));
}

}  // namespace qmm
