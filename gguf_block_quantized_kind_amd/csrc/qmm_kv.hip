// qmm_kv.hip -- writing new tokens into the paged key/value cache (quantized
// to its kind, with or without the rotation of the keys and queries) and
// reading tokens back.  Layout and quantizer: qmm_kv.h.
//
// Both kernels give a workgroup a window of 32 tokens of one head's keys or
// values and pass it through LDS, because rows lie along the elements and
// cache units across tokens:
//   write  rows -> LDS (f32; rotated there), block scales, then every thread
//          encodes the elements of one cache unit and stores it: 16, 8 or 4
//          bytes of one key token, or eight tokens of an element pair of the
//          values.
//   read   the reverse; keys need no LDS, a unit of theirs being a run of one
//          row's elements.
// Value units hold eight consecutive tokens.  The window's tokens are taken in
// octets that start where the first token's slot is a multiple of eight, so a
// prompt's tokens fill whole units wherever it starts; an octet whose slots
// are not eight consecutive aligned ones (other sequences, skipped tokens, the
// window's ends) goes byte by byte.
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

constexpr int kWindow = 32;
constexpr int kOctets = kWindow / 8 + 1;

// Where the window's tokens lie.
struct Window {
  int64_t base[kWindow];  // first byte of the token's group
  int slot[kWindow];      // -1: skipped or past the end
  int r[kWindow];         // token of its group
  int whole[kOctets];     // the octet is one aligned unit
  int phase;              // octet o covers tokens 8 o - phase + [0, 8)
};

__device__ __forceinline__ void find_window(Window &w, const Cache &c, const int32_t *slots, int64_t t0, int nt, int kind,
                                            int head) {
  const int tid = threadIdx.x;
  if (tid < kWindow) {
    int slot = tid < nt ? slots[t0 + tid] : -1;
    if (slot >= c.n_slots) slot = -1;
    slot = max(slot, -1);
    w.slot[tid] = slot;
    w.base[tid] = slot < 0 ? 0 : group_at(c, kind, slot, head);
    w.r[tid] = slot < 0 ? 0 : (slot % c.page_size) % kGroup;
    if (tid == 0) w.phase = slot < 0 ? 0 : slot % 8;
  }
  __syncthreads();
  if (tid < kOctets) {
    const int t = 8 * tid - w.phase;
    bool whole = t >= 0 && t + 8 <= kWindow && w.slot[max(t, 0)] >= 0 && w.slot[max(t, 0)] % 8 == 0;
    for (int e = 1; e < 8 && whole; ++e) whole = w.slot[t + e] == w.slot[t] + e;
    w.whole[tid] = whole;
  }
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

// The block scales of a window's rows, four lanes per (token, block) with
// eight elements each: stored in the cache, and as steps for the encoding.
template <int KIND, int NB>
__device__ __forceinline__ void write_scales(uint8_t *pages, const Window &w, float *rows, Step *steps) {
  constexpr int pitch = NB * 32 + 4;
#pragma unroll
  for (int i0 = 0; i0 < NB * kWindow * 4; i0 += 256) {
    const int i = i0 + threadIdx.x, t = (i >> 2) & (kWindow - 1), b = i >> 7;
    if (b >= NB || w.slot[t] < 0) continue;  // (all four lanes)
    float *e = rows + t * pitch + b * 32 + (i & 3) * 8;
    const floatx4 u = *(const floatx4 *)e, v = *(const floatx4 *)(e + 4);
    float hi = u[0], lo = u[0];
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      hi = fmaxf(hi, fmaxf(u[k], v[k]));
      lo = fminf(lo, fminf(u[k], v[k]));
      bits = max(bits, max(magnitude_bits(u[k]), magnitude_bits(v[k])));
    }
#pragma unroll
    for (int k = 1; k < 4; k <<= 1) {
      hi = fmaxf(hi, __shfl_xor(hi, k, 4));
      lo = fminf(lo, __shfl_xor(lo, k, 4));
      bits = max(bits, (uint32_t)__shfl_xor((int)bits, k, 4));
    }
    const _Float16 h = block_scale<KIND>(hi, lo, bits);
    if (bits >= 0x7f800000u) *(floatx4 *)e = *(floatx4 *)(e + 4) = floatx4{0, 0, 0, 0};
    if ((i & 3) == 0) {
      steps[b * kWindow + t] = step_of(h);
      *(_Float16 *)(pages + w.base[t] + scale_offset(KIND, NB, b, w.r[t])) = h;
    }
  }
}

template <int KIND, int NB>
__device__ __forceinline__ void write_keys(uint8_t *pages, const Window &w, const float *rows, const Step *steps) {
  constexpr int pitch = NB * 32 + 4;
#pragma unroll
  for (int i0 = 0; i0 < NB * 4 * kWindow; i0 += 256) {
    const int i = i0 + threadIdx.x, t = i & (kWindow - 1), G = (i >> 5) & 3, b = i >> 7;
    if (b >= NB || w.slot[t] < 0) continue;
    const float *e = rows + t * pitch + b * 32;
    uint8_t *p = pages + w.base[t] + code_offset<KIND, false>(b, w.r[t], KIND == C_Q4_0 ? 4 * G : 8 * G);
    const floatx4 u = *(const floatx4 *)(e + (KIND == C_Q4_0 ? 4 * G : 8 * G));
    const floatx4 v = *(const floatx4 *)(e + (KIND == C_Q4_0 ? 16 + 4 * G : 8 * G + 4));
    if constexpr (KIND == C_F16) {
      *(u32x4 *)p = u32x4{pack_h(u[0], u[1]), pack_h(u[2], u[3]), pack_h(v[0], v[1]), pack_h(v[2], v[3])};
    } else {
      const Step st = steps[b * kWindow + t];
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lo = put(lo, k, encode<KIND>(u[k], st));
        hi = put(hi, k, encode<KIND>(v[k], st));
      }
      if constexpr (KIND == C_Q8_0) *(u32x2 *)p = u32x2{lo, hi};
      else *(uint32_t *)p = lo | hi << 4;
    }
  }
}

template <int KIND, int NB>
__device__ __forceinline__ void write_values(uint8_t *pages, int nt, const Window &w, const float *rows,
                                             const Step *steps) {
  constexpr int pitch = NB * 32 + 4;
  for (int i = threadIdx.x; i < kOctets * NB * 16; i += 256) {
    const int j = i & 15, b = (i >> 4) % NB, o = (i >> 4) / NB;
    const int t0 = 8 * o - w.phase;
    if (w.whole[o]) {
      const float *e = rows + t0 * pitch + b * 32 + j;
      uint8_t *p = pages + w.base[t0] + code_offset<KIND, true>(b, w.r[t0], j);
      if constexpr (KIND == C_F16) {
        u32x4 a, v;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = pack_h(e[2 * k * pitch], e[(2 * k + 1) * pitch]);
          v[k] = pack_h(e[2 * k * pitch + 16], e[(2 * k + 1) * pitch + 16]);
        }
        *(u32x4 *)p = a;
        *(u32x4 *)(p + 1024) = v;
      } else {
        uint32_t q[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const Step st = steps[b * kWindow + t0 + k];
          q[k >> 2] = put(q[k >> 2], k & 3, encode<KIND>(e[k * pitch], st));
          q[2 + (k >> 2)] = put(q[2 + (k >> 2)], k & 3, encode<KIND>(e[k * pitch + 16], st));
        }
        if constexpr (KIND == C_Q8_0) *(u32x4 *)p = u32x4{q[0], q[1], q[2], q[3]};
        else *(u32x2 *)p = u32x2{q[0] | q[2] << 4, q[1] | q[3] << 4};
      }
    } else {
      for (int t = max(t0, 0); t < min(t0 + 8, nt); ++t) {
        if (w.slot[t] < 0) continue;
        const float *e = rows + t * pitch + b * 32 + j;
        uint8_t *p = pages + w.base[t];
        if constexpr (KIND == C_F16) {
          *(_Float16 *)(p + code_offset<KIND, true>(b, w.r[t], j)) = (_Float16)e[0];
          *(_Float16 *)(p + code_offset<KIND, true>(b, w.r[t], j + 16)) = (_Float16)e[16];
        } else {
          const Step st = steps[b * kWindow + t];
          const uint32_t q = put(put(0, 0, encode<KIND>(e[0], st)), 1, encode<KIND>(e[16], st));
          if constexpr (KIND == C_Q8_0) {
            p[code_offset<KIND, true>(b, w.r[t], j)] = (uint8_t)q;
            p[code_offset<KIND, true>(b, w.r[t], j + 16)] = (uint8_t)(q >> 8);
          } else {
            p[code_offset<KIND, true>(b, w.r[t], j)] = (uint8_t)(q | q >> 4);
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
  int64_t kv_wgs;  // workgroups of the cache part; the rest rotate q
  Rope rope;
  Rotate q;
  int q_out_f16, q_wide;
};

template <typename T, int NB, bool ROPE>
__global__ __launch_bounds__(256) void kv_write_kernel(WriteArgs a) {
  if ((int64_t)blockIdx.x >= a.kv_wgs) {
    if constexpr (ROPE) rotate_any<T>(a.q, a.q_out_f16, a.q_wide, ((int64_t)blockIdx.x - a.kv_wgs) * 256 + threadIdx.x);
    return;
  }
  constexpr int D = NB * 32, pitch = D + 4;
  __shared__ Window w;
  __shared__ float rows[kWindow * pitch];
  __shared__ Step steps[NB * kWindow];
  const int tid = threadIdx.x, n = a.cache.n_kv;
  const int64_t win = (int64_t)((uint32_t)blockIdx.x / (uint32_t)(2 * n));
  const int rest = (int)(blockIdx.x - win * 2 * n), is_v = rest >= n, head = is_v ? rest - n : rest;
  const int kind = is_v ? a.v_kind : a.k_kind;
  const int64_t t0 = win * kWindow, stride = is_v ? a.v_stride : a.k_stride;
  const int nt = (int)min((int64_t)kWindow, a.T - t0);

  // Rows, slots and the first rotations' angles in one round of loads.
  const T *x = (const T *)(is_v ? a.v : a.k) + t0 * stride + head * D;
  const bool vec = is_v ? a.v_vec : a.k_vec;
#pragma unroll
  for (int i0 = 0; i0 < kWindow * (D / 4); i0 += 256) {
    const int i = i0 + tid, t = i / (D / 4), d = (i % (D / 4)) * 4;
    if (t < nt) *(floatx4 *)(rows + t * pitch + d) = load4(x + t * stride + d, vec);
  }
  const int half = ROPE ? a.rope.n_rot >> 1 : 0;
  float co = 1.0f, si = 0.0f;
  if (ROPE && !is_v && tid < nt * half) rotation(a.pos[t0 + tid / half], a.rope.freqs[tid % half], co, si);
  find_window(w, a.cache, a.slots, t0, nt, kind, head);
  __syncthreads();
  if (ROPE && !is_v) {
    for (int i = tid; i < nt * half; i += 256) {
      const int t = i / half, p = i - t * half;
      if (i >= 256) rotation(a.pos[t0 + t], a.rope.freqs[p], co, si);
      float *u = rows + t * pitch + (a.rope.interleaved ? 2 * p : p), *v = u + (a.rope.interleaved ? 1 : half);
      const float c = co * a.rope.mscale, s = si * a.rope.mscale, xa = *u, xb = *v;
      *u = xa * c - xb * s;
      *v = xa * s + xb * c;
    }
    __syncthreads();
  }
  uint8_t *pages = is_v ? a.cache.v_pages : a.cache.k_pages;
  auto go = [&](auto k) {
    constexpr int KIND = decltype(k)::value;
    if constexpr (KIND != C_F16) {
      write_scales<KIND, NB>(pages, w, rows, steps);
      __syncthreads();
    }
    if (is_v) write_values<KIND, NB>(pages, nt, w, rows, steps);
    else write_keys<KIND, NB>(pages, w, rows, steps);
  };
  if (kind == C_Q8_0) go(std::integral_constant<int, C_Q8_0>{});
  else if (kind == C_Q4_0) go(std::integral_constant<int, C_Q4_0>{});
  else go(std::integral_constant<int, C_F16>{});
}

struct ReadArgs {
  Cache cache;
  int k_kind, v_kind;
  const int32_t *slots;
  void *k_out, *v_out;
  int64_t T;
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

template <int KIND, int NB, typename O>
__device__ __forceinline__ void read_keys(const Cache &c, O *out, int64_t out_stride, int nt, const Window &w) {
#pragma unroll
  for (int i0 = 0; i0 < kWindow * NB * 4; i0 += 256) {
    const int i = i0 + threadIdx.x, t = i / (NB * 4), p = i % (NB * 4), b = p >> 2, G = p & 3;
    if (t >= nt) continue;
    O *o = out + t * out_stride + b * 32 + (KIND == C_Q4_0 ? 4 * G : 8 * G);
    floatx4 u = {0, 0, 0, 0}, v = u;
    if (w.slot[t] >= 0) {
      const uint8_t *g = c.k_pages + w.base[t];
      const uint8_t *at = g + code_offset<KIND, false>(b, w.r[t], KIND == C_Q4_0 ? 4 * G : 8 * G);
      if constexpr (KIND == C_F16) {
        const half8 h = *(const half8 *)at;
        u = floatx4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
        v = floatx4{(float)h[4], (float)h[5], (float)h[6], (float)h[7]};
      } else {
        const float d = (float)*(const _Float16 *)(g + scale_offset(KIND, NB, b, w.r[t])), z = kOffset<KIND> * d;
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
__device__ __forceinline__ void read_values(const Cache &c, O *out, int64_t out_stride, int nt, const Window &w, O *rows) {
  constexpr int D = NB * 32, pitch = D + 16 / (int)sizeof(O);
  for (int i = threadIdx.x; i < kOctets * NB * 16; i += 256) {
    const int j = i & 15, b = (i >> 4) % NB, o = (i >> 4) / NB;
    const int t0 = 8 * o - w.phase;
    if (w.whole[o]) {
      const uint8_t *g = c.v_pages + w.base[t0], *p = g + code_offset<KIND, true>(b, w.r[t0], j);
      O *e = rows + t0 * pitch + b * 32 + j;
      if constexpr (KIND == C_F16) {
        const half8 u = *(const half8 *)p, v = *(const half8 *)(p + 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k * pitch] = (O)(float)u[k], e[k * pitch + 16] = (O)(float)v[k];
      } else {
        const half8 h = *(const half8 *)(g + scale_offset(KIND, NB, b, w.r[t0]));
        u32x4 q;
        if constexpr (KIND == C_Q8_0) {
          q = *(const u32x4 *)p;
        } else {
          const u32x2 n = *(const u32x2 *)p;
          q = u32x4{n[0] & 0x0f0f0f0f, n[1] & 0x0f0f0f0f, n[0] >> 4 & 0x0f0f0f0f, n[1] >> 4 & 0x0f0f0f0f};
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float d = (float)h[k], z = kOffset<KIND> * d;
          e[k * pitch] = (O)value(q[k >> 2], k & 3, d, z);
          e[k * pitch + 16] = (O)value(q[2 + (k >> 2)], k & 3, d, z);
        }
      }
    } else {
      for (int t = max(t0, 0); t < min(t0 + 8, nt); ++t) {
        float u = 0.0f, v = 0.0f;
        if (w.slot[t] >= 0) {
          const uint8_t *g = c.v_pages + w.base[t], *p = g + code_offset<KIND, true>(b, w.r[t], j);
          if constexpr (KIND == C_F16) {
            u = (float)*(const _Float16 *)p, v = (float)*(const _Float16 *)(p + 1024);
          } else {
            const float d = (float)*(const _Float16 *)(g + scale_offset(KIND, NB, b, w.r[t])), z = kOffset<KIND> * d;
            if constexpr (KIND == C_Q8_0) u = value(p[0], 0, d, z), v = value(p[8], 0, d, z);
            else u = value(p[0] & 15, 0, d, z), v = value(p[0] >> 4, 0, d, z);
          }
        }
        rows[t * pitch + b * 32 + j] = (O)u;
        rows[t * pitch + b * 32 + j + 16] = (O)v;
      }
    }
  }
  __syncthreads();
  constexpr int per = 16 / sizeof(O);
#pragma unroll
  for (int i0 = 0; i0 < kWindow * (D / per); i0 += 256) {
    const int i = i0 + threadIdx.x, t = i / (D / per), d = (i % (D / per)) * per;
    if (t < nt) *(u32x4 *)(out + t * out_stride + d) = *(const u32x4 *)(rows + t * pitch + d);
  }
}

template <typename O, int NB>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadArgs a) {
  constexpr int D = NB * 32;
  __shared__ Window w;
  __shared__ u32x4 tile[kWindow * (D * sizeof(O) + 16) / 16];
  const int n = a.cache.n_kv;
  const int64_t win = (int64_t)((uint32_t)blockIdx.x / (uint32_t)(2 * n));
  const int rest = (int)(blockIdx.x - win * 2 * n), is_v = rest >= n, head = is_v ? rest - n : rest;
  const int kind = is_v ? a.v_kind : a.k_kind;
  const int64_t t0 = win * kWindow;
  const int nt = (int)min((int64_t)kWindow, a.T - t0);
  find_window(w, a.cache, a.slots, t0, nt, kind, head);
  __syncthreads();
  O *out = (O *)(is_v ? a.v_out : a.k_out) + (t0 * n + head) * D;
  auto go = [&](auto k) {
    constexpr int KIND = decltype(k)::value;
    if (is_v) read_values<KIND, NB, O>(a.cache, out, (int64_t)n * D, nt, w, (O *)tile);
    else read_keys<KIND, NB, O>(a.cache, out, (int64_t)n * D, nt, w);
  };
  if (kind == C_Q8_0) go(std::integral_constant<int, C_Q8_0>{});
  else if (kind == C_Q4_0) go(std::integral_constant<int, C_Q4_0>{});
  else go(std::integral_constant<int, C_F16>{});
}

static Cache make_cache(const KvCache &k) {
  return Cache{(uint8_t *)k.k_pages, (uint8_t *)k.v_pages, k.n_pages * k.page_size, (int)k.page_size, (int)k.n_kv,
               (int)(k.head_dim / 32)};
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
  a.kv_wgs = (w.T + kWindow - 1) / kWindow * 2 * kc.n_kv;
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
  const ReadArgs a{make_cache(kc), kc.k_kind, kc.v_kind, slots, k_out, v_out, T};
  const dim3 grid((unsigned)((T + kWindow - 1) / kWindow * 2 * kc.n_kv));
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
