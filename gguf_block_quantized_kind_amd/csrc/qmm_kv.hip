// qmm_kv.hip -- writing new tokens into the paged key/value cache (quantized
// to its kind, with or without the rotation of the keys and queries) and
// reading tokens back.  Layout and quantizer: qmm_kv.h.
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {
namespace kv {

// One rotated element d of a row: x[d] with its partner of the pair.
template <typename T>
__device__ __forceinline__ float rotated(const Rope &rp, const T *x, int d, int pos) {
  const float v = (float)x[d];
  if (d >= rp.n_rot) return v;
  const int half = rp.n_rot >> 1;
  const bool second = rp.interleaved ? (d & 1) : d >= half;
  const int pair = rp.interleaved ? d >> 1 : second ? d - half : d;
  const int other = rp.interleaved ? d ^ 1 : second ? d - half : d + half;
  float c, s;
  rotation(pos, rp.freqs[pair], c, s);
  c *= rp.mscale;
  s *= rp.mscale;
  const float u = (float)x[other];
  return second ? u * s + v * c : v * c - u * s;
}

// One block of 32 elements per half wave: lane c holds element c.
template <int KIND, bool IS_V>
__device__ __forceinline__ void store_block(uint8_t *group, int NB, int b, int r, int c, float x) {
  uint8_t *p = group + code_offset<KIND, IS_V>(b, r, c);
  if constexpr (KIND == C_F16) {
    *(_Float16 *)p = (_Float16)x;
  } else {
    float hi = x, lo = x;
    uint32_t bits = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
#pragma unroll
    for (int k = 16; k; k >>= 1) {
      hi = fmaxf(hi, __shfl_xor(hi, k, 32));
      lo = fminf(lo, __shfl_xor(lo, k, 32));
      bits = max(bits, (uint32_t)__shfl_xor((int)bits, k, 32));
    }
    const _Float16 h = block_scale<KIND>(hi, lo, bits);
    uint32_t q = encode<KIND>(x, h);
    if constexpr (KIND == C_Q4_0) {
      q |= (uint32_t)__shfl_xor((int)q, 16, 32) << 4;
      if (c < 16) *p = (uint8_t)q;
    } else {
      *p = (uint8_t)q;
    }
    if (c == 0) *(_Float16 *)(group + scale_offset(KIND, NB, b, r)) = h;
  }
}

struct WriteArgs {
  Cache cache;
  const void *k, *v, *q;
  int64_t k_stride, v_stride, q_stride;
  void *q_out;
  int64_t q_out_stride;
  const int32_t *pos, *slots;
  int64_t kv_wgs;  // workgroups of the cache part; the rest rotate q
  int64_t kv_blocks, q_pairs;
  int n_q;
  Rope rope;
};

// Per-token write: a half wave owns one block of 32 elements of one token's
// key or value head.  The reads are whole rows; the codes go out as single
// bytes (a token's bytes lie apart in the group).
template <int KK, int VK, typename T, typename QO, bool ROPE>
__global__ __launch_bounds__(256) void kv_write_kernel(WriteArgs a) {
  const int NB = a.cache.NB, D = NB * 32;
  if ((int64_t)blockIdx.x < a.kv_wgs) {
    const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (task >= a.kv_blocks) return;  // a whole half wave
    const int c = threadIdx.x & 31;
    const int per = a.cache.n_kv * 2 * NB;
    const int64_t t = task / per;
    int rest = (int)(task - t * per);
    const int is_v = rest / (a.cache.n_kv * NB);
    rest -= is_v * a.cache.n_kv * NB;
    const int head = rest / NB, b = rest - head * NB;
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.cache.n_slots) return;
    const int r = (slot % a.cache.page_size) % kGroup;
    if (is_v) {
      const T *x = (const T *)a.v + t * a.v_stride + head * D;
      store_block<VK, true>(a.cache.v_pages + group_at(a.cache, VK, slot, head), NB, b, r, c, (float)x[b * 32 + c]);
    } else {
      const T *x = (const T *)a.k + t * a.k_stride + head * D;
      const float y = ROPE ? rotated(a.rope, x, b * 32 + c, a.pos[t]) : (float)x[b * 32 + c];
      store_block<KK, false>(a.cache.k_pages + group_at(a.cache, KK, slot, head), NB, b, r, c, y);
    }
  } else if constexpr (ROPE) {
    const int64_t p = ((int64_t)blockIdx.x - a.kv_wgs) * 256 + threadIdx.x;
    if (p >= a.q_pairs) return;
    const int64_t row = p / (D / 2);  // t * n_q + head
    const int i = (int)(p - row * (D / 2)), half = a.rope.n_rot >> 1;
    const int64_t t = row / a.n_q;
    const int head = (int)(row - t * a.n_q);
    const T *x = (const T *)a.q + t * a.q_stride + (int64_t)head * D;
    QO *y = (QO *)a.q_out + t * a.q_out_stride + (int64_t)head * D;
    const bool turned = i < half;
    const int da = turned ? (a.rope.interleaved ? 2 * i : i) : 2 * i;
    const int db = turned && !a.rope.interleaved ? i + half : da + 1;
    const float u = (float)x[da], v = (float)x[db];
    float c = 1.0f, s = 0.0f;
    if (turned) {
      rotation(a.pos[t], a.rope.freqs[i], c, s);
      c *= a.rope.mscale;
      s *= a.rope.mscale;
    }
    y[da] = (QO)(turned ? u * c - v * s : u);
    y[db] = (QO)(turned ? u * s + v * c : v);
  }
}

template <int KIND, bool IS_V>
__device__ __forceinline__ float load_element(const uint8_t *group, int NB, int b, int r, int c) {
  const uint8_t *p = group + code_offset<KIND, IS_V>(b, r, c);
  if constexpr (KIND == C_F16) return (float)*(const _Float16 *)p;
  const float d = (float)*(const _Float16 *)(group + scale_offset(KIND, NB, b, r));
  if constexpr (KIND == C_Q8_0) return d * (float)((int)*p - 128);
  return d * (float)(((int)*p >> (c >> 4) * 4 & 15) - 8);
}

struct ReadArgs {
  Cache cache;
  const int32_t *slots;
  void *k_out, *v_out;
  int64_t blocks;
};

template <int KK, int VK, typename O>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadArgs a) {
  const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (task >= a.blocks) return;
  const int NB = a.cache.NB, c = threadIdx.x & 31;
  const int per = a.cache.n_kv * 2 * NB;
  const int64_t t = task / per;
  int rest = (int)(task - t * per);
  const int is_v = rest / (a.cache.n_kv * NB);
  rest -= is_v * a.cache.n_kv * NB;
  const int head = rest / NB, b = rest - head * NB;
  const int slot = a.slots[t];
  const int64_t o = (t * a.cache.n_kv + head) * (NB * 32) + b * 32 + c;
  if (slot < 0 || slot >= a.cache.n_slots) {
    ((O *)(is_v ? a.v_out : a.k_out))[o] = (O)0.0f;
    return;
  }
  const int r = (slot % a.cache.page_size) % kGroup;
  if (is_v)
    ((O *)a.v_out)[o] = (O)load_element<VK, true>(a.cache.v_pages + group_at(a.cache, VK, slot, head), NB, b, r, c);
  else
    ((O *)a.k_out)[o] = (O)load_element<KK, false>(a.cache.k_pages + group_at(a.cache, KK, slot, head), NB, b, r, c);
}

static Cache make_cache(const KvCache &k) {
  return Cache{(uint8_t *)k.k_pages, (uint8_t *)k.v_pages, k.n_pages * k.page_size, (int)k.page_size, (int)k.n_kv,
               (int)(k.head_dim / 32)};
}

template <int KK, int VK>
static hipError_t write_kinds(const KvCache &kc, const KvWrite &w, hipStream_t s) {
  WriteArgs a{};
  a.cache = make_cache(kc);
  a.k = w.k, a.v = w.v, a.q = w.q;
  a.k_stride = w.k_stride, a.v_stride = w.v_stride, a.q_stride = w.q_stride;
  a.q_out = w.q_out, a.q_out_stride = w.q_out_stride;
  a.pos = w.pos, a.slots = w.slots;
  a.kv_blocks = w.T * kc.n_kv * 2 * a.cache.NB;
  a.kv_wgs = (a.kv_blocks + 7) / 8;
  a.n_q = (int)w.n_q;
  a.q_pairs = w.rope ? w.T * w.n_q * (kc.head_dim / 2) : 0;
  if (w.rope) a.rope = Rope{w.freqs, (int)w.n_rot, w.interleaved, w.mscale};
  const dim3 grid((unsigned)(a.kv_wgs + (a.q_pairs + 255) / 256));
#define QMM_LAUNCH(T, QO, R) hipLaunchKernelGGL((kv_write_kernel<KK, VK, T, QO, R>), grid, dim3(256), 0, s, a)
  if (!w.rope) {
    if (w.f16) QMM_LAUNCH(_Float16, _Float16, false);
    else QMM_LAUNCH(float, float, false);
  } else if (w.f16) {
    if (w.q_out_f16) QMM_LAUNCH(_Float16, _Float16, true);
    else QMM_LAUNCH(_Float16, float, true);
  } else {
    if (w.q_out_f16) QMM_LAUNCH(float, _Float16, true);
    else QMM_LAUNCH(float, float, true);
  }
#undef QMM_LAUNCH
  return hipGetLastError();
}

template <int KK, int VK>
static hipError_t read_kinds(const KvCache &kc, const int32_t *slots, int64_t T, void *k_out, void *v_out, int f16,
                             hipStream_t s) {
  ReadArgs a{make_cache(kc), slots, k_out, v_out, 0};
  a.blocks = T * kc.n_kv * 2 * a.cache.NB;
  const dim3 grid((unsigned)((a.blocks + 7) / 8));
  if (f16) hipLaunchKernelGGL((kv_read_kernel<KK, VK, _Float16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((kv_read_kernel<KK, VK, float>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace kv

#define QMM_KV_KINDS(F)                                                                            \
  F(1, 1) F(1, 8) F(1, 2) F(8, 1) F(8, 8) F(8, 2) F(2, 1) F(2, 8) F(2, 2)

hipError_t launch_kv_write(const KvCache &c, const KvWrite &w, hipStream_t s) {
#define QMM_CASE(K, V) \
  if (c.k_kind == K && c.v_kind == V) return kv::write_kinds<K, V>(c, w, s);
  QMM_KV_KINDS(QMM_CASE)
#undef QMM_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_kv_read(const KvCache &c, const int32_t *slots, int64_t T, void *k_out, void *v_out, int f16,
                          hipStream_t s) {
#define QMM_CASE(K, V) \
  if (c.k_kind == K && c.v_kind == V) return kv::read_kinds<K, V>(c, slots, T, k_out, v_out, f16, s);
  QMM_KV_KINDS(QMM_CASE)
#undef QMM_CASE
  return hipErrorInvalidValue;
}

int64_t kv_page_bytes(int kind, int64_t page_size, int64_t n_kv, int64_t head_dim) {
  return page_size / kv::kGroup * n_kv * kv::group_bytes(kind, (int)(head_dim / 32));
}

}  // namespace qmm
