// qmm_attn.hip -- single-token attention over the paged cache: workspace,
// dispatch by kinds, and the join of a sequence's splits.
#include "qmm_attn.h"

namespace qmm {
namespace attn {

// The splits of more than 64 sequences, by one workgroup: as find_split, with
// sums in 64 bits.
__global__ __launch_bounds__(1024) void plan_kernel(Args a) {
  __shared__ double dsum[16];
  __shared__ uint32_t usum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto block_sum = [&](double v) {
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) v += __shfl_xor(v, k, 64);
    if (lane == 0) dsum[wave] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < 16; ++w) v += dsum[w];
    __syncthreads();
    return v;
  };
  const int nh = a.n_kv * a.tiles;
  const float slots = (float)a.slots;
  double v = 0.0;
  for (int b = tid; b < a.B; b += 1024) v += (double)span_of(a, b).n;
  const float groups = (float)(block_sum(v) * nh);
  int c = per_split(groups, 2.0f * slots);
  if ((int64_t)a.B * nh <= a.slots) {
    int once = per_split(groups, slots);
    for (int i = 0; i < 3; ++i) {
      v = 0.0;
      for (int b = tid; b < a.B; b += 1024) v += (double)splits_of(span_of(a, b).n, once, 1.0f / (float)once);
      const float items = (float)(block_sum(v) * nh);
      if (items <= slots) break;
      once = fewer(once, items, slots);
    }
    c = choose(once, c, groups, slots);
  }
  const float inv = 1.0f / (float)c;
  uint32_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 1024) {
    const int b = b0 + tid;
    const uint32_t splits = b < a.B ? (uint32_t)splits_of(span_of(a, b).n, c, inv) : 0;
    const uint32_t incl = scan(splits);
    if (lane == 63) usum[wave] = incl;
    __syncthreads();
    uint32_t first = before + incl - splits;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) first += usum[w];
      before += usum[w];
    }
    if (b < a.B) {
      a.plan[2 * b] = (int32_t)first;
      a.plan[2 * b + 1] = (int32_t)splits;
      for (uint32_t i = 0; i < splits; ++i) a.units[1 + first + i] = b;
    }
    __syncthreads();
  }
  if (tid == 0) a.units[0] = (int32_t)before;
}

hipError_t launch_plan(const Args &a, hipStream_t s) {
  hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

// One workgroup per H query heads of a sequence: the splits' parts, weighted by
// 2^(R_i - max R), over the weighted sums (plus the sink's share).  Sequences
// of one split were finished by the attention kernel.  256 / H threads of a
// head compute its weights and sums together and read its parts in ways of
// D / 4 lanes, so that a sequence of a thousand splits costs no chain of a
// thousand loads.  H = 1 spreads few heads with many splits over the GPU (32
// heads of 96 splits 6 us), H = 4 makes fewer workgroups of many heads with few
// splits (48 sequences of 64 heads, 3 splits: 7.5 -> 4.7 us).  The change at 1024
// heads in all, sequences of 4096 with heads of 128, H = 1 and 4: 32 heads 5.4 and
// 5.9 us, 256 to 768 both 4.2 to 4.6, 1024 4.8 and 4.6, 1536 5.6 and 4.6, 2048 6.2
// and 4.6.
template <typename QT, int H>
__global__ __launch_bounds__(256) void join_kernel(Args a, int D) {
  constexpr int kThreads = 256 / H, kChunk = 1024 / H;
  __shared__ float weight[H][kChunk];
  __shared__ float red[H][8];
  __shared__ floatx4 part[256];
  const int sub = threadIdx.x / kThreads, tid = threadIdx.x % kThreads, lane = tid & 63, wave = tid >> 6;
  const int per_b = (a.n_q + H - 1) / H, b = blockIdx.x / per_b, hq = min((blockIdx.x - b * per_b) * H + sub, a.n_q - 1);
  const int first = a.plan[2 * b], splits = a.plan[2 * b + 1];
  if (splits <= 1) return;
  const int kvh = hq / a.G, in = hq - kvh * a.G, tile = in / 16, h = in - tile * 16;
  const int64_t nh = (int64_t)a.n_kv * a.tiles, item0 = first * nh + tile * a.n_kv + kvh;
  const float *ml = a.part + a.items * a.heads * D;

  // The first parts load beside the references, whose weights they wait for.
  const int lanes = D / 4, ways = kThreads / lanes, way = tid / lanes, d4 = tid - way * lanes;
  const float *parts = a.part + (item0 * a.heads + h) * D + 4 * d4;
  const int64_t step = nh * a.heads * D;
  const bool early = way < ways && way < splits;
  floatx4 o = {0, 0, 0, 0};
  if (early) o = *(const floatx4 *)(parts + way * step);

  float Rm = kFloor;
  for (int i = tid; i < splits; i += kThreads) Rm = fmaxf(Rm, ml[((item0 + i * nh) * a.heads + h) * 2]);
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) Rm = fmaxf(Rm, __shfl_xor(Rm, k, 64));
  if constexpr (kThreads > 64) {
    if (lane == 0) red[sub][wave] = Rm;
    __syncthreads();
    Rm = fmaxf(fmaxf(red[sub][0], red[sub][1]), fmaxf(red[sub][2], red[sub][3]));
  }

  float l = 0.0f;
  for (int i0 = 0; i0 < splits; i0 += kChunk) {
    const int n = min(kChunk, splits - i0);
    if (i0) __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const float *m = ml + ((item0 + (i0 + i) * nh) * a.heads + h) * 2;
      const float w = __builtin_amdgcn_exp2f(m[0] - Rm);
      weight[sub][i] = w;
      l = __builtin_fmaf(w, m[1], l);
    }
    __syncthreads();
    if (i0 == 0 && early) o *= weight[sub][way];
    if (way < ways) {
#pragma unroll 4
      for (int i = way + (i0 ? 0 : ways); i < n; i += ways) o += weight[sub][i] * *(const floatx4 *)(parts + (i0 + i) * step);
    }
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) l += __shfl_xor(l, k, 64);
  if constexpr (kThreads > 64) {
    if (lane == 0) red[sub][4 + wave] = l;
  }
  part[threadIdx.x] = o;
  __syncthreads();
  if (tid >= lanes) return;
  if constexpr (kThreads > 64) l = (red[sub][4] + red[sub][5]) + (red[sub][6] + red[sub][7]);
  for (int k = 1; k < ways; ++k) o += part[sub * kThreads + k * lanes + tid];
  store_out((QT *)a.out + ((int64_t)b * a.n_q + hq) * D + 4 * tid, o, l, Rm, a.sinks, hq);
}

template <typename QT>
static void launch_join(const Args &a, int D, hipStream_t s) {
  if (a.B * a.n_q < 1024) hipLaunchKernelGGL((join_kernel<QT, 1>), dim3((unsigned)(a.B * a.n_q)), dim3(256), 0, s, a, D);
  else hipLaunchKernelGGL((join_kernel<QT, 4>), dim3((unsigned)(a.B * ((a.n_q + 3) / 4))), dim3(256), 0, s, a, D);
}

// The plan and, beyond 64 sequences, the splits' sequences: at most 2 slots /
// heads + one a sequence of them (per_split).
static size_t plan_bytes(int64_t B) {
  return (size_t)((B * 8 + (B > kLanes ? (1 + 2 * kMaxSlots + B) * 4 : 0) + 15) / 16 * 16);
}

}  // namespace attn

size_t attn_workspace_bytes(int64_t B, int64_t n_q, int64_t n_kv, int64_t head_dim) {
  const int64_t G = n_q / n_kv, heads = G < 16 ? G : 16, items = 2 * attn::kMaxSlots + B * n_kv * ((G + 15) / 16);
  return attn::plan_bytes(B) + (size_t)(items * heads * (head_dim + 2) * 4);
}

hipError_t launch_attn_decode(const KvCache &kc, const AttnDecode &d, hipStream_t s) {
  using namespace attn;
  Args a{};
  a.kp = (const uint8_t *)kc.k_pages, a.vp = (const uint8_t *)kc.v_pages;
  a.k_page_bytes = kv_page_bytes(kc.k_kind, kc.page_size, kc.n_kv, kc.head_dim);
  a.v_page_bytes = kv_page_bytes(kc.v_kind, kc.page_size, kc.n_kv, kc.head_dim);
  a.n_pages = kc.n_pages;
  a.page_groups = (int)(kc.page_size / kv::kGroup);
  a.n_kv = (int)kc.n_kv, a.n_q = (int)d.n_q, a.G = a.n_q / a.n_kv;
  a.tiles = (a.G + 15) / 16, a.heads = a.G < 16 ? a.G : 16;
  a.q = d.q, a.q_stride = d.q_stride;
  a.table = d.table, a.max_pages = d.max_pages, a.lens = d.lens, a.B = (int)d.B;
  a.scale2 = d.scale * 1.44269504088896f;
  a.window = d.window, a.sinks = d.sinks, a.out = d.out;
  a.plan = (int32_t *)d.workspace;
  a.units = a.plan + 2 * d.B;
  a.part = (float *)((uint8_t *)d.workspace + plan_bytes(d.B));
  const int NB = (int)(kc.head_dim / 32);
  hipError_t e = hipErrorInvalidValue;
#define QMM_CASE(K, V, F) \
  if (kc.k_kind == K && kc.v_kind == V) e = F(a, NB, d.f16, s);
  QMM_CASE(C_F16, C_F16, launch_f16_f16)
  QMM_CASE(C_F16, C_Q8_0, launch_f16_q8)
  QMM_CASE(C_F16, C_Q4_0, launch_f16_q4)
  QMM_CASE(C_Q8_0, C_F16, launch_q8_f16)
  QMM_CASE(C_Q8_0, C_Q8_0, launch_q8_q8)
  QMM_CASE(C_Q8_0, C_Q4_0, launch_q8_q4)
  QMM_CASE(C_Q4_0, C_F16, launch_q4_f16)
  QMM_CASE(C_Q4_0, C_Q8_0, launch_q4_q8)
  QMM_CASE(C_Q4_0, C_Q4_0, launch_q4_q4)
#undef QMM_CASE
  if (e != hipSuccess) return e;
  // (A table of at most one split's tokens: the attention kernel has finished
  // every sequence.)
  if (a.max_pages * a.page_groups <= kMinGroups) return hipSuccess;
  if (d.f16) launch_join<_Float16>(a, (int)kc.head_dim, s);
  else launch_join<float>(a, (int)kc.head_dim, s);
  return hipGetLastError();
}

}  // namespace qmm
