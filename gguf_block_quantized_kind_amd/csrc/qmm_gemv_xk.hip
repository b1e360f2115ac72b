// qmm_gemv_xk.hip -- products of up to 8 tokens with an epilogue where there are few
// tiles of 16 weight rows: a workgroup a tile, its S waves split K.
//
// A wave does its k-blocks without the others: the tokens' activations of a
// k-block go, rounded to f16, through a part of LDS of its own into fragment
// order, the weights come as repacked records or as native rows, and the S sums
// meet in LDS at the end.  One k-block is decoded while the next one's loads are in
// flight; the rest of the waiting is hidden by the other waves of the SIMD, so a
// wave stays within the 128 registers that let sixteen share a compute unit.
//
// Native rows are loaded as the 16-byte granules that hold any byte of a k-block,
// neighbouring lanes neighbouring granules, and put in LDS; the lanes read their
// fields there.  A lane's fields in place, sixteen rows apart from its neighbours',
// cost the L1 an access each, 790 a k-block of Q6_K against 200.  Activations are
// loaded in element order for the same reason.
//
// The decoders are those of qmm_gemv_mfma.h.  Rows of the activation operand past
// the last token hold whatever is in LDS: each reaches its own row of the product
// alone, and those rows are not stored.
#include <algorithm>
#include <type_traits>

#include "qmm_epilogue.h"
#include "qmm_gemv_mfma.h"
#include "qmm_internal.h"

namespace qmm {
namespace gv {

// Fields of a block that begins `by` bytes into a word (wide reads of LDS from
// between words take a cycle a lane).
template <int WORDS>
__device__ __forceinline__ void words_at(const uint32_t *p, int by, uint32_t (&v)[WORDS]) {
  uint32_t w[WORDS + 1];
#pragma unroll
  for (int i = 0; i <= WORDS; ++i) w[i] = p[i];
#pragma unroll
  for (int i = 0; i < WORDS; ++i) v[i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], by);
}
__device__ __forceinline__ u32x4 four_at(const uint32_t *p, int by) {
  uint32_t v[4];
  words_at(p, by, v);
  return u32x4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ u32x2 two_at(const uint32_t *p, int by) {
  uint32_t v[2];
  words_at(p, by, v);
  return u32x2{v[0], v[1]};
}
__device__ __forceinline__ uint32_t one_at(const uint32_t *p, int by) {
  uint32_t v[1];
  words_at(p, by, v);
  return v[0];
}
__device__ __forceinline__ void fields_at(const uint32_t *p, int by, int G, DecQ6K::Raw &r) {
  const int h = G >> 1, a = G & 1;
  r.ql0 = four_at(p + 16 * h + 4 * a, by);
  r.ql1 = four_at(p + 16 * h + 8 + 4 * a, by);
  r.qh = four_at(p + 32 + 8 * h + 4 * a, by);
  r.sc = two_at(p + 48 + 2 * h, by);
  r.d = one_at(p + 52, by);  // in the low half
}
__device__ __forceinline__ void fields_at(const uint32_t *p, int by, int G, DecQ3K::Raw &r) {
  r.hm = four_at(p + 4 * (G & 1), by);
  r.q = four_at(p + 8 + 4 * G, by);
  r.lo = two_at(p + 24, by);
  r.hi = one_at(p + 26, by);
  r.d = one_at(p + 27, by);
}

// A k-block of 16 native rows as granules: granule c % kRow of row c / kRow to lane c
// % 64's part c / 64.  In LDS rows are an odd number of granules apart, so that the
// same field of 16 rows falls on different banks.
template <typename Dd>
struct Granules {
  static constexpr int kRow = (Dd::BYTES + 30) / 16, kParts = (16 * kRow + 63) / 64;
  static constexpr int kStride = 16 * (kRow | 1), kBytes = 16 * kStride;
  struct Held { u32x4 part[kParts]; };
  const uint8_t *base;        // the tile's first row, rounded down to a granule
  int start[kParts], mine;    // from base to the beginning of a part's row, of row j
  __device__ __forceinline__ void init(const uint8_t *P, int64_t tile, int64_t N, int64_t row_bytes, int lane, int j) {
    const uint8_t *first = P + tile * 16 * row_bytes;
    const int low = (int)((uintptr_t)first & 15), last = (int)min<int64_t>(N - 1 - tile * 16, 15);
    base = first - low;
#pragma unroll
    for (int i = 0; i < kParts; ++i) start[i] = low + min((64 * i + lane) / kRow, last) * (int)row_bytes;
    mine = low + min(j, last) * (int)row_bytes;
  }
  __device__ __forceinline__ void load(int kb, int lane, Held &h) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const int from = start[i] + kb * Dd::BYTES;
      h.part[i] = lda16(base + min((from & ~15) + (64 * i + lane) % kRow * 16, (from + Dd::BYTES - 1) & ~15));
    }
  }
  __device__ __forceinline__ void store(uint8_t *lds, int lane, const Held &h) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const int c = 64 * i + lane;
      if (c < 16 * kRow) *reinterpret_cast<u32x4 *>(lds + c / kRow * kStride + c % kRow * 16) = h.part[i];
    }
  }
  __device__ __forceinline__ void fields(const uint8_t *lds, int kb, int j, int G, typename Dd::Raw &r) const {
    const int at = mine + kb * Dd::BYTES & 15;
    if constexpr (Dd::BYTES % 4 == 0) Dd::load(lds + j * kStride + at, G, r);
    else fields_at(reinterpret_cast<const uint32_t *>(lds + j * kStride + (at & 12)), at & 3, G, r);
  }
};

// Fragments in LDS: a group's tokens side by side, so that a read of them is one run;
// groups MT + 1 apart and steps two more than their groups take, so that a write's
// groups, steps and halves fall on different banks in each decoder's order.
constexpr int group_of(int MT) { return MT + 1; }
constexpr int step_of(int MT) { return 4 * group_of(MT) + 2; }
template <int KIND, int MT, bool PACKED>
constexpr int wave_bytes() {
  return Dec<KIND>::NSTEP * step_of(MT) * 16 + (PACKED ? 0 : Granules<Dec<KIND>>::kBytes);
}

template <int KIND, typename XT, int MT, int S, bool PACKED>
__global__ __launch_bounds__(64 * S) void gemv_xk_kernel(const uint8_t *__restrict__ P, const XT *__restrict__ X,
                                                         const Epilogue Y, int M, int64_t N, int K, int64_t row_bytes) {
  using Dd = Dec<KIND>;
  using X4 = typename XVec<XT>::type;
  constexpr int kStep = step_of(MT);
  constexpr int64_t kRec = 16 * Dd::BYTES;  // one repacked record
  static_assert(Dd::KB == 256 && Dd::NSTEP == 8, "a half of four elements a lane and token");
  extern __shared__ u32x4 lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int j = lane & 15, G = lane >> 4;
  const int64_t tile = blockIdx.x;
  const int nkb = K / Dd::KB, kb0 = (int)((int64_t)wave * nkb / S), kb1 = (int)((int64_t)(wave + 1) * nkb / S);
  uint8_t *own = reinterpret_cast<uint8_t *>(lds) + wave * wave_bytes<KIND, MT, PACKED>();
  uint8_t *rows = own + Dd::NSTEP * kStep * 16;

  // Lane u stages elements 4 u .. 4 u + 3 of every token.  Each bit of (half, group,
  // step) moves x_off by a power of two of its own.
  auto bit = [&](int by) { return lane / (by / 4) & 1; };
  const int g2 = bit(Dd::x_off(0, 1, 0)) | bit(Dd::x_off(0, 2, 0)) << 1;
  const int st = bit(Dd::x_off(1, 0, 0)) | bit(Dd::x_off(2, 0, 0)) << 1 | bit(Dd::x_off(4, 0, 0)) << 2;
  uint8_t *to = own + (st * kStep + g2 * group_of(MT)) * 16 + 8 * bit(Dd::x_off(0, 0, 1));
  const u32x4 *from = reinterpret_cast<const u32x4 *>(own) + G * group_of(MT) + j % MT;

  typename std::conditional<PACKED, typename Rec<KIND>::Packed, typename Granules<Dd>::Held>::type raw[2];
  Granules<Dd> gran;
  if constexpr (!PACKED) gran.init(P, tile, N, row_bytes, lane, j);
  X4 x[MT];
  auto load_w = [&](int kb, int slot) {
    if constexpr (PACKED) Rec<KIND>::load(P + (tile * nkb + kb) * kRec, lane, j, G, raw[slot]);
    else gran.load(kb, lane, raw[slot]);
  };
  auto load_x = [&](int kb) {
#pragma unroll
    for (int i = 0; i < MT; ++i) __builtin_memcpy(&x[i], X + (int64_t)min(i, M - 1) * K + kb * Dd::KB + 4 * lane, sizeof(X4));
  };
  // Between this wave's writes and reads of LDS, which it does in order.
  auto ordered = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };

  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  auto round = [&](int kb, int slot) {
    ordered();
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const half2v p0 = {(_Float16)x[i][0], (_Float16)x[i][2]}, p1 = {(_Float16)x[i][1], (_Float16)x[i][3]};
      *reinterpret_cast<u32x2 *>(to + 16 * i) = u32x2{as_u(p0), as_u(p1)};
    }
    if constexpr (!PACKED) gran.store(rows, lane, raw[slot]);
    const int next = min(kb + 1, kb1 - 1);
    load_x(next);
    load_w(next, slot ^ 1);
    ordered();
    typename Dd::Raw fr;
    if constexpr (PACKED) fr = Rec<KIND>::unpack(raw[slot], G);
    else gran.fields(rows, kb, j, G, fr);
    const typename Dd::Sc sc = Dd::prep(fr, G);
    if constexpr (Dd::STEP_SCALE) {
#pragma unroll
      for (int s = 0; s < Dd::NSTEP; ++s) {
        const half8 a = __builtin_bit_cast(half8, from[s * kStep]);
        acc = Dd::post_step(acc, mfma16(a, Dd::bop(fr, sc, s, 0), floatx4{0.f, 0.f, 0.f, 0.f}), fr, s);
      }
    } else {
      floatx4 D[Dd::NPART], xsum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < Dd::NPART; ++p) D[p] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < Dd::NSTEP; ++s) {
        const half8 a = __builtin_bit_cast(half8, from[s * kStep]);
        if constexpr (Dd::HAS_MIN) {
          const _Float16 v = Dd::ind(s, G, j) ? (_Float16)1.0f : (_Float16)0.0f;
          xsum = mfma16(half8{v, v, v, v, v, v, v, v}, a, xsum);
        }
#pragma unroll
        for (int p = 0; p < Dd::NPART; ++p) D[p] = mfma16(a, Dd::bop(fr, sc, s, p), D[p]);
      }
      acc = Dd::post(acc, D, xsum, sc);
    }
  };

  if (kb0 < kb1) {
    load_x(kb0);
    load_w(kb0, 0);
    int kb = kb0;
    for (; kb + 2 <= kb1; kb += 2) {
      round(kb, 0);
      round(kb + 1, 1);
    }
    if (kb < kb1) round(kb, 0);
  }

  // Lane (j, G) of the first wave stores D[token 4G + q][row j]; what goes into that
  // besides the sum is loaded while the others end.
  const int64_t row = tile * 16 + j;
  Operands around[4];
  if (wave == 0 && row < N) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (4 * G + q < M) around[q] = operands(Y, 4 * G + q, row);
  }
  __syncthreads();  // every wave is done with its part of LDS
  floatx4 *red = reinterpret_cast<floatx4 *>(lds);
  if (wave > 0) red[(wave - 1) * 64 + lane] = acc;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int q = 1; q < S; ++q) acc += red[(q - 1) * 64 + lane];
  if (row >= N) return;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (4 * G + q < M) put(Y, 4 * G + q, row, N, acc[q], around[q]);
}

template <int KIND, typename XT, int MT, int S, bool PACKED>
static hipError_t run_xk(const uint8_t *P, const XT *x, const Epilogue &y, int M, int64_t N, int64_t K, hipStream_t s) {
  const size_t lds = std::max<size_t>((size_t)S * wave_bytes<KIND, MT, PACKED>(), (size_t)(S - 1) * 64 * 16);
  hipLaunchKernelGGL((gemv_xk_kernel<KIND, XT, MT, S, PACKED>), dim3((unsigned)((N + 15) / 16)), dim3(64 * S), lds, s, P, x,
                     y, M, N, (int)K, (K / Geometry<KIND>::elems) * Geometry<KIND>::bytes);
  return hipGetLastError();
}

template <int KIND, typename XT, bool PACKED, int S>
static hipError_t run_xk_m(const uint8_t *P, const XT *x, const Epilogue &y, int M, int64_t N, int64_t K, hipStream_t s) {
  if (M <= 2) return run_xk<KIND, XT, 2, S, PACKED>(P, x, y, M, N, K, s);
  if (M <= 4) return run_xk<KIND, XT, 4, S, PACKED>(P, x, y, M, N, K, s);
  return run_xk<KIND, XT, 8, S, PACKED>(P, x, y, M, N, K, s);
}

template <int KIND, typename XT, bool PACKED>
static hipError_t run_xk_s(const uint8_t *P, const XT *x, const Epilogue &y, int M, int64_t N, int64_t K, hipStream_t s) {
  const int64_t tiles = (N + 15) / 16, nkb = K / 256, cus = device_cus();
  if (nkb <= 4 || K > (int64_t)1 << 20) return hipErrorNotSupported;
  if (tiles <= cus) {
    if constexpr (std::is_same<XT, _Float16>::value && (PACKED || (KIND != Q6_K && KIND != Q5_K)))
      if (nkb <= 32) return run_xk_m<KIND, XT, PACKED, 16>(P, x, y, M, N, K, s);
    return run_xk_m<KIND, XT, PACKED, 8>(P, x, y, M, N, K, s);
  }
  if constexpr (!PACKED && (KIND == Q6_K || KIND == Q3_K))
    if (KIND == Q6_K || tiles <= 2 * cus) return run_xk_m<KIND, XT, PACKED, 4>(P, x, y, M, N, K, s);
  return hipErrorNotSupported;
}

template <int KIND, bool PACKED>
static hipError_t run_xk_x(const uint8_t *P, const void *x, int x_f16, const Epilogue &y, int M, int64_t N, int64_t K,
                           hipStream_t s) {
  if (x_f16) return run_xk_s<KIND, _Float16, PACKED>(P, static_cast<const _Float16 *>(x), y, M, N, K, s);
  return run_xk_s<KIND, float, PACKED>(P, static_cast<const float *>(x), y, M, N, K, s);
}

}  // namespace gv

// hipErrorNotSupported where qmm_gemv_xs.hip's shapes are faster (figures: eight
// tokens in us, those shapes first).
//
// Up to a tile a compute unit: eight waves of K, sixteen up to 32 k-blocks where a
// wave stays within 128 registers (f16 activations, Q4_K 4096 x 4096 7.4 with eight,
// 6.7).  4096 x 14336 native Q6_K 23.4 -> 19.1, Q4_K 17.6 -> 13.6, Q5_K 21.6 -> 16.9,
// repacked Q4_0 13.7 -> 12.1, Q8_0 19.1 -> 18.0; 4096 x 4096 native Q6_K 11.3 -> 9.2,
// Q4_K 8.9 -> 6.7, Q5_K 10.4 -> 8.1, repacked Q8_0 8.5 -> 7.4, Q4_0 7.3 -> 6.1.
//
// More tiles: four waves of K for the native kinds whose fields lie between words.
// Q6_K 14336 x 4096 23.7 -> 22.2, 32768 x 4096 44.1 -> 40.3; Q3_K 8192 x 4096 13.0 ->
// 12.4, 5120 x 5120 13.8 -> 12.9, 14336 x 4096 even.  (Repacked Q6_K 8192 x 4096 10.8
// -> 11.4, Q8_0 11.6 -> 12.2.)
//
// (All with operands from memory; where they stay in the 256 MB behind L2 the first takes
// 15.6.)
//
// Bound: 4096 x 14336 Q6_K is 48 MB, 8.7 us at a large read's rate; launch, first loads and
// the sums' meeting take 6 us of any call, the decoding 270 instructions a wave and
// k-block.
hipError_t launch_gemv_xk(int kind, const uint8_t *W, bool packed, const void *x, int x_f16, const Epilogue &y, int M, int64_t N,
                          int64_t K, hipStream_t s) {
  if (packed) {
    switch (kind) {
#define QMM_CASE(K_) \
  case K_: return gv::run_xk_x<K_, true>(W, x, x_f16, y, M, N, K, s);
      QMM_FOR_EACH_KIND(QMM_CASE)
#undef QMM_CASE
      default: return hipErrorNotSupported;
    }
  }
  switch (kind) {
#define QMM_CASE(K_) \
  case K_: return gv::run_xk_x<K_, false>(W, x, x_f16, y, M, N, K, s);
    QMM_CASE(Q4_K) QMM_CASE(Q6_K) QMM_CASE(Q2_K) QMM_CASE(Q3_K) QMM_CASE(Q5_K)
#undef QMM_CASE
    default: return hipErrorNotSupported;
  }
}

}  // namespace qmm
