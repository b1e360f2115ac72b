// qmm_gemm_w16.hip -- the prefill product of many tokens, with an epilogue: the
// weights are decoded once to f16 into a workspace, f32 activations once into
// two f16 planes, and an f16 GEMM multiplies those.
//
// Decoding inside a GEMM is done again for every token tile; at a thousand
// tokens it, and the registers it takes, hold those kernels to a third of the
// matrix cores' rate, while writing and reading N K f16 weights takes a small
// part of the product's time.  Numerics are those of the other GEMMs: each weight
// rounded once to f16, f16 activations exact, f32 ones as hi = RN_f16(a) and lo
// = RN_f16(a - hi), both multiplied; f32 accumulation in a fixed order.
//
// GEMM.  A workgroup of WM x WN waves owns BM tokens by BN weight rows; a wave
// TM x TN tiles of 16 x 16.  Both operands are rows of K, staged 32 elements
// (64 bytes) at a time through LDS by direct-to-LDS loads in four rings: stage t
// + 3 is loading while stage t is multiplied and stage t + 1's fragments are read
// into the registers that stage t's leave, so neither LDS nor memory is waited
// for in between, and one barrier a stage orders the rings.  A row's four
// 16-byte chunks lie at chunk ^ (row / 2 % 4): the 16 rows of a fragment read
// fall on all banks.  The matrix instruction takes weights as its rows, so a lane
// ends with four neighbouring columns of one token; the epilogue passes them
// through LDS and takes eight columns a thread, whole rows a wave.
//
// Workgroups are numbered so that each XCD (workgroup i runs on XCD i mod 8)
// takes a contiguous range of tiles, eight token tiles after one another for a
// weight tile, then the next weight tile: the 32 that an XCD works on at a time read
// 8 + 4 operand tiles through its L2 (8192 tokens, 8192 x 4096 Q4_K, no
// activation: 497 us; all token tiles after one another 535).
//
// Bound (2048 tokens, 8192 x 4096: 118 us in one round of tiles): the matrix
// instructions fill 58% of its cycles, at the 1.6 to 1.9 GHz that the power leaves
// (activations of zeros take 20% less time, a library's f16 product 12% less).
// Measured and left: five rings, fewer waves with 128 x 128 each, 32 x 32 matrix
// tiles and 256 x 224 tiles all took as long or longer.
#include "qmm_device.h"
#include "qmm_epilogue.h"
#include "qmm_internal.h"
#include "qmm_records.h"

namespace qmm {
namespace w16 {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// --------------------------------------------------------------------------
// Weights and activations to f16
// --------------------------------------------------------------------------
__device__ __forceinline__ void store16(_Float16 *out, const float (&v)[16]) {
  half8 h[2];
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i / 8][i % 8] = (_Float16)v[i];
  reinterpret_cast<half8 *>(out)[0] = h[0];
  reinterpret_cast<half8 *>(out)[1] = h[1];
}

// 16 elements a thread; rows are stored back to back, as the blocks are.
template <int KIND>
__global__ __launch_bounds__(256) void decode_kernel(const uint8_t *__restrict__ W, _Float16 *__restrict__ out,
                                                     int64_t n_subs) {
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (t >= n_subs) return;
  float v[16];
  decode16<KIND>(W + t / kSubs<KIND> * Geometry<KIND>::bytes, (int)(t % kSubs<KIND>), v);
  store16(out + t * 16, v);
}

// The same from repacked records: a workgroup puts a record's bytes back into
// sixteen native k-blocks in LDS and decodes those.
template <int KIND>
__global__ __launch_bounds__(256) void decode_records_kernel(const uint8_t *__restrict__ P, _Float16 *__restrict__ out,
                                                             int64_t N, int64_t nkb, int64_t records) {
  constexpr int B = rp::Map<KIND>::shape.B;
  __shared__ uint8_t rows[16 * B];
  const int64_t rec = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (rec >= records) return;  // the whole workgroup
  for (int o = 4 * threadIdx.x; o < 16 * B; o += 4 * 256) {
    const uint32_t v = *reinterpret_cast<const uint32_t *>(P + rec * 16 * B + o);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      int j, off;
      rp::source<KIND>(o + b, j, off);
      rows[j * B + off] = (uint8_t)(v >> (8 * b));
    }
  }
  __syncthreads();
  const int j = threadIdx.x / 16, sub = threadIdx.x % 16;
  const int64_t tile = rec / nkb, kb = rec - tile * nkb, row = tile * 16 + j;
  if (row >= N) return;
  float v[16];
  decode16<KIND>(rows + j * B + sub / kSubs<KIND> * Geometry<KIND>::bytes, sub % kSubs<KIND>, v);
  store16(out + (row * nkb + kb) * 256 + sub * 16, v);
}

// Planes hi and lo of n f32 activations (n a multiple of 4).
__global__ __launch_bounds__(256) void split_kernel(const float *__restrict__ A, _Float16 *__restrict__ hi,
                                                    _Float16 *__restrict__ lo, int64_t n) {
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (4 * t >= n) return;
  float a[4];
  __builtin_memcpy(a, A + 4 * t, sizeof a);
  half4 h, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = (_Float16)a[i];
    l[i] = (_Float16)(a[i] - (float)h[i]);
  }
  reinterpret_cast<half4 *>(hi)[t] = h;
  reinterpret_cast<half4 *>(lo)[t] = l;
}

// --------------------------------------------------------------------------
// The GEMM
// --------------------------------------------------------------------------
constexpr int kRsrcWord3 = 0x00020000;  // buffer descriptor word 3 (raw 32-bit data)
constexpr int vmcnt_imm(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0F70; }
constexpr int kRing = 4;
constexpr int kGroup = 8;  // token tiles that share weight tiles, one after another

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t *lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, voff, soff, 0, 0);
}

// Columns n .. n + 7 of token m.
__device__ __forceinline__ void load8(const void *p, int f16, int64_t at, float (&r)[8]) {
  if (f16) {
    half8 h;
    __builtin_memcpy(&h, static_cast<const _Float16 *>(p) + at, sizeof h);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (float)h[i];
  } else {
    __builtin_memcpy(r, static_cast<const float *>(p) + at, sizeof r);
  }
}
template <int ACT>
__device__ __forceinline__ void activate8(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activated(ACT, v[i]);
}
__device__ __forceinline__ void put8(const Epilogue &e, int64_t m, int64_t n, int64_t N, float (&v)[8]) {
  if (n + 8 > N) {
    for (int i = 0; i < 8 && n + i < N; ++i) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) x = k == i ? v[k] : x;
      put(e, m, n + i, N, x);
    }
    return;
  }
  float b[8], f[8], r[8];
  if (e.bias) load8(e.bias, 0, n, b);
  if (e.mul) load8(e.mul, e.mul_f16, m * e.mul_stride + n, f);
  if (e.residual) load8(e.residual, e.residual_f16, m * e.residual_stride + n, r);
  if (e.bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  switch (e.act) {
    case QMM_ACT_RELU: activate8<QMM_ACT_RELU>(v); break;
    case QMM_ACT_SILU: activate8<QMM_ACT_SILU>(v); break;
    case QMM_ACT_GELU: activate8<QMM_ACT_GELU>(v); break;
    case QMM_ACT_GELU_TANH: activate8<QMM_ACT_GELU_TANH>(v); break;
    default: break;
  }
  if (e.mul) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= f[i];
  }
  if (e.residual) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  if (e.out_f16) {
    half8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
    __builtin_memcpy(static_cast<_Float16 *>(e.out) + m * e.out_stride + n, &h, sizeof h);
  } else {
    __builtin_memcpy(static_cast<float *>(e.out) + m * e.out_stride + n, v, sizeof v);
  }
}

// A: `planes` planes of [M][K], one after the other; W [N][K].  K a multiple
// of BK (32 or 64).
template <int WM, int WN, int TM, int TN, int BK>
__global__ __launch_bounds__(64 * WM * WN, 1) void gemm_kernel(const _Float16 *__restrict__ W,
                                                               const _Float16 *__restrict__ A, const Epilogue C,
                                                               int M, int N, int K, int planes, int tiles_m) {
  constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN, NW = WM * WN;
  constexpr int RB = BK * 2, CPR = RB / 16, RPL = 64 / CPR;  // bytes and chunks of a row, rows of a wave's load
  constexpr int kLoadsA = BM / RPL / NW, kLoadsW = BN / RPL / NW, kLoads = kLoadsA + kLoadsW;  // a wave's, a stage
  constexpr int kBytes = (BM + BN) * RB;                     // of a ring
  constexpr int KS = BK / 32;
  static_assert(BM % (RPL * NW) == 0 && BN % (RPL * NW) == 0, "as many loads of either operand for every wave");
  // Where chunk c of row r lies: c ^ key(r), so that a fragment read's 16 rows
  // fall on all banks.
  auto key = [](int r) { return CPR >= 8 ? r & 7 : (r >> 1) & 3; };
  __shared__ __attribute__((aligned(16))) uint8_t ring0[kBytes], ring1[kBytes], ring2[kBytes], ring3[kBytes];
  asm volatile("" ::"v"(ring0), "v"(ring1), "v"(ring2), "v"(ring3) : "memory");
  auto ring = [&](int u) -> uint8_t * { return u == 0 ? ring0 : u == 1 ? ring1 : u == 2 ? ring2 : ring3; };
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int G = lane >> 4, j = lane & 15;

  const int T = gridDim.x, L = blockIdx.x;
  const int xcd = L & 7, jx = L >> 3, q8 = T >> 3, r8 = T & 7;
  const int V = xcd < r8 ? xcd * (q8 + 1) + jx : r8 * (q8 + 1) + (xcd - r8) * q8 + jx;
  const int wide = kGroup * ((N + BN - 1) / BN), g0 = V / wide * kGroup, tall = min(kGroup, tiles_m - g0);
  const int m0 = (g0 + V % wide % tall) * BM, n0 = V % wide / tall * BN;

  // Loads: RPL rows each, lane l row l / CPR's chunk at position l % CPR.
  // Offsets are from the tile's first row; rows past the end read the last one.
  int voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const bool ofA = i < kLoadsA;
    const int r = (ofA ? wave * kLoadsA + i : wave * kLoadsW + i - kLoadsA) * RPL + lane / CPR;
    const int chunk = lane % CPR ^ key(r);
    voff[i] = min(r, ofA ? M - 1 - m0 : N - 1 - n0) * K * 2 + chunk * 16;
  }
  const int nst = K / BK * planes;
  // The next load's plane and bytes into its rows; past the last stage it stays there.
  const _Float16 *plane = A + (int64_t)m0 * K;
  int at = 0, left = planes - 1;
  const __amdgpu_buffer_rsrc_t wrs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16 *>(W + (int64_t)n0 * K), 0, 0x7FFFFFFF, kRsrcWord3);
  auto load = [&](int u) {
    const __amdgpu_buffer_rsrc_t ars = __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16 *>(plane), 0, 0x7FFFFFFF, kRsrcWord3);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool ofA = i < kLoadsA;
      dma16(ofA ? ars : wrs, ring(u) + 1024 * (ofA ? wave * kLoadsA + i : BM / RPL + wave * kLoadsW + i - kLoadsA), voff[i], at);
    }
    const bool end = at + RB == 2 * K, more = end && left > 0;
    at = more ? 0 : end ? at : at + RB;
    plane += more ? (int64_t)M * K : 0;
    left -= more;
  };

  int frag[KS];
#pragma unroll
  for (int h = 0; h < KS; ++h) frag[h] = j * RB + ((4 * h + G) ^ key(j)) * 16;
  half8 a[2][KS][TM], w[2][KS][TN];
  auto read = [&](int u, int p) {
    const uint8_t *ra = ring(u) + wm * TM * 16 * RB, *rw = ring(u) + (BM + wn * TN * 16) * RB;
#pragma unroll
    for (int h = 0; h < KS; ++h) {
#pragma unroll
      for (int i = 0; i < TN; ++i) w[p][h][i] = *reinterpret_cast<const half8 *>(rw + 16 * RB * i + frag[h]);
#pragma unroll
      for (int i = 0; i < TM; ++i) a[p][h][i] = *reinterpret_cast<const half8 *>(ra + 16 * RB * i + frag[h]);
    }
  };
  floatx4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int n = 0; n < TN; ++n) acc[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};

  // Until the loads of the stage before the last `later` issued ones are in
  // LDS, for every wave.
  auto arrive = [&](int imm) {
    __builtin_amdgcn_sched_barrier(0);
    if (imm == 2) __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * kLoads));
    else __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoads));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage t at ring u = t mod 4: its fragments are in registers p.
  auto stage = [&](int t, int u, int p) {
    arrive(1);                       // stage t + 1 is there; every wave has multiplied stage t - 1
    load((u + 3) % kRing);           // stage t + 3, over stage t - 1
    read((u + 1) % kRing, p ^ 1);
#pragma unroll
    for (int h = 0; h < KS; ++h)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int n = 0; n < TN; ++n)
          acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[p][h][n], a[p][h][i], acc[i][n], 0, 0, 0);
    // Products first, as both waves of a SIMD come here at once; then a fragment read
    // after every few, the loads between them.
    constexpr int kReads = KS * (TM + TN), kBetween = TM * TN / (TM + TN) > 0 ? TM * TN / (TM + TN) : 1;
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kBetween, 0);
      if ((i + 1) * kLoads / kReads > i * kLoads / kReads) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
  };

#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) load(s);
  arrive(2);
  read(0, 0);
  int t = 0;
  for (; t + kRing <= nst; t += kRing) {
#pragma unroll
    for (int u = 0; u < kRing; ++u) stage(t + u, u, u & 1);
  }
#pragma unroll
  for (int u = 0; u < kRing - 1; ++u)
    if (t + u < nst) stage(t + u, u, u & 1);
  // The last loads may still be landing in the rings.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();

  // The tile through LDS, 16 tokens of every wave at a time, so that rows are read
  // and written whole: 16-byte chunk c of row r (four columns) lies at chunk c ^
  // (r mod 16), which spreads a wave's writes of 16 rows over the banks.  Four rings
  // in turn: the barrier before a pass's reads also ends the reads of three passes
  // before.
  static_assert(16 * WM * BN * 4 <= kBytes && BN % 64 == 0, "a pass fits a ring, whole swizzles a row");
#pragma unroll 1
  for (int pass = 0; pass < TM; ++pass) {
    uint8_t *buf = ring(pass % kRing);
    // (Registers are named, not indexed: one branch a pass of this loop.)
#pragma unroll
    for (int k = 0; k < TM; ++k) {
      if (k != pass) continue;
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        const int c = (wn * TN + n) * 4 + G;
        *reinterpret_cast<floatx4 *>(buf + (wm * 16 + j) * BN * 4 + 16 * (c ^ j)) = acc[k][n];
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int x = threadIdx.x; x < 16 * WM * BN / 8; x += 64 * NW) {
      const int row = x / (BN / 8), c = x % (BN / 8) * 2;
      const int m = m0 + (row / 16 * TM + pass) * 16 + row % 16, n = n0 + 4 * c;
      if (m >= M || n >= N) continue;
      const floatx4 lo = *reinterpret_cast<const floatx4 *>(buf + row * BN * 4 + 16 * (c ^ (row & 15)));
      const floatx4 hi = *reinterpret_cast<const floatx4 *>(buf + row * BN * 4 + 16 * ((c + 1) ^ (row & 15)));
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      put8(C, m, n, N, v);
    }
  }
}

constexpr int64_t kGridX = 1 << 20;
dim3 grid_of(int64_t groups) {
  const int64_t wide = groups < kGridX ? groups : kGridX;
  return dim3((unsigned)wide, (unsigned)((groups + wide - 1) / wide));
}

template <int WM, int WN, int TM, int TN, int BK>
hipError_t run(const _Float16 *W, const _Float16 *A, const Epilogue &C, int64_t M, int64_t N, int64_t K, int planes,
               hipStream_t s) {
  constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN;
  const int64_t tm = (M + BM - 1) / BM, tn = (N + BN - 1) / BN;
  hipLaunchKernelGGL((gemm_kernel<WM, WN, TM, TN, BK>), dim3((unsigned)(tm * tn)), dim3(64 * WM * WN), 0, s, W, A, C, (int)M,
                     (int)N, (int)K, planes, (int)tm);
  return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace w16

// The crossings below were measured at 4096 x 4096, 14336 x 4096 and 4096 x 14336
// (rows x K); times in us.  Over 64, 256 and 1024 rows of 2048 and 7168 (64 to 4096
// tokens; Q8_0 and Q4_K as rows and as records, Q6_K) they are within a tenth of the
// fastest way at nine sizes of ten.  The others lie beside a crossing: f16 up to 1.5
// times (4096 tokens, 64 x 2048 Q8_0 17.2, decoded 12.1; 2048 tokens, 256 x 7168 Q4_K
// 43.3, decoded 28.0), f32 up to 1.9 (512 tokens, 1024 x 2048 repacked 26.5, by the
// GEMV's kernels 13.6, which round f32 activations to f16).
Way way_of(int kind, bool packed, int64_t M, int64_t N, int64_t K, int a_f16) {
  // Sixteen tokens at a time while the tiles of all of them are few: the GEMMs'
  // tiles of 64 tokens leave most compute units without work.  16 tokens, 4096 x
  // 4096: Q6_K 13.6 (GEMM 113, decoded 34), Q4_K 11.7 (24, 36), native Q8_0 10.8
  // (47, 34), repacked 9.6 (22, 34); at seven tiles a compute unit (32 tokens, 14336
  // x 4096) 39.7 (114, 47), 23.8 (26, 47), 42.7 (47, 49), 20.7 (23, 54), and beyond
  // them the others win.  IQ4_XS's GEMM over native rows wins from four on.
  const int64_t tiles = (N + 15) / 16 * ((M + 15) / 16);
  if (K % 256 == 0 && K <= (int64_t)1 << 20 && tiles <= device_cus() * (kind == IQ4_XS && !packed ? 4 : 7)) return Way::kGemv;
  // Offsets within a tile are 32-bit, and tiles are counted in 32 bits.
  const bool fits = K <= (int64_t)1 << 20 && (M + 63) / 64 * ((N + 63) / 64) < (int64_t)1 << 24;
  if (packed && !gemm_packed_supported(kind)) return Way::kDecoded;
  if (!fits) return Way::kGemm;
  // Decoded weights: their decoding costs as much at any number of tokens, the
  // GEMM over them less for each.  t: 64 x 64 tiles.
  const int64_t t = (M + 63) / 64 * ((N + 63) / 64);
  bool decoded;
  if (packed) {
    // f16: 512 tokens, 4096 x 4096 Q8_0 26.6 (decoded 43.6), 768 tokens 49.4 (43.5);
    // 512 tokens, 14336 x 4096 Q4_0 101 (86).  f32 takes two products: 256 tokens
    // 60 (46), unless its tiles of 64 x 128 just fill the units: 512 tokens 62 (70).
    // Records of 2^31 bytes and more are beyond that GEMM's offsets.
    const int64_t wide = (M + 63) / 64 * ((N + 127) / 128);
    decoded = packed_bytes_of(kind, N, K) >= (int64_t)1 << 31 || M > 512 || t >= 1792 ||
              (!a_f16 && !(2 * wide > device_cus() && wide <= device_cus()));
  } else {
    switch (kind) {
      // 64 tokens, 4096 x 4096 115 (33); 128 tokens, 14336 x 4096 66 (58).
      case Q6_K: decoded = true; break;
      // 512 tokens, 4096 x 4096 40.4 (42.1), 768 tokens 57.8 (42.9); f32 256 tokens
      // 42.6 (47.3), 512 tokens 78.7 (69.4).
      case Q4_K: decoded = t >= (a_f16 ? 640 : 480); break;
      // 512 tokens, 4096 x 4096 39.2 (44.7), 768 tokens 55.4 (46.5); f32 78.3 (73.1).
      case IQ4_XS: decoded = t >= (a_f16 ? 704 : 512); break;
      // 128 tokens, 14336 x 4096 Q5_K 46.9 (56.3), Q2_K 50.4 (55.5), 512 tokens, 4096
      // x 4096 48.2 (41.5), 51.1 (42.0); f32 256 tokens 51.4 (46.7), 53.7 (48.9).
      case Q5_K: case Q2_K: decoded = t >= (a_f16 ? 480 : 256); break;
      // 256 tokens, 4096 x 4096 39.3 (33.4), f32 59.5 (48.5).
      case Q3_K: decoded = t >= 256; break;
      // The 32-element kinds: 64 tokens, 4096 x 4096 Q8_0 48.5 (32.6), Q4_0 41.0
      // (34.3), 14336 x 4096 256 tokens 60.5 (60.0), 51.2 (56.6), 512 tokens 117 (88),
      // 99 (84); f32 64 tokens 80 (45).
      default: decoded = !a_f16 || N <= 8192 || t > 896; break;
    }
  }
  return decoded ? Way::kDecoded : Way::kGemm;
}

size_t gemm_w16_workspace_bytes(int kind, bool packed, int64_t M, int64_t N, int64_t K, int a_f16) {
  if (M <= QMM_GEMV_MAX_M || way_of(kind, packed, M, N, K, a_f16) != Way::kDecoded) return 0;
  return w16::align256((size_t)N * K * 2) + (a_f16 ? 0 : (size_t)M * K * 4);
}

hipError_t launch_gemm_w16(int kind, const uint8_t *W, bool packed, const void *A, int a_f16, Epilogue C, int64_t M,
                           int64_t N, int64_t K, void *ws, hipStream_t s) {
  using namespace w16;
  _Float16 *weights = static_cast<_Float16 *>(ws);
  const int64_t subs = N * K / 16, records = (N + 15) / 16 * (K / 256);
  switch (kind) {
#define QMM_CASE(K_)                                                                                                   \
  case K_:                                                                                                             \
    if (packed)                                                                                                        \
      hipLaunchKernelGGL(decode_records_kernel<K_>, grid_of(records), dim3(256), 0, s, W, weights, N, K / 256, records); \
    else                                                                                                               \
      hipLaunchKernelGGL(decode_kernel<K_>, grid_of((subs + 255) / 256), dim3(256), 0, s, W, weights, subs);            \
    break;
    QMM_FOR_EACH_KIND(QMM_CASE)
#undef QMM_CASE
    default: return hipErrorNotSupported;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const _Float16 *acts = static_cast<const _Float16 *>(A);
  if (!a_f16) {
    _Float16 *hi = reinterpret_cast<_Float16 *>(static_cast<uint8_t *>(ws) + align256((size_t)N * K * 2));
    hipLaunchKernelGGL(split_kernel, grid_of((M * K / 4 + 255) / 256), dim3(256), 0, s, static_cast<const float *>(A), hi,
                       hi + M * K, M * K);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    acts = hi;
  }
  // Tiles: of the three sizes the one whose rounds of the compute units take
  // least, a round counted as 95 (256 x 256), 34 (128 x 128) or 16 (64 x 64), its
  // measured time in us at K = 4096; smaller tiles go by longer stages of K where K
  // is whole ones.  1024 x 4096 x 4096: 95 / 45 / 71 us in all, 2048 x 14336 x 4096
  // 245 / 272 / 490, 256 x 4096 x 4096 97 / 42 / 31.
  const int planes = a_f16 ? 1 : 2;
  auto rounds = [&](int64_t bm, int64_t bn) {
    return ((M + bm - 1) / bm * ((N + bn - 1) / bn) + device_cus() - 1) / device_cus();
  };
  const int64_t large = 95 * rounds(256, 256), mid = 34 * rounds(128, 128), small = 16 * rounds(64, 64);
  if (large <= mid && large <= small) return run<2, 4, 8, 4, 32>(weights, acts, C, M, N, K, planes, s);
  if (mid <= small) {
    if (K % 64 == 0) return run<2, 4, 4, 2, 64>(weights, acts, C, M, N, K, planes, s);
    return run<2, 4, 4, 2, 32>(weights, acts, C, M, N, K, planes, s);
  }
  if (K % 128 == 0) return run<2, 2, 2, 2, 128>(weights, acts, C, M, N, K, planes, s);
  return run<2, 2, 2, 2, 32>(weights, acts, C, M, N, K, planes, s);
}

}  // namespace qmm
