// qmm_repack.hip -- the load-time repack of native GGUF rows into the
// lane-ordered records that the repacked GEMV reads (Vulkore quant_test.cpp,
// section 4, "repacked fast path": a one-time transform at load so that the
// matvec reads aligned planes).
//
// Record layout (also described at Rec in qmm_gemv_mfma.h): rows are grouped
// in tiles of 16, the last tile padded with zero rows; K in k-blocks of 256
// elements, B bytes per row per k-block.  Tile t, k-block b is one record of
// 16 B bytes at (t * n_kblocks + b) * 16 B.  A record is n_lane lane sections
// of 1024 bytes (slot 16 G + j: 16 bytes of row j chosen by G), then row
// sections (slot j: w bytes of row j).  The repack is a byte permutation, so
// it is lossless and the repacked tensor is the native size plus padding.
#include "qmm_device.h"
#include "qmm_internal.h"
#include "qmm_records.h"

namespace qmm {
namespace rp {

// One thread per 4 bytes of the repacked tensor (records are multiples of
// 16 bytes).  Rows past N read as zero.
template <int KIND>
__global__ __launch_bounds__(256) void repack_kernel(const uint8_t *__restrict__ W, uint32_t *__restrict__ P,
                                                     int64_t N, int64_t nkb, int64_t words) {
  constexpr int B = Map<KIND>::shape.B;
  constexpr int kRec = 16 * B;
  const int64_t w = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (w >= words) return;
  const int64_t byte = 4 * w;
  const int64_t rec = byte / kRec;
  const int o = (int)(byte - rec * kRec);
  const int64_t tile = rec / nkb, kb = rec - tile * nkb;
  const int64_t row_bytes = nkb * B;
  uint32_t v = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    int j, off;
    source<KIND>(o + b, j, off);
    const int64_t row = tile * 16 + j;
    const uint32_t x = row < N ? W[row * row_bytes + kb * B + off] : 0u;
    v |= x << (8 * b);
  }
  P[w] = v;
}

template <int KIND>
hipError_t run(const uint8_t *W, void *P, int64_t N, int64_t K, hipStream_t s) {
  const int64_t nkb = K / 256;
  const int64_t words = packed_bytes_of(KIND, N, K) / 4;
  const int64_t blocks = (words + 255) / 256;
  hipLaunchKernelGGL(repack_kernel<KIND>, dim3((unsigned)blocks), dim3(256), 0, s, W, (uint32_t *)P, N, nkb, words);
  return hipGetLastError();
}

}  // namespace rp

int64_t packed_bytes_of(int kind, int64_t N, int64_t K) {
  int B;
  switch (kind) {
    case Q4_0: case IQ4_NL: case Q4_K: B = 144; break;
    case MXFP4: case IQ4_XS: B = 136; break;
    case Q5_0: B = 176; break;
    case Q8_0: B = 272; break;
    case Q6_K: B = 210; break;
    case Q5_K: B = 176; break;
    case Q2_K: B = 84; break;
    case Q3_K: B = 110; break;
    default: return -1;
  }
  if (K <= 0 || K % 256 != 0 || N <= 0) return -1;
  return (N + 15) / 16 * 16 * (K / 256) * B;
}

hipError_t launch_repack(int kind, const uint8_t *W, void *P, int64_t N, int64_t K, hipStream_t s) {
  switch (kind) {
    case Q4_0: return rp::run<Q4_0>(W, P, N, K, s);
    case IQ4_NL: return rp::run<IQ4_NL>(W, P, N, K, s);
    case MXFP4: return rp::run<MXFP4>(W, P, N, K, s);
    case Q5_0: return rp::run<Q5_0>(W, P, N, K, s);
    case Q8_0: return rp::run<Q8_0>(W, P, N, K, s);
    case IQ4_XS: return rp::run<IQ4_XS>(W, P, N, K, s);
    case Q4_K: return rp::run<Q4_K>(W, P, N, K, s);
    case Q6_K: return rp::run<Q6_K>(W, P, N, K, s);
    case Q5_K: return rp::run<Q5_K>(W, P, N, K, s);
    case Q2_K: return rp::run<Q2_K>(W, P, N, K, s);
    case Q3_K: return rp::run<Q3_K>(W, P, N, K, s);
    default: break;
  }
  return hipErrorNotSupported;
}

}  // namespace qmm
