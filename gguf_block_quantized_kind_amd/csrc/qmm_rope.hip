// qmm_rope.hip -- rotary positions.  Pair (a, b) of a row at position p turns
// by the angle phi = p * freqs[i]:
//   y_a = m (x_a cos phi - x_b sin phi),  y_b = m (x_a sin phi + x_b cos phi)
// with (a, b) = (i, i + n_rot / 2) or (2i, 2i + 1); elements past n_rot pass.
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {
namespace kv {

// One pair (or two passing elements) per thread, read before it is written,
// so y may be x.
template <typename T, typename O>
__global__ __launch_bounds__(256) void rope_kernel(Rope rp, const T *x, int64_t x_stride, O *y, int64_t y_stride,
                                                   const int32_t *__restrict__ pos, int64_t pairs, int H, int D) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= pairs) return;
  const int64_t row = p / (D / 2), t = row / H;
  const int i = (int)(p - row * (D / 2)), half = rp.n_rot >> 1;
  const int64_t h = (row - t * H) * D;
  const bool turned = i < half;
  const int da = turned && !rp.interleaved ? i : 2 * i;
  const int db = turned && !rp.interleaved ? i + half : 2 * i + 1;
  const float u = (float)x[t * x_stride + h + da], v = (float)x[t * x_stride + h + db];
  float c = 1.0f, s = 0.0f;
  if (turned) {
    rotation(pos[t], rp.freqs[i], c, s);
    c *= rp.mscale;
    s *= rp.mscale;
  }
  y[t * y_stride + h + da] = (O)(turned ? u * c - v * s : u);
  y[t * y_stride + h + db] = (O)(turned ? u * s + v * c : v);
}

}  // namespace kv

hipError_t launch_rope(const KvWrite &w, int64_t H, int64_t D, hipStream_t s) {
  const kv::Rope rp{w.freqs, (int)w.n_rot, w.interleaved, w.mscale};
  const int64_t pairs = w.T * H * (D / 2);
  const dim3 grid((unsigned)((pairs + 255) / 256));
#define QMM_LAUNCH(T, O)                                                                                         \
  hipLaunchKernelGGL((kv::rope_kernel<T, O>), grid, dim3(256), 0, s, rp, (const T *)w.q, w.q_stride, (O *)w.q_out, \
                     w.q_out_stride, w.pos, pairs, (int)H, (int)D)
  if (w.f16) {
    if (w.q_out_f16) QMM_LAUNCH(_Float16, _Float16);
    else QMM_LAUNCH(_Float16, float);
  } else {
    if (w.q_out_f16) QMM_LAUNCH(float, _Float16);
    else QMM_LAUNCH(float, float);
  }
#undef QMM_LAUNCH
  return hipGetLastError();
}

}  // namespace qmm
