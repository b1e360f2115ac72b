// qmm_rope.hip -- rotary positions.  Pair (a, b) of a row at position p turns
// by the angle phi = p * freqs[i]:
//   y_a = m (x_a cos phi - x_b sin phi),  y_b = m (x_a sin phi + x_b cos phi)
// with (a, b) = (i, i + n_rot / 2) or (2i, 2i + 1); elements past n_rot pass.
// Each element is read and written once, by the thread that holds its pair
// (so y may be x): the bound is the memory traffic.  8192 tokens of 32 heads of
// 128, f32 to f16 (201 MB): 39.4 us, 5.1 TB/s, the rate of a large copy; a
// thread per pair that finds its own angle took 65.
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {
namespace kv {

template <typename T, typename O, int V>
__global__ __launch_bounds__(256) void rope_kernel(Rotate r) {
  rotate_rows<T, O, V>(r, (int64_t)blockIdx.x * 256 + threadIdx.x);
}

template <typename T, typename O>
static hipError_t run_rope(Rotate &r, hipStream_t s) {
  int64_t threads;
  const bool wide = plan_rotate(r, sizeof(T), sizeof(O), threads);
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (wide) hipLaunchKernelGGL((rope_kernel<T, O, 4>), grid, dim3(256), 0, s, r);
  else hipLaunchKernelGGL((rope_kernel<T, O, 1>), grid, dim3(256), 0, s, r);
  return hipGetLastError();
}

}  // namespace kv

hipError_t launch_rope(const KvWrite &w, int64_t H, int64_t D, hipStream_t s) {
  kv::Rotate r{};
  r.x = w.q, r.y = w.q_out, r.x_stride = w.q_stride, r.y_stride = w.q_out_stride;
  r.pos = w.pos, r.T = w.T, r.H = (int)H, r.D = (int)D;
  r.rope = kv::Rope{w.freqs, (int)w.n_rot, w.interleaved, w.mscale};
  if (w.f16) return w.q_out_f16 ? kv::run_rope<_Float16, _Float16>(r, s) : kv::run_rope<_Float16, float>(r, s);
  return w.q_out_f16 ? kv::run_rope<float, _Float16>(r, s) : kv::run_rope<float, float>(r, s);
}

}  // namespace qmm
