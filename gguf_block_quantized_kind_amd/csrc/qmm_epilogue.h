// qmm_epilogue.h -- what a product does with each sum before it is stored.
//
// The product kernels write through QMM_OUT and put().  In their own files
// QMM_OUT is the f32 result; the *_ep.hip files define QMM_WITH_EPILOGUE and
// include the same kernels with an Epilogue (qmm_internal.h) in its place:
//   out[m][n] = act(sum + bias[n]) * mul[m][n] + residual[m][n]
// in f32, rounded once to out's type.  Every element is read and written by
// one thread, its operands before its result, so out may be mul or residual.
#pragma once

#include <hip/hip_runtime.h>

#include "qmm.h"
#include "qmm_internal.h"

namespace qmm {

// v / (1 + exp(-x)) for an x of v's sign, where t + rest = -|x| log2(e) / 2: within 7 steps of
// f32 relative (2^-20 is eight), by the hardware's 2^t and reciprocal (one step each).
// With e = 2^(t + rest) it is v / (1 + e^2) above 0 and v e^2 / (1 + e^2) below: e^2 never
// overflows, and below 0 it is multiplied in by halves, so that what underflows is the result
// alone.  (One exponential of -x overflows at -88.72, where silu is still 2.6e-37.)  t is
// rounded to f32; what that leaves out goes into rest, as it alone would be |x| steps of the
// result.  A GEMM's epilogue overlaps with nothing, so its instructions count: silu(product)
// * factor, 8192 tokens, 8192 x 4096 Q4_K 568 us (561 with that one exponential, 546 without
// an activation), 2048 tokens, 14336 x 4096 293 (290, 283).
__device__ __forceinline__ float times_sigmoid(float v, float t, float rest) {
  constexpr float kLn2 = 0.69314718055994531f;
  const float e = __builtin_amdgcn_exp2f(t) * fmaf(rest, kLn2, 1.0f);
  const float r = v * __builtin_amdgcn_rcpf(fmaf(e, e, 1.0f)), below = v < 0.f ? e : 1.0f;
  return r * below * below;  // a NaN in v stays one
}

__device__ __forceinline__ float silu(float v) {
  constexpr float kHi = -0.72134751081466674805f, kLo = -9.629815167500055e-9f;  // -log2(e) / 2
  const float y = fminf(fabsf(v), 250.f);  // past it e is 0
  const float t = y * kHi;
  return times_sigmoid(v, t, fmaf(y, kLo, fmaf(y, kHi, -t)));
}

// v (1 + tanh(u)) / 2 = v / (1 + exp(-2 u)), 2 u = 2 sqrt(2 / pi) (v + 0.044715 v^3).  In 64
// bits up to t: 2 u is a number of up to 88 where the result leaves f32's normal range, and
// each rounding of it to f32 would be up to 88 steps of the result (in all 12 times 2^-20 at
// -9; 8192 tokens as above 571 us, 563 in f32).
__device__ __forceinline__ float gelu_tanh(float v) {
  constexpr double kV = -1.1511040990721626, kV3 = kV * 0.044715;  // -log2(e) sqrt(2 / pi)
  const double y = (double)fminf(fabsf(v), 16.f);  // past it e is 0
  const double u = y * fma(kV3 * y, y, kV);
  const float t = (float)u;
  return times_sigmoid(v, t, (float)(u - (double)t));
}

// v erfc(-v / sqrt(2)) / 2 within 2^-20 relative (from -13.2 down, where it leaves f32's
// normal range, 2^-126 absolute).  With y = |v| and t = 1 / (1 + 0.33 y),
// erfc(y / sqrt(2)) exp(y^2 / 2) / t is a polynomial of degree 9 in t to 2e-8 on 0 <= y
// <= 14.5 (a least squares fit of the function's values with weights raised where
// the relative error was largest), where the exponential leaves f32's range; 3e-7 as it
// is evaluated, 6.5e-7 with 2^x and the reciprocal each a step off.  The square is
// taken in two parts, as its rounding alone would be y^2 / 2 steps of the result.
// gelu(product) * factor, 8192 tokens, 8192 x 4096 Q4_K 581 us (546 without an activation;
// erfcf took 6% longer), 2048 tokens, 14336 x 4096 299 (283); 499 tokens with a bias, 4096 x
// 4096 repacked Q8_0 33.4 (32.8).
__device__ __forceinline__ float gelu(float v) {
  constexpr float kC[10] = {-0.0219160002f, 0.0707042441f, -0.00149240822f, -0.226902843f, 0.213063121f,
                            0.00304379361f, 0.207221866f, 0.229145855f, 0.263853908f, 0.263278455f};
  constexpr float kHi = -0.7213475108146667f, kLo = -9.629815167500055e-9f, kLn2 = 0.69314718055994531f;  // -log2(e) / 2
  const float y = fminf(fabsf(v), 14.5f);  // a NaN is still one in v
  const float t = __builtin_amdgcn_rcpf(fmaf(0.33f, y, 1.0f));
  float q = kC[0];
#pragma unroll
  for (int i = 1; i < 10; ++i) q = fmaf(q, t, kC[i]);
  const float s = y * y, x = s * kHi;
  const float rest = fmaf(fmaf(y, y, -s), kHi, fmaf(s, kLo, fmaf(s, kHi, -x)));
  // (y comes in before the exponential, whose product with the rest alone is subnormal earlier.)
  const float tail = y * (0.5f * q * t) * (__builtin_amdgcn_exp2f(x) * fmaf(rest, kLn2, 1.0f));
  return v < 0.f ? -tail : v - tail;
}

// f32 activations.  Each is written so that its tail keeps its relative
// accuracy: gelu through erfc (1 + erf loses everything below -4), silu and gelu's tanh form
// through e^x below 0.
__device__ __forceinline__ float activated(int act, float v) {
  switch (act) {
    case QMM_ACT_RELU: return v < 0.f ? 0.f : v;  // a NaN stays one
    case QMM_ACT_SILU: return silu(v);
    case QMM_ACT_GELU: return gelu(v);
    case QMM_ACT_GELU_TANH: return gelu_tanh(v);
    default: return v;
  }
}

// An element's operands as they lie in memory: a kernel asks for them before its
// sums meet, so that they arrive meanwhile (eight tokens, residual in f32, 4096 x 4096
// Q4_K 8.6 -> 6.8 us, 14336 x 4096 15.8 -> 14.8).  For the plain result there are none.
struct Operands {
  float bias;
  uint32_t mul, residual;
};
struct NoOperands {};
__device__ __forceinline__ uint32_t bits_at(const void *p, int f16, int64_t i) {
  return f16 ? (uint32_t)static_cast<const uint16_t *>(p)[i] : static_cast<const uint32_t *>(p)[i];
}
__device__ __forceinline__ float value_of(uint32_t bits, int f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)bits) : __uint_as_float(bits);
}
__device__ __forceinline__ Operands operands(const Epilogue &e, int64_t m, int64_t n) {
  Operands o{};
  if (e.bias) o.bias = e.bias[n];
  if (e.mul) o.mul = bits_at(e.mul, e.mul_f16, m * e.mul_stride + n);
  if (e.residual) o.residual = bits_at(e.residual, e.residual_f16, m * e.residual_stride + n);
  return o;
}
__device__ __forceinline__ void put(const Epilogue &e, int64_t m, int64_t n, int64_t, float v, const Operands &o) {
  if (e.bias) v += o.bias;
  v = activated(e.act, v);
  if (e.mul) v *= value_of(o.mul, e.mul_f16);
  if (e.residual) v += value_of(o.residual, e.residual_f16);
  if (e.out_f16)
    static_cast<_Float16 *>(e.out)[m * e.out_stride + n] = (_Float16)v;
  else
    static_cast<float *>(e.out)[m * e.out_stride + n] = v;
}
__device__ __forceinline__ NoOperands operands(float *, int64_t, int64_t) { return {}; }
__device__ __forceinline__ void put(float *Y, int64_t m, int64_t n, int64_t N, float v, const NoOperands &) { Y[m * N + n] = v; }
template <typename Result>
__device__ __forceinline__ void put(const Result &e, int64_t m, int64_t n, int64_t N, float v) {
  put(e, m, n, N, v, operands(e, m, n));
}

#ifdef QMM_WITH_EPILOGUE
#define QMM_OUT const Epilogue
using Out = Epilogue;
#else
#define QMM_OUT float *__restrict__
using Out = float *;
#endif

}  // namespace qmm
