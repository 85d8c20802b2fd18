// Activations of the linear layer's epilogue, in fp32.
#pragma once

#include "../../include/oidnx.h"

namespace oidnx {

// 1 / (1 + e^-z): the hardware's exp2 and reciprocal are good to about 2^-22,
// far below the 16-bit rounding that follows.  e^-z overflows to infinity
// for z < -88, which gives the limit 0.
__device__ __forceinline__ float sigmoid_fast(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// z Phi(z), with erfc of the positive argument from Abramowitz and Stegun
// 7.1.26 (a polynomial in 1 / (1 + p x) times e^-x^2, off by at most 1.5e-7):
// a third of the instructions of erff, which made the epilogue of a 128 x 128
// tile 3.4 us long.
__device__ __forceinline__ float gelu(float z) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float half_erfc = 0.5f * (q * t) * __expf(-x * x);
  // (from z = 14 on half_erfc is zero; the bound keeps infinity out of its product)
  return z < 0.f ? z * half_erfc : fmaf(-fminf(z, 16.f), half_erfc, z);
}

template <int ACT> __device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == OIDNX_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays one
  if constexpr (ACT == OIDNX_ACT_GELU) return gelu(z);
  // 0.5 z (1 + tanh u) = z / (1 + e^-2u)
  if constexpr (ACT == OIDNX_ACT_GELU_TANH)
    return z * sigmoid_fast(1.5957691216057308f * fmaf(0.044715f * z, z * z, z));
  if constexpr (ACT == OIDNX_ACT_SILU) return z * sigmoid_fast(z);
  return z;
}

template <int N> __device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  switch (act) {
    case OIDNX_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate<OIDNX_ACT_RELU>(v[i]);
      break;
    case OIDNX_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate<OIDNX_ACT_GELU>(v[i]);
      break;
    case OIDNX_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate<OIDNX_ACT_GELU_TANH>(v[i]);
      break;
    case OIDNX_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate<OIDNX_ACT_SILU>(v[i]);
      break;
    default: break;
  }
}

}  // namespace oidnx
