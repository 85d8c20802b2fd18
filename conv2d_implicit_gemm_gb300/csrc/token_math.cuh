// Activations of the linear layer's epilogue, in fp32.
#pragma once

#include "../../include/oidnx.h"

namespace oidnx {

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case OIDNX_ACT_RELU: return z < 0.f ? 0.f : z;  // a NaN stays one
    case OIDNX_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case OIDNX_ACT_GELU_TANH: {
      const float u = 0.79788456080286536f * fmaf(0.044715f * z, z * z, z);
      return 0.5f * z * (1.f + tanhf(u));
    }
    case OIDNX_ACT_SILU: return z / (1.f + expf(-z));
    default: return z;
  }
}

}  // namespace oidnx
