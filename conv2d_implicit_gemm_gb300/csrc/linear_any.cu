// Linear layer, any sizes and strides: fp32 products in 64 x 64 tiles.
#include "ptx.cuh"
#include "token.h"
#include "token_math.cuh"

namespace oidnx {
namespace {

constexpr int kT = 64, kK = 16;

template <typename T>
__global__ void __launch_bounds__(256) linear_any_kernel(const LinearParams p) {
  __shared__ float xs[kK][kT + 1], ws[kK][kT + 1];
  griddep_launch_dependents();
  griddep_wait();
  const int i0 = blockIdx.y * kT, j0 = blockIdx.x * kT;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const T* x = static_cast<const T*>(p.x);
  const T* w = static_cast<const T*>(p.w);
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += kK) {
    for (int e = threadIdx.x; e < kT * kK; e += 256) {
      const int r = e / kK, c = e % kK;
      xs[c][r] = i0 + r < p.m && k0 + c < p.k ? to_f32<T>(x[(i0 + r) * p.ldx + k0 + c]) : 0.f;
      ws[c][r] = j0 + r < p.n && k0 + c < p.k ? to_f32<T>(w[(j0 + r) * p.ldw + k0 + c]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kK; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[c][ty + 16 * i], ws[c][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int r = i0 + ty + 16 * i;
    if (r >= p.m) break;
    for (int j = 0; j < 4; ++j) {
      const int c = j0 + tx + 16 * j;
      if (c >= p.n) break;
      float z = acc[i][j];
      if (p.bias) z += to_f32<T>(static_cast<const T*>(p.bias)[c]);
      z = activate(z, p.act);
      if (p.residual) z += to_f32<T>(static_cast<const T*>(p.residual)[r * p.ldr + c]);
      static_cast<T*>(p.y)[r * p.ldy + c] = from_f32<T>(z);
    }
  }
}

}  // namespace

cudaError_t launch_linear_any(const LinearParams& p, int precision, cudaStream_t stream) {
  const dim3 grid((p.n + kT - 1) / kT, (p.m + kT - 1) / kT);
  return precision == OIDNX_PRECISION_BF16
             ? launch_pdl(linear_any_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, p)
             : launch_pdl(linear_any_kernel<__half>, grid, dim3(256), 0, stream, p);
}

}  // namespace oidnx
