// Copies of heads [sequence][token][head][value] of any strides and alignment to
// heads of whole 16-byte pieces, or back: for operands that the tensor-core forms
// cannot load as they lie.  Values past the source's are zeros.  Bound by its
// requests, two bytes a lane: a slow way in for calls that are rare.
#include <algorithm>

#include "cross.h"
#include "token_ptx.cuh"

namespace oidnx {
namespace {

constexpr int kThreads = 256;
constexpr int kMostCopies = 3;
struct Copies {
  HeadsCopy c[kMostCopies];
};

// A warp a head: 32 consecutive values a step.
__global__ void __launch_bounds__(kThreads) heads_copy_kernel(const __grid_constant__ Copies all) {
  griddep_launch_dependents();
  griddep_wait();
  const HeadsCopy& p = all.c[blockIdx.y];
  const int lane = threadIdx.x & 31;
  const int64_t heads = static_cast<int64_t>(p.n[0]) * p.n[1] * p.n[2];
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const uint16_t sign = p.negate ? 0x8000u : 0u;
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); at < heads; at += step) {
    const int h = static_cast<int>(at % p.n[2]), i = static_cast<int>(at / p.n[2] % p.n[1]);
    const int b = static_cast<int>(at / p.n[2] / p.n[1]);
    const uint16_t* from = static_cast<const uint16_t*>(p.from) + b * p.from_s[0] + i * p.from_s[1] + h * p.from_s[2];
    uint16_t* to = static_cast<uint16_t*>(p.to) + b * p.to_s[0] + i * p.to_s[1] + h * p.to_s[2];
#pragma unroll 8
    for (int c = lane; c < p.d_to; c += 32) to[c] = c < p.d ? static_cast<uint16_t>(from[c] ^ sign) : uint16_t(0);
  }
}

}  // namespace

cudaError_t launch_heads_copy(const HeadsCopy* copies, int count, int device, int sms, cudaStream_t stream) {
  Copies all = {};
  int64_t most = 0;
  for (int i = 0; i < count; ++i) {
    all.c[i] = copies[i];
    most = std::max(most, static_cast<int64_t>(copies[i].n[0]) * copies[i].n[1] * copies[i].n[2]);
  }
  const int64_t ctas = std::min((most + kThreads / 32 - 1) / (kThreads / 32), static_cast<int64_t>(sms) * 8);
  static Kernel handle;
  return handle.launch(heads_copy_kernel, device, dim3(static_cast<unsigned>(std::max<int64_t>(ctas, 1)), count), kThreads, 0, 1,
                       stream, all);
}

}  // namespace oidnx
