// Window attention, any head size, stride and alignment: one warp per query
// and head.  Used where the tensor-core forms cannot load the operands in
// 16-byte pieces, the head exceeds 128 values or the scale is not positive.
#include "attn_row.cuh"

namespace oidnx {
namespace {

constexpr int kWarps = 4;

// NR: head values per lane (d <= 32 NR).
template <typename T, int NR>
__global__ void __launch_bounds__(kWarps * 32) attn_any_kernel(const AttnParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(p.b) * p.hq * p.tq) return;
  const int h = static_cast<int>(item % p.hq);
  const int i = static_cast<int>(item / p.hq % p.tq);
  const int b = static_cast<int>(item / p.hq / p.tq);
  attend_row<T, NR>(p, b, i, h, lane);
}

template <typename T, int NR>
cudaError_t launch(const AttnParams& p, int device, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.b) * p.hq * p.tq;
  static Kernel handle;
  return handle.launch(attn_any_kernel<T, NR>, device, dim3(static_cast<unsigned>((items + kWarps - 1) / kWarps)),
                       kWarps * 32, 0, 1, stream, p);
}

template <typename T>
cudaError_t launch_t(const AttnParams& p, int device, cudaStream_t stream) {
  if (p.d <= 64) return launch<T, 2>(p, device, stream);
  if (p.d <= 128) return launch<T, 4>(p, device, stream);
  return launch<T, 8>(p, device, stream);
}

}  // namespace

cudaError_t launch_attn_any(const AttnParams& p, int precision, int device, cudaStream_t stream) {
  return precision == OIDNX_PRECISION_BF16 ? launch_t<__nv_bfloat16>(p, device, stream) : launch_t<__half>(p, device, stream);
}

}  // namespace oidnx
