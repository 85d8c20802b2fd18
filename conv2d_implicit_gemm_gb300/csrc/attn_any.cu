// Window attention, any head size, stride and alignment: one warp per query
// and head, fp32 throughout, one pass over the visible keys with the running
// maximum and sum of the softmax.  Used where the tensor-core forms cannot
// load the operands in 16-byte pieces or the head exceeds 128 values.
#include "ptx.cuh"
#include "token.h"

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
  const int kvh = h / (p.hq / p.hk);
  const int n = attn_kv_len(p, b), nq = attn_q_len(p, b);
  const int pos = i < nq ? n - nq + i : -1;

  float q[NR], o[NR];
  const T* qp = static_cast<const T*>(p.q) + b * p.q_s[0] + i * p.q_s[1] + h * p.q_s[2];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int c = lane + 32 * r;
    q[r] = c < p.d && pos >= 0 ? to_f32<T>(qp[c]) : 0.f;
    o[r] = 0.f;
  }
  const T* kb = static_cast<const T*>(p.k) + b * p.k_s[0] + kvh * p.k_s[2];
  const T* vb = static_cast<const T*>(p.v) + b * p.v_s[0] + kvh * p.v_s[2];
  const int sink_end = min(min(p.held_sinks, n), pos + 1);
  const int ring = attn_ring_begin(p, n);
  const int begin = p.window > 0 ? max(ring, pos - p.window + 1) : ring;
  float top = -INFINITY, sum = 0.f;
  for (int part = 0; part < 2; ++part) {
    const int lo = part == 0 ? 0 : begin, hi = part == 0 ? sink_end : pos + 1;
    for (int j = lo; j < hi; ++j) {
      const int64_t slot = attn_slot(p, j);
      const T* kp = kb + slot * p.k_s[1];
      const T* vp = vb + slot * p.v_s[1];
      float dot = 0.f;
#pragma unroll
      for (int r = 0; r < NR; ++r)
        if (lane + 32 * r < p.d) dot = fmaf(q[r], to_f32<T>(kp[lane + 32 * r]), dot);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, s);
      dot *= p.scale;
      const float up = fmaxf(top, dot);
      const float base = up == -INFINITY ? 0.f : up;
      const float old = expf(top - base), e = expf(dot - base);
      top = up;
      sum = fmaf(sum, old, e);
#pragma unroll
      for (int r = 0; r < NR; ++r)
        if (lane + 32 * r < p.d) o[r] = fmaf(o[r], old, e * to_f32<T>(vp[lane + 32 * r]));
    }
  }
  T* op = static_cast<T*>(p.o) + b * p.o_s[0] + i * p.o_s[1] + h * p.o_s[2];
  // an empty row gives zeros; a NaN sum stays one
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int r = 0; r < NR; ++r)
    if (lane + 32 * r < p.d) op[lane + 32 * r] = from_f32<T>(o[r] * inv);
  if (p.lse && lane == 0)
    p.lse[(static_cast<int64_t>(b) * p.hq + h) * p.tq + i] = sum == 0.f ? -INFINITY : top + logf(sum);
}

template <typename T>
cudaError_t launch_t(const AttnParams& p, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.b) * p.hq * p.tq;
  const dim3 grid(static_cast<unsigned>((items + kWarps - 1) / kWarps)), block(kWarps * 32);
  if (p.d <= 64) return launch_pdl(attn_any_kernel<T, 2>, grid, block, 0, stream, p);
  if (p.d <= 128) return launch_pdl(attn_any_kernel<T, 4>, grid, block, 0, stream, p);
  return launch_pdl(attn_any_kernel<T, 8>, grid, block, 0, stream, p);
}

}  // namespace

cudaError_t launch_attn_any(const AttnParams& p, int precision, cudaStream_t stream) {
  return precision == OIDNX_PRECISION_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<__half>(p, stream);
}

}  // namespace oidnx
