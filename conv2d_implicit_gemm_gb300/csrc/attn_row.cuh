// One query head's attention by one warp, in fp32, for any head size, stride
// and alignment: one pass over the visible keys with the running maximum and
// sum of the softmax.  The plain form of the operator, and what the
// tensor-core form falls back on for tiles whose values are no numbers.
#pragma once

#include "token_ptx.cuh"
#include "token.h"

namespace oidnx {

// NR: head values per lane (d <= 32 NR).
template <typename T, int NR>
__device__ __forceinline__ void attend_row(const AttnParams& p, int b, int i, int h, int lane) {
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

}  // namespace oidnx
