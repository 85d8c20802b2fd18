// Norm of each query and key head, rotation by the token's position and the
// append of keys and values to a cache, in one pass.
//
//   r = 1 / sqrt(mean(x^2) + eps);  y = x r w;
//   pairs (a, b) of the first rot values: (a c - b s, b c + a s)
//
// with c, s the table rows of the token's position.  Each value is read and
// written once, so the bound is memory; everything between is fp32.
#include <type_traits>

#include "ptx.cuh"
#include "token.h"

namespace oidnx {
namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7FC00000); }

// Pairs of fp32 values, two operations an instruction.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_of(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Four pairs of one head: the first values and the second values of each.
template <typename T> struct Pairs {
  using Raw = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;  // four values
  Raw a, b;
  // first: pairs (a_i, b_i) as two packed registers each
  __device__ __forceinline__ void unpack(bool interleaved, uint64_t (&x)[2], uint64_t (&y)[2]) const {
    float f[4], g[4];
    if constexpr (sizeof(T) == 4) {
      f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
      g[0] = __uint_as_float(b.x), g[1] = __uint_as_float(b.y), g[2] = __uint_as_float(b.z), g[3] = __uint_as_float(b.w);
    } else {
      const float2 p = unpack2<T>(a.x), q = unpack2<T>(a.y), r = unpack2<T>(b.x), s = unpack2<T>(b.y);
      f[0] = p.x, f[1] = p.y, f[2] = q.x, f[3] = q.y;
      g[0] = r.x, g[1] = r.y, g[2] = s.x, g[3] = s.y;
    }
    if (interleaved) {  // (f0 f1) (f2 f3) (g0 g1) (g2 g3)
      x[0] = f2(f[0], f[2]), x[1] = f2(g[0], g[2]);
      y[0] = f2(f[1], f[3]), y[1] = f2(g[1], g[3]);
    } else {
      x[0] = f2(f[0], f[1]), x[1] = f2(f[2], f[3]);
      y[0] = f2(g[0], g[1]), y[1] = f2(g[2], g[3]);
    }
  }
  __device__ __forceinline__ void pack(bool interleaved, const uint64_t (&x)[2], const uint64_t (&y)[2]) {
    const float2 p = f2_of(x[0]), q = f2_of(x[1]), r = f2_of(y[0]), s = f2_of(y[1]);
    float f[4], g[4];
    if (interleaved) {
      f[0] = p.x, f[1] = r.x, f[2] = p.y, f[3] = r.y;
      g[0] = q.x, g[1] = s.x, g[2] = q.y, g[3] = s.y;
    } else {
      f[0] = p.x, f[1] = p.y, f[2] = q.x, f[3] = q.y;
      g[0] = r.x, g[1] = r.y, g[2] = s.x, g[3] = s.y;
    }
    if constexpr (sizeof(T) == 4) {
      a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      b = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
    } else {
      a = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
      b = make_uint2(pack2<T>(g[0], g[1]), pack2<T>(g[2], g[3]));
    }
  }
};

// Heads in pieces of eight values, four rotation pairs a lane, so that a pair
// never leaves its lane: 8 consecutive values where pairs are adjacent, else 4
// of each half (of the rotated part, or of the rest, which turns by nothing).
//   LPH   lanes a head: 4, 8, 16, 32, or 0: p.d / 8 of them, packed into warps
//   U     heads of one token that a lane group has in flight together; the
//         rotation's values stay in registers for them
// A CTA takes as many tokens as its lane groups hold.
template <typename T, int LPH, int U, bool IL>
__global__ void __launch_bounds__(kNormThreads, sizeof(T) == 4 ? 3 : 4) qk_norm_rope_vec_kernel(const NormParams p) {
  using Raw = typename Pairs<T>::Raw;
  const int lanes = LPH ? LPH : p.d / 8;
  const int per_warp = LPH ? 32 / (LPH ? LPH : 1) : 32 / lanes;
  const int wl = threadIdx.x & 31;
  const int group_w = wl / lanes;        // group within the warp
  const int lane = wl - group_w * lanes;
  const bool spare = group_w >= per_warp;  // lanes that no whole group is left for
  const int groups = per_warp * (kNormThreads / 32);
  const int group = (threadIdx.x >> 5) * per_warp + group_w;
  const int hq = p.heads[0], hk = p.heads[1], total = hq + hk + p.heads[2];
  const int heads_y = (total + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);  // of this CTA row
  const int first_head = blockIdx.y * heads_y, end_head = min(total, first_head + heads_y);
  const int gt = (heads_y + U - 1) / U;  // groups a token
  const int tokens = groups / gt;
  const int tl = group / gt, slot_h = group - tl * gt;
  const int token = blockIdx.x * tokens + tl;
  const bool idle = spare || tl >= tokens || token >= p.t;
  griddep_launch_dependents();
  griddep_wait();

  // first and second values of this lane's pairs
  const int half = p.rot / 2, j = lane * 4;
  const int ea = IL ? lane * 8 : j < half ? j : j + half;
  const int eb = IL ? lane * 8 + 4 : j < half ? j + half : j + half + (p.d - p.rot) / 2;
  const bool turns = j < half;
  const bool mine = lane * 8 < p.d;  // lanes past the head's end (LPH > d / 8)

  Pairs<T> x[U];
  int kind[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = first_head + slot_h + u * gt;
    kind[u] = idle || !mine || h >= end_head ? -1 : h < hq ? 0 : h < hq + hk ? 1 : 2;
    x[u].a = x[u].b = Raw{};
    if (kind[u] < 0) continue;
    const int hh = h - (kind[u] > 0 ? hq : 0) - (kind[u] > 1 ? hk : 0);
    const T* src = static_cast<const T*>(p.in[kind[u]]) + token * p.in_t[kind[u]] + hh * p.in_h[kind[u]];
    x[u].a = *reinterpret_cast<const Raw*>(src + ea);
    x[u].b = *reinterpret_cast<const Raw*>(src + eb);
  }
  const int at = idle ? 0 : token;
  const int64_t row = p.slots ? p.slots[at] : at;  // of the keys and values
  const bool kept = row >= 0 && row < p.cache_rows;
  uint64_t cs[2] = {0, 0}, sn[2] = {0, 0};
  if (turns && mine) {
    const int pos = p.positions[at];
    if (pos >= 0 && pos < p.table_rows) {
      const int64_t o = static_cast<int64_t>(pos) * half + j;
      const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos_t + o));
      const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin_t + o));
      cs[0] = f2(c.x, c.y), cs[1] = f2(c.z, c.w), sn[0] = f2(s.x, s.y), sn[1] = f2(s.z, s.w);
    } else {
      cs[0] = cs[1] = sn[0] = sn[1] = f2(quiet_nan(), quiet_nan());
    }
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint64_t a[2], b[2];
    x[u].unpack(IL, a, b);
    uint64_t sq = mul2(a[0], a[0]);
    sq = fma2(a[1], a[1], sq), sq = fma2(b[0], b[0], sq), sq = fma2(b[1], b[1], sq);
    const float2 s2 = f2_of(sq);
    float sum = s2.x + s2.y;
    if constexpr (LPH != 0) {
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float up = __shfl_down_sync(0xFFFFFFFFu, sum, o);
        if (lane + o < lanes) sum += up;
      }
      sum = __shfl_sync(0xFFFFFFFFu, sum, wl - lane);
    }
    if (kind[u] < 0 || (kind[u] > 0 && !kept)) continue;
    const int h = first_head + slot_h + u * gt;
    const int hh = h - (kind[u] > 0 ? hq : 0) - (kind[u] > 1 ? hk : 0);
    T* dst = static_cast<T*>(p.out[kind[u]]) + (kind[u] ? row : token) * p.out_t[kind[u]] + hh * p.out_h[kind[u]];
    if (kind[u] < 2) {
      const float r = 1.0f / sqrtf(sum / static_cast<float>(p.d) + p.eps);
      const uint64_t r2 = f2(r, r);
      const T* weight = static_cast<const T*>(p.weight[kind[u]]);
      uint64_t wa[2] = {r2, r2}, wb[2] = {r2, r2};
      if (weight) {
        Pairs<T> w;
        w.a = __ldg(reinterpret_cast<const Raw*>(weight + ea));
        w.b = __ldg(reinterpret_cast<const Raw*>(weight + eb));
        w.unpack(IL, wa, wb);
#pragma unroll
        for (int i = 0; i < 2; ++i) wa[i] = mul2(wa[i], r2), wb[i] = mul2(wb[i], r2);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = mul2(a[i], wa[i]), b[i] = mul2(b[i], wb[i]);
        if (!turns) continue;
        const uint64_t as = mul2(a[i], sn[i]), bs = mul2(b[i], sn[i] ^ 0x8000000080000000ull);
        a[i] = fma2(a[i], cs[i], bs), b[i] = fma2(b[i], cs[i], as);
      }
      x[u].pack(IL, a, b);
    }
    *reinterpret_cast<Raw*>(dst + ea) = x[u].a;
    *reinterpret_cast<Raw*>(dst + eb) = x[u].b;
  }
}

// Any alignment, stride or even head size: one warp per head, single values.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_any_kernel(const NormParams p) {
  const int lane = threadIdx.x & 31;
  const int hq = p.heads[0], hk = p.heads[1], total = hq + hk + p.heads[2];
  const int token = blockIdx.x;
  const int h = blockIdx.y * (kNormThreads / 32) + (threadIdx.x >> 5);
  griddep_launch_dependents();
  griddep_wait();
  if (h >= total) return;
  const int kind = h < hq ? 0 : h < hq + hk ? 1 : 2;
  const int hh = kind == 0 ? h : kind == 1 ? h - hq : h - hq - hk;
  const int64_t slot = kind && p.slots ? p.slots[token] : token;
  if (kind && (slot < 0 || slot >= p.cache_rows)) return;
  const T* src = static_cast<const T*>(p.in[kind]) + token * p.in_t[kind] + hh * p.in_h[kind];
  T* dst = static_cast<T*>(p.out[kind]) + slot * p.out_t[kind] + hh * p.out_h[kind];
  if (kind == 2) {
    for (int i = lane; i < p.d; i += 32) dst[i] = src[i];
    return;
  }
  const int pos = p.rot ? p.positions[token] : 0;
  const bool known = pos >= 0 && pos < p.table_rows;
  float sum = 0.f;
  for (int i = lane; i < p.d; i += 32) {
    const float v = to_f32<T>(src[i]);
    sum = fmaf(v, v, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const float r = 1.0f / sqrtf(sum / static_cast<float>(p.d) + p.eps);
  const T* weight = static_cast<const T*>(p.weight[kind]);
  const int half = p.rot / 2;
  // the lane that reads a pair also writes it, so the output may be the input
  for (int i = lane; i < half; i += 32) {
    const int ia = p.interleaved ? 2 * i : i, ib = p.interleaved ? 2 * i + 1 : i + half;
    const float a = to_f32<T>(src[ia]) * r * (weight ? to_f32<T>(weight[ia]) : 1.f);
    const float b = to_f32<T>(src[ib]) * r * (weight ? to_f32<T>(weight[ib]) : 1.f);
    const int64_t at = static_cast<int64_t>(pos) * half + i;
    const float c = known ? p.cos_t[at] : quiet_nan(), s = known ? p.sin_t[at] : quiet_nan();
    dst[ia] = from_f32<T>(fmaf(a, c, -b * s));
    dst[ib] = from_f32<T>(fmaf(b, c, a * s));
  }
  for (int i = p.rot + lane; i < p.d; i += 32)
    dst[i] = from_f32<T>(to_f32<T>(src[i]) * r * (weight ? to_f32<T>(weight[i]) : 1.f));
}

template <typename T, int LPH, int U>
cudaError_t launch_vec(const NormParams& p, int gy, cudaStream_t stream) {
  const int total = p.heads[0] + p.heads[1] + p.heads[2];
  const int groups = kNormThreads / 32 * (32 / (LPH ? LPH : p.d / 8));
  const int heads_y = (total + gy - 1) / gy, gt = (heads_y + U - 1) / U, tokens = groups / gt;
  const dim3 grid((p.t + tokens - 1) / tokens, gy);
  return p.interleaved ? launch_pdl(qk_norm_rope_vec_kernel<T, LPH, U, true>, grid, dim3(kNormThreads), 0, stream, p)
                       : launch_pdl(qk_norm_rope_vec_kernel<T, LPH, U, false>, grid, dim3(kNormThreads), 0, stream, p);
}

template <typename T, int LPH>
cudaError_t launch_heads(const NormParams& p, cudaStream_t stream) {
  const int total = p.heads[0] + p.heads[1] + p.heads[2];
  const int groups = kNormThreads / 32 * (32 / (LPH ? LPH : p.d / 8));
  // the heads of a token over as few CTAs as hold them at three a group
  const int gy = (total + 3 * groups - 1) / (3 * groups);
  const int u = ((total + gy - 1) / gy + groups - 1) / groups;
  if (u <= 1) return launch_vec<T, LPH, 1>(p, gy, stream);
  if (u == 2) return launch_vec<T, LPH, 2>(p, gy, stream);
  return launch_vec<T, LPH, 3>(p, gy, stream);
}

template <typename T>
cudaError_t launch_vec_t(const NormParams& p, cudaStream_t stream) {
  switch (p.d / 8) {
    case 4: return launch_heads<T, 4>(p, stream);
    case 8: return launch_heads<T, 8>(p, stream);
    case 16: return launch_heads<T, 16>(p, stream);
    case 32: return launch_heads<T, 32>(p, stream);
    default: return launch_heads<T, 0>(p, stream);
  }
}

template <typename T>
cudaError_t launch_any_t(const NormParams& p, cudaStream_t stream) {
  const int total = p.heads[0] + p.heads[1] + p.heads[2], per = kNormThreads / 32;
  return launch_pdl(qk_norm_rope_any_kernel<T>, dim3(p.t, (total + per - 1) / per), dim3(kNormThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_norm_vec(const NormParams& p, int precision, cudaStream_t stream) {
  if (precision == OIDNX_PRECISION_FP32) return launch_vec_t<float>(p, stream);
  if (precision == OIDNX_PRECISION_BF16) return launch_vec_t<__nv_bfloat16>(p, stream);
  return launch_vec_t<__half>(p, stream);
}

cudaError_t launch_norm_any(const NormParams& p, int precision, cudaStream_t stream) {
  if (precision == OIDNX_PRECISION_FP32) return launch_any_t<float>(p, stream);
  if (precision == OIDNX_PRECISION_BF16) return launch_any_t<__nv_bfloat16>(p, stream);
  return launch_any_t<__half>(p, stream);
}

}  // namespace oidnx
