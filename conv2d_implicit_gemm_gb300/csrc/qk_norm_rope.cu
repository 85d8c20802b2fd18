// Norm of each query and key head, rotation by the token's position and the
// append of keys and values to a cache, in one pass.
//
//   r = 1 / sqrt(mean(x^2) + eps);  y = x r w;
//   pairs (a, b) of the first rot values: (a c - b s, b c + a s)
//
// with c, s the table rows of the token's position.  Each value is read and
// written once, so the bound is memory; everything between is fp32.  16384 tokens
// x 48 heads x 128 in bf16: 90 us, 4.6 TB/s, 68% of the measured copy rate: with
// 78 registers 24 warps an SM do not quite cover the rotation's and the sums'
// latency (issue slots 49% busy).  One token: 2.2 us on the device.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "ptx.cuh"
#include "token.h"

namespace oidnx {
namespace {

constexpr int kAnyThreads = 256;
constexpr int kCtasPerSm = 2;
constexpr int kDepth = 4;           // tokens of a lane group in flight, at most,
constexpr int kRing = 48 * 1024;    // and within this much shared memory

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7FC00000); }

// 1 / sqrt(x) to fp32's last place or two: the hardware's 2^-22 and one Newton
// step.  Zero and infinity keep the hardware's answer (infinity and zero).
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  const float e = fmaf(-x * r, r, 1.f);
  return x > 0.f && x < INFINITY ? fmaf(0.5f * r, e, r) : r;
}

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

// P rotation pairs of one head: the first values and the second values of
// each (half-split), or the pairs one after the other (adjacent).
template <typename T, int P> struct Pairs {
  using Raw = typename std::conditional<sizeof(T) * P == 8, uint2, uint4>::type;  // P values
  Raw a, b;

  static __device__ __forceinline__ void values(Raw r, float (&f)[P]) {
    uint32_t w[sizeof(Raw) / 4];
    if constexpr (sizeof(Raw) == 8) w[0] = r.x, w[1] = r.y;
    else w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(Raw) / 4); ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        const float2 v = unpack2<T>(w[i]);
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
      }
    }
  }
  static __device__ __forceinline__ Raw raw(const float (&f)[P]) {
    uint32_t w[sizeof(Raw) / 4];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(Raw) / 4); ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    }
    if constexpr (sizeof(Raw) == 8) return make_uint2(w[0], w[1]);
    else return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // two pairs a packed register: x their first, y their second values
  template <bool IL> __device__ __forceinline__ void unpack(uint64_t (&x)[P / 2], uint64_t (&y)[P / 2]) const {
    float f[P], g[P];
    values(a, f);
    values(b, g);
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      if constexpr (IL) {
        const float* v = i < P / 4 ? f + 4 * i : g + 4 * (i - P / 4);
        x[i] = f2(v[0], v[2]), y[i] = f2(v[1], v[3]);
      } else {
        x[i] = f2(f[2 * i], f[2 * i + 1]), y[i] = f2(g[2 * i], g[2 * i + 1]);
      }
    }
  }
  template <bool IL> __device__ __forceinline__ void pack(const uint64_t (&x)[P / 2], const uint64_t (&y)[P / 2]) {
    float f[P], g[P];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float2 u = f2_of(x[i]), v = f2_of(y[i]);
      if constexpr (IL) {
        float* o = i < P / 4 ? f + 4 * i : g + 4 * (i - P / 4);
        o[0] = u.x, o[1] = v.x, o[2] = u.y, o[3] = v.y;
      } else {
        f[2 * i] = u.x, f[2 * i + 1] = u.y, g[2 * i] = v.x, g[2 * i + 1] = v.y;
      }
    }
    a = raw(f), b = raw(g);
  }
};

template <int N> __device__ __forceinline__ void async_copy(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// Heads in pieces of 2 P values, P rotation pairs a lane, so that a pair never
// leaves its lane: 2 P consecutive values where pairs are adjacent, else P of
// each half (of the rotated part, or of the rest, which does not turn).
//   P     8 (16-byte loads of 16-bit values), or 4
//   LPH   lanes a head: a power of two, or 0: d / 2P of them, packed into warps
//   NT    threads of a CTA, which takes as many tokens at a time as it holds
//         and strides over the tokens
template <typename T, int P, int LPH, int NT, bool IL>
__global__ void __launch_bounds__(NT, kCtasPerSm) qk_norm_rope_vec_kernel(const NormParams p) {
  using Raw = typename Pairs<T, P>::Raw;
  const int lanes = LPH ? LPH : p.d / (2 * P);
  const int per_warp = 32 / lanes;
  const int wl = threadIdx.x & 31;
  const int group_w = wl / lanes;        // group within the warp
  const int lane = wl - group_w * lanes;
  const bool spare = group_w >= per_warp;  // lanes that no whole group is left for
  const int groups = per_warp * (NT / 32);
  const int group = (threadIdx.x >> 5) * per_warp + group_w;
  const int hq = p.heads[0], hk = p.heads[1], total = hq + hk + p.heads[2];
  const int heads_y = (total + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);  // of this CTA row
  const int tokens = groups / heads_y;
  const int tl = group / heads_y;
  const int h = blockIdx.y * heads_y + group - tl * heads_y;
  griddep_launch_dependents();
  griddep_wait();

  // first and second values of this lane's pairs
  const int half = p.rot / 2, j = lane * P;
  const int ea = IL ? 2 * j : j < half ? j : j + half;
  const int eb = IL ? 2 * j + P : j < half ? j + half : j + half + (p.d - p.rot) / 2;
  // this group's head: 0 of the queries, 1 of the keys, 2 of the values, -1 none
  const int kind = spare || tl >= tokens || h >= total ? -1 : h < hq ? 0 : h < hq + hk ? 1 : 2;
  const int k = kind < 0 ? 0 : kind;
  const bool turns = j < half && (kind == 0 || kind == 1);
  const int hh = h - (k > 0 ? hq : 0) - (k > 1 ? hk : 0);
  const int tstep = gridDim.x * tokens;
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * tokens + tl;
  const T* src = static_cast<const T*>(p.in[k]) + hh * p.in_h[k] + token0 * p.in_t[k];  // the token to fetch next
  const int64_t src_step = tstep * p.in_t[k];
  T* const dst = static_cast<T*>(p.out[k]) + hh * p.out_h[k];
  const int64_t dst_row = p.out_t[k];
  const bool weighted = kind >= 0 && k < 2 && p.weight[k];
  Pairs<T, P> weight;
  weight.a = weight.b = Raw{};
  if (weighted) {
    weight.a = __ldg(reinterpret_cast<const Raw*>(static_cast<const T*>(p.weight[k]) + ea));
    weight.b = __ldg(reinterpret_cast<const Raw*>(static_cast<const T*>(p.weight[k]) + eb));
  }

  // The heads of the next kStages - 1 tokens are on their way to shared memory
  // (each thread's own values: no barrier); position and row are read one
  // token ahead, so that only the rotation's load waits for another.
  constexpr int kSlot = 2 * sizeof(Raw);
  constexpr int kStages = kRing / (NT * kSlot) < kDepth ? kRing / (NT * kSlot) : kDepth;
  static_assert(kStages >= 2, "one token ahead at least");
  __shared__ __align__(16) uint8_t ring[kStages][NT][kSlot];
  const auto fetch = [&](int64_t token, int stage) {
    if (kind >= 0 && token < p.t) {
      const uint32_t to = smem_u32(ring[stage][threadIdx.x]);
      async_copy<sizeof(Raw)>(to, src + ea);
      async_copy<sizeof(Raw)>(to + sizeof(Raw), src + eb);
    }
    src += src_step;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int pos_n = 0, row_n = 0;
  const auto where = [&](int64_t token) {
    if (token >= p.t) return;
    row_n = p.slots ? p.slots[token] : static_cast<int>(token);  // of the keys and values
    if (p.rot) pos_n = p.positions[token];
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(token0 + static_cast<int64_t>(s) * tstep, s);
  where(token0);
  const float inv_d = 1.f / static_cast<float>(p.d);
  int stage = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * tokens; base < p.t; base += tstep) {
    const int64_t token = base + tl;
    const int pos = pos_n, row = row_n;
    float4 c[P / 4], s[P / 4];
    if (turns) {
      const bool known = pos >= 0 && pos < p.table_rows;
      const int64_t o = static_cast<int64_t>(pos) * half + j;
#pragma unroll
      for (int i = 0; i < P / 4; ++i) {
        if (known) {
          c[i] = __ldg(reinterpret_cast<const float4*>(p.cos_t + o) + i);
          s[i] = __ldg(reinterpret_cast<const float4*>(p.sin_t + o) + i);
        } else {
          c[i] = s[i] = make_float4(quiet_nan(), quiet_nan(), quiet_nan(), quiet_nan());
        }
      }
    }
    where(token + tstep);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    Pairs<T, P> x;
    {
      const Raw* at = reinterpret_cast<const Raw*>(ring[stage][threadIdx.x]);
      x.a = at[0], x.b = at[1];
    }
    fetch(token + static_cast<int64_t>(kStages - 1) * tstep, stage == 0 ? kStages - 1 : stage - 1);
    if (++stage == kStages) stage = 0;
    uint64_t a[P / 2], b[P / 2];
    x.template unpack<IL>(a, b);
    uint64_t sq[2] = {mul2(a[0], a[0]), mul2(b[0], b[0])};
#pragma unroll
    for (int i = 1; i < P / 2; ++i) sq[0] = fma2(a[i], a[i], sq[0]), sq[1] = fma2(b[i], b[i], sq[1]);
    const float2 s0 = f2_of(sq[0]), s1 = f2_of(sq[1]);
    float sum = (s0.x + s0.y) + (s1.x + s1.y);
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
    const bool kept = row >= 0 && row < p.cache_rows;
    if (kind < 0 || token >= p.t || (kind > 0 && !kept)) continue;
    if (kind < 2) {
      const float r = inverse_root(fmaf(sum, inv_d, p.eps));
      const uint64_t r2 = f2(r, r);
#pragma unroll
      for (int i = 0; i < P / 2; ++i) a[i] = mul2(a[i], r2), b[i] = mul2(b[i], r2);
      if (weighted) {
        uint64_t wa[P / 2], wb[P / 2];
        weight.template unpack<IL>(wa, wb);
#pragma unroll
        for (int i = 0; i < P / 2; ++i) a[i] = mul2(a[i], wa[i]), b[i] = mul2(b[i], wb[i]);
      }
      if (j < half) {
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          const float4 cc = c[i / 2], ss = s[i / 2];
          const uint64_t cs = i % 2 ? f2(cc.z, cc.w) : f2(cc.x, cc.y), sn = i % 2 ? f2(ss.z, ss.w) : f2(ss.x, ss.y);
          const uint64_t as = mul2(a[i], sn), bs = mul2(b[i], sn ^ 0x8000000080000000ull);
          a[i] = fma2(a[i], cs, bs), b[i] = fma2(b[i], cs, as);
        }
      }
      x.template pack<IL>(a, b);
    }
    T* to = dst + (kind ? row : static_cast<int>(token)) * dst_row;
    *reinterpret_cast<Raw*>(to + ea) = x.a;
    *reinterpret_cast<Raw*>(to + eb) = x.b;
  }
}

// Any alignment, stride or even head size: one warp per head, single values.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads) qk_norm_rope_any_kernel(const NormParams p) {
  const int lane = threadIdx.x & 31;
  const int hq = p.heads[0], hk = p.heads[1], total = hq + hk + p.heads[2];
  const int token = blockIdx.x;
  const int h = blockIdx.y * (kAnyThreads / 32) + (threadIdx.x >> 5);
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

template <typename T, int P, int LPH, int NT>
cudaError_t launch_vec(const NormParams& p, int gy, int device, int sms, cudaStream_t stream) {
  const int total = p.heads[0] + p.heads[1] + p.heads[2];
  const int tokens = NT / 32 * (32 / (LPH ? LPH : p.d / (2 * P))) / ((total + gy - 1) / gy);
  const int most = (kCtasPerSm * sms + gy - 1) / gy;  // resident together
  const dim3 grid(std::min((p.t + tokens - 1) / tokens, most), gy);
  static Kernel adjacent, halves;
  return p.interleaved
             ? adjacent.launch(qk_norm_rope_vec_kernel<T, P, LPH, NT, true>, device, grid, NT, 0, 1, stream, p)
             : halves.launch(qk_norm_rope_vec_kernel<T, P, LPH, NT, false>, device, grid, NT, 0, 1, stream, p);
}

// 8 or 12 warps, whichever leaves fewer lane groups without a head; a token
// with more heads is split over CTA rows.
template <typename T, int P, int LPH>
cudaError_t launch_heads(const NormParams& p, int device, int sms, cudaStream_t stream) {
  const int total = p.heads[0] + p.heads[1] + p.heads[2], per_warp = 32 / (LPH ? LPH : p.d / (2 * P));
  const auto busy = [&](int warps, int* gy) {
    const int groups = warps * per_warp;
    *gy = (total + groups - 1) / groups;
    const int heads = (total + *gy - 1) / *gy;
    return static_cast<float>(groups / heads * heads) / groups;
  };
  int gy8, gy12;
  const float b8 = busy(8, &gy8), b12 = busy(12, &gy12);
  return b12 > b8 ? launch_vec<T, P, LPH, 384>(p, gy12, device, sms, stream) : launch_vec<T, P, LPH, 256>(p, gy8, device, sms, stream);
}

template <typename T>
cudaError_t launch_vec_t(const NormParams& p, int device, int sms, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (p.wide && p.d == 64) return launch_heads<T, 8, 4>(p, device, sms, stream);
    if (p.wide && p.d == 128) return launch_heads<T, 8, 8>(p, device, sms, stream);
    if (p.wide) return launch_heads<T, 8, 0>(p, device, sms, stream);
  } else {
    if (p.d == 64) return launch_heads<T, 4, 8>(p, device, sms, stream);
    if (p.d == 128) return launch_heads<T, 4, 16>(p, device, sms, stream);
  }
  return launch_heads<T, 4, 0>(p, device, sms, stream);
}

template <typename T>
cudaError_t launch_any_t(const NormParams& p, int device, cudaStream_t stream) {
  const int total = p.heads[0] + p.heads[1] + p.heads[2], per = kAnyThreads / 32;
  static Kernel handle;
  return handle.launch(qk_norm_rope_any_kernel<T>, device, dim3(p.t, (total + per - 1) / per), kAnyThreads, 0, 1, stream, p);
}

}  // namespace

cudaError_t launch_norm_vec(const NormParams& p, int precision, int device, int sms, cudaStream_t stream) {
  if (precision == OIDNX_PRECISION_FP32) return launch_vec_t<float>(p, device, sms, stream);
  if (precision == OIDNX_PRECISION_BF16) return launch_vec_t<__nv_bfloat16>(p, device, sms, stream);
  return launch_vec_t<__half>(p, device, sms, stream);
}

cudaError_t launch_norm_any(const NormParams& p, int precision, int device, cudaStream_t stream) {
  if (precision == OIDNX_PRECISION_FP32) return launch_any_t<float>(p, device, stream);
  if (precision == OIDNX_PRECISION_BF16) return launch_any_t<__nv_bfloat16>(p, device, stream);
  return launch_any_t<__half>(p, device, stream);
}

}  // namespace oidnx
