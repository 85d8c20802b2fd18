// Norm of each query and key head, rotation by the token's position and the
// append of keys and values to a cache, in one pass.
//
//   r = 1 / sqrt(mean(x^2) + eps);  y = x r w;
//   pairs (a, b) of the first rot values: (a c - b s, b c + a s)
//
// with c, s the table rows of the token's position.  Each value is read and
// written once, so the bound is memory; everything between is fp32.  16384 tokens
// x 48 heads x 128 in bf16: 76 us, 5.4 TB/s, 80% of the measured copy rate (a copy
// of the same bytes takes 65 us; without the arithmetic this kernel takes 70).  One
// warp keeps a token's rotation in registers for all its heads: read again for
// every head, and with one head a lane group of a persistent CTA, it took 90 us.
// One token: 1.9 us on the device.  8192 tokens in fp32: 65 us, 6.3 TB/s, 93% (bf16 42,
// where each byte costs twice the arithmetic).
#include <algorithm>
#include <type_traits>

#include "token_ptx.cuh"
#include "token.h"

namespace oidnx {
namespace {

constexpr int kAnyThreads = 256;
constexpr int kVecThreads = 128;
constexpr int kCtasPerSm = 6;  // 80 registers a thread; at 5 and 7 (spills) 81 and 77 us where 6 take 76

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

// Heads in pieces of 2 P values, P rotation pairs a lane, so that a pair never
// leaves its lane: 2 P consecutive values where pairs are adjacent, else P of
// each half (of the rotated part, or of the rest, which does not turn).
//   P     8 (16-byte loads of 16-bit values), or 4
//   LPH   lanes a head: a power of two, or 0: d / 2P of them, packed into warps
// A warp takes one token's position, row and rotation once, then `steps` times
// as many heads as it has lanes for, the next ones on their way meanwhile.
template <typename T, int P, int LPH, bool IL>
__global__ void __launch_bounds__(kVecThreads, kCtasPerSm) qk_norm_rope_vec_kernel(const NormParams p, const int chunks, const int steps) {
  using Raw = typename Pairs<T, P>::Raw;
  const int lanes = LPH ? LPH : p.d / (2 * P);
  const int per_warp = 32 / lanes;
  const int wl = threadIdx.x & 31;
  const int group = wl / lanes;  // this lane's head of the warp's
  const int lane = wl - group * lanes;
  const int hq = p.heads[0], hk = p.heads[1], total = hq + hk + p.heads[2];
  const unsigned item = blockIdx.x * (kVecThreads / 32) + (threadIdx.x >> 5);  // below 2^31: the launch sees to it
  const int token = static_cast<int>(item / static_cast<unsigned>(chunks));
  griddep_launch_dependents();
  griddep_wait();
  if (token >= p.t) return;
  // first and second values of this lane's pairs
  const int half = p.rot / 2, j = lane * P;
  const int ea = IL ? 2 * j : j < half ? j : j + half;
  const int eb = IL ? 2 * j + P : j < half ? j + half : j + half + (p.d - p.rot) / 2;
  const int first = static_cast<int>(item - static_cast<unsigned>(token) * static_cast<unsigned>(chunks)) * steps * per_warp;  // head
  const int last = group < per_warp ? min(total, first + steps * per_warp) : 0;  // lanes beyond the groups have none
  const int row = p.slots ? p.slots[token] : token;  // of the keys and values
  const int pos = p.rot ? p.positions[token] : 0;

  // the head that is fetched next, one step ahead of the one at work
  const auto kind_of = [&](int h) { return h < hq ? 0 : h < hq + hk ? 1 : 2; };
  const auto start_of = [&](int kind) { return kind == 0 ? 0 : kind == 1 ? hq : hq + hk; };
  Pairs<T, P> next;
  next.a = next.b = Raw{};
  const T* src = nullptr;
  int h_n = first + group, kind_n = -1;
  const auto fetch = [&] {
    if (h_n < last) {
      const int kind = kind_of(h_n);
      if (kind != kind_n) {
        kind_n = kind;
        src = static_cast<const T*>(p.in[kind]) + token * p.in_t[kind] + (h_n - start_of(kind)) * p.in_h[kind];
      }
      next.a = *reinterpret_cast<const Raw*>(src + ea);
      next.b = *reinterpret_cast<const Raw*>(src + eb);
      src += per_warp * p.in_h[kind];
    }
    h_n += per_warp;
  };
  fetch();
  float4 c[P / 4], s[P / 4];
  if (j < half) {
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
  const bool kept = row >= 0 && row < p.cache_rows;
  const float inv_d = 1.f / static_cast<float>(p.d);
  Pairs<T, P> weight;
  weight.a = weight.b = Raw{};
  T* dst = nullptr;
  int kind = -1;
  bool weighted = false;
  for (int i = 0, h = first + group; i < steps; ++i, h += per_warp) {
    Pairs<T, P> x = next;
    fetch();
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
    if (h >= last) continue;
    if (kind_of(h) != kind) {
      kind = kind_of(h);
      dst = static_cast<T*>(p.out[kind]) + (kind ? row : token) * p.out_t[kind] + (h - start_of(kind)) * p.out_h[kind];
      weighted = kind < 2 && p.weight[kind];
      if (weighted) {
        weight.a = __ldg(reinterpret_cast<const Raw*>(static_cast<const T*>(p.weight[kind]) + ea));
        weight.b = __ldg(reinterpret_cast<const Raw*>(static_cast<const T*>(p.weight[kind]) + eb));
      }
    }
    if (kind > 0 && !kept) continue;
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
    *reinterpret_cast<Raw*>(dst + ea) = x.a;
    *reinterpret_cast<Raw*>(dst + eb) = x.b;
    dst += per_warp * p.out_h[kind];
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

// A warp takes a whole token where that fills the GPU; with fewer tokens each is
// split over as many warps as the GPU holds (2040 tokens x 21 heads x 72: two
// warps a token 6.0 us, three 7.2; 16384 x 48 x 128: one 75.7, two 77.7).
template <typename T, int P, int LPH>
cudaError_t launch_heads(const NormParams& p, int device, int sms, cudaStream_t stream) {
  const int per_warp = 32 / (LPH ? LPH : p.d / (2 * P));
  const int most = (p.heads[0] + p.heads[1] + p.heads[2] + per_warp - 1) / per_warp;  // steps of a token
  const int resident = kCtasPerSm * sms * (kVecThreads / 32);
  const int split = std::min((resident - 1) / p.t + 1, most);
  const int steps = (most + split - 1) / split, chunks = (most + steps - 1) / steps;
  const int64_t items = static_cast<int64_t>(p.t) * chunks;
  const dim3 grid(static_cast<unsigned>((items + kVecThreads / 32 - 1) / (kVecThreads / 32)));
  static Kernel adjacent, halves;
  return p.interleaved
             ? adjacent.launch(qk_norm_rope_vec_kernel<T, P, LPH, true>, device, grid, kVecThreads, 0, 1, stream, p, chunks, steps)
             : halves.launch(qk_norm_rope_vec_kernel<T, P, LPH, false>, device, grid, kVecThreads, 0, 1, stream, p, chunks, steps);
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
