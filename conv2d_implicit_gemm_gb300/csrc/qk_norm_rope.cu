// Norm of each query and key head, rotation by the token's position and the
// append of keys and values to a cache, in one pass.
//
//   r = 1 / sqrt(mean(x^2) + eps);  y = x r w;
//   pairs (a, b) of the first rot values: (a c - b s, b c + a s)
//
// with c, s the table rows of the token's position.  Each value is read and
// written once, so the bound is memory; everything between is fp32.
#include "token.h"
#include "ptx.cuh"

namespace oidnx {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormHeadsPerGroup = 4;  // heads that a lane group keeps in flight

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7FC00000); }

// One token per CTA (and 4 x 256 / LPH heads).  A head is NC 16-byte chunks on
// each of LPH lanes; the lane group keeps the token's rotation in registers
// and has the loads of its (up to four) heads in flight together.  The
// rotation pairs of the half-split form are whole chunks rot / 2 values
// apart, exchanged as raw words between lanes; adjacent pairs lie within a
// chunk.
template <typename T, int LPH, int NC>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_vec_kernel(const NormParams p) {
  constexpr int V = Vec16<T>::N;
  constexpr int G = kNormThreads / LPH;
  constexpr int U = kNormHeadsPerGroup;
  const int lane = threadIdx.x % LPH;
  const int group = threadIdx.x / LPH;
  const int token = blockIdx.x;
  const int hq = p.heads[0], hk = p.heads[1], total = hq + hk + p.heads[2];
  const int chunks = p.d / V;
  const int rot_chunks = p.rot / V;
  const int half_chunks = p.interleaved ? 0 : rot_chunks / 2;
  griddep_launch_dependents();
  griddep_wait();

  const int pos = p.rot ? p.positions[token] : 0;
  const bool known = pos >= 0 && pos < p.table_rows;
  const int64_t slot = p.slots ? p.slots[token] : token;
  const bool kept = slot >= 0 && slot < p.cache_rows;

  uint4 raw[U][NC];
  int64_t to[U];  // output element offset of the head, or -1
  const int first = blockIdx.y * G * U + group;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = first + u * G;
    to[u] = -1;
#pragma unroll
    for (int i = 0; i < NC; ++i) raw[u][i] = make_uint4(0u, 0u, 0u, 0u);
    if (h >= total) continue;
    const int kind = h < hq ? 0 : h < hq + hk ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - hq : h - hq - hk;
    if (kind > 0 && !kept) continue;
    to[u] = (kind ? slot : token) * p.out_t[kind] + hh * p.out_h[kind];
    const T* src = static_cast<const T*>(p.in[kind]) + token * p.in_t[kind] + hh * p.in_h[kind];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + i * LPH;
      if (c < chunks) raw[u][i] = *reinterpret_cast<const uint4*>(src + c * V);
    }
  }

  // rotation of this lane's chunks: out = own * cs + partner * sn
  float cs[NC][V], sn[NC][V];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = lane + i * LPH;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      cs[i][e] = 1.f;
      sn[i][e] = 0.f;
    }
    if (c < rot_chunks) {
      if (!known) {
#pragma unroll
        for (int e = 0; e < V; ++e) cs[i][e] = sn[i][e] = quiet_nan();
      } else {
        const int64_t row = static_cast<int64_t>(pos) * (p.rot / 2);
        if (p.interleaved) {
          const float* ct = p.cos_t + row + c * (V / 2);
          const float* st = p.sin_t + row + c * (V / 2);
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            cs[i][2 * e] = cs[i][2 * e + 1] = ct[e];
            sn[i][2 * e] = -st[e];
            sn[i][2 * e + 1] = st[e];
          }
        } else {
          const bool low = c < half_chunks;
          const int at = (low ? c : c - half_chunks) * V;
          const float4* ct = reinterpret_cast<const float4*>(p.cos_t + row + at);
          const float4* st = reinterpret_cast<const float4*>(p.sin_t + row + at);
          const float sign = low ? -1.f : 1.f;
#pragma unroll
          for (int e = 0; e < V / 4; ++e) {
            const float4 a = ct[e], b = st[e];
            cs[i][4 * e] = a.x, cs[i][4 * e + 1] = a.y, cs[i][4 * e + 2] = a.z, cs[i][4 * e + 3] = a.w;
            sn[i][4 * e] = sign * b.x, sn[i][4 * e + 1] = sign * b.y;
            sn[i][4 * e + 2] = sign * b.z, sn[i][4 * e + 3] = sign * b.w;
          }
        }
      }
    }
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = first + u * G;
    const int kind = h < hq ? 0 : h < hq + hk ? 1 : 2;
    float v[NC][V], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      Vec16<T>::unpack(raw[u][i], v[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) sum = fmaf(v[i][e], v[i][e], sum);
    }
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o, 32);
    const float r = 1.0f / sqrtf(sum / static_cast<float>(p.d) + p.eps);
    const T* weight = kind < 2 ? static_cast<const T*>(p.weight[kind]) : nullptr;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + i * LPH;
      // partner chunk (itself where nothing is exchanged)
      const int pc = c >= rot_chunks || !half_chunks ? c : c < half_chunks ? c + half_chunks : c - half_chunks;
      uint4 other = raw[u][i];
      if (half_chunks) {
        uint4 got[NC];
#pragma unroll
        for (int s = 0; s < NC; ++s) {
          got[s].x = __shfl_sync(0xFFFFFFFFu, raw[u][s].x, pc, LPH);
          got[s].y = __shfl_sync(0xFFFFFFFFu, raw[u][s].y, pc, LPH);
          got[s].z = __shfl_sync(0xFFFFFFFFu, raw[u][s].z, pc, LPH);
          got[s].w = __shfl_sync(0xFFFFFFFFu, raw[u][s].w, pc, LPH);
        }
        other = got[0];
        if (NC > 1 && pc >= LPH) other = got[NC - 1];
      }
      if (to[u] < 0 || c >= chunks) continue;
      T* dst = static_cast<T*>(p.out[kind]) + to[u] + c * V;
      if (kind == 2) {
        *reinterpret_cast<uint4*>(dst) = raw[u][i];
        continue;
      }
      float w[V], ov[V], ow[V];
      if (weight) {
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(weight + c * V), w);
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(weight + pc * V), ow);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = ow[e] = 1.f;
      }
      Vec16<T>::unpack(other, ov);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[e] = v[i][e] * r * w[e];
        ov[e] = ov[e] * r * ow[e];
      }
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float b = p.interleaved ? w[e ^ 1] : ov[e];
        y[e] = c < rot_chunks ? fmaf(w[e], cs[i][e], b * sn[i][e]) : w[e];
      }
      *reinterpret_cast<uint4*>(dst) = Vec16<T>::pack(y);
    }
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

template <typename T, int LPH, int NC>
cudaError_t launch_vec(const NormParams& p, cudaStream_t stream) {
  const int total = p.heads[0] + p.heads[1] + p.heads[2];
  const int per = kNormThreads / LPH * kNormHeadsPerGroup;
  return launch_pdl(qk_norm_rope_vec_kernel<T, LPH, NC>, dim3(p.t, (total + per - 1) / per), dim3(kNormThreads), 0,
                    stream, p);
}

template <typename T>
cudaError_t launch_vec_t(const NormParams& p, cudaStream_t stream) {
  const int chunks = p.d / Vec16<T>::N;
  if (chunks <= 4) return launch_vec<T, 4, 1>(p, stream);
  if (chunks <= 8) return launch_vec<T, 8, 1>(p, stream);
  if (chunks <= 16) return launch_vec<T, 16, 1>(p, stream);
  if (chunks <= 32) return launch_vec<T, 32, 1>(p, stream);
  return launch_vec<T, 32, 2>(p, stream);
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
