// Norm after a branch, gate, residual, and the norm before the next branch, in
// one pass:
//
//   s = alpha residual + beta g(gate) post(x);  y = pre(s) (1 + scale) + shift
//
// A row's values stay in registers between their one read and the two writes, in
// fp32; means and variances are taken from the values themselves (the mean first,
// then the squares of what is left), so that nothing cancels.  The bound is memory.
#include <algorithm>
#include <type_traits>

#include "token_math.cuh"
#include "token_ptx.cuh"
#include "token.h"

namespace oidnx {
namespace {

constexpr int kMostThreads = 512;

__device__ __forceinline__ float gate_of(float g, int act) {
  if (act == OIDNX_GATE_TANH) return tanhf(g);
  if (act == OIDNX_GATE_SIGMOID) return 1.f / (1.f + expf(-g));
  return g;
}

// V consecutive values as they lie in memory: 16-byte pieces for V = 8, else one.
template <typename T, int V> struct Piece {
  static constexpr int N = V == 8 ? 8 * sizeof(T) / 16 : 1;
  using Raw = typename std::conditional<V == 8, uint4, T>::type;
  Raw r[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = reinterpret_cast<const Raw*>(p)[i];
  }
  __device__ __forceinline__ void load_const(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = __ldg(reinterpret_cast<const Raw*>(p) + i);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<Raw*>(p)[i] = r[i];
  }
  __device__ __forceinline__ void unpack(float (&f)[V]) const {
    if constexpr (V == 1) {
      f[0] = to_f32<T>(r[0]);
    } else {
      constexpr int M = Vec16<T>::N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float part[M];
        Vec16<T>::unpack(r[i], part);
#pragma unroll
        for (int k = 0; k < M; ++k) f[i * M + k] = part[k];
      }
    }
  }
  __device__ __forceinline__ void pack(const float (&f)[V]) {
    if constexpr (V == 1) {
      r[0] = from_f32<T>(f[0]);
    } else {
      constexpr int M = Vec16<T>::N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float part[M];
#pragma unroll
        for (int k = 0; k < M; ++k) part[k] = f[i * M + k];
        r[i] = Vec16<T>::pack(part);
      }
    }
  }
};

// Sum over the TH threads of a row, the same in all of them.  `parts` alternates
// between two buffers: who writes one has passed the barrier behind its last use.
template <int TH> __device__ __forceinline__ float row_sum(float v, float (*parts)[kMostThreads / 32], int& flip) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (TH > 32) {
    float* at = parts[flip];
    flip ^= 1;
    if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TH / 32; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(at + i);
      v += (q.x + q.y) + (q.z + q.w);
    }
  }
  return v;
}

// Rows of up to TH x CH x V values, V consecutive ones of each chunk a thread.
template <typename T, typename S, int V, int CH, int TH>
__global__ void __launch_bounds__(TH < 128 ? 128 : TH) block_norm_kernel(const BlockParams p) {
  constexpr int ROWS = TH < 128 ? 128 / TH : 1;  // of a CTA at a time
  __shared__ __align__(16) float parts[2][kMostThreads / 32];
  const int sub = TH < 128 ? threadIdx.x / TH : 0, tid = TH < 128 ? threadIdx.x % TH : threadIdx.x;
  const T* x = static_cast<const T*>(p.x);
  const S* residual = static_cast<const S*>(p.residual);
  const float inv_n = 1.f / static_cast<float>(p.n);
  int flip = 0;
  griddep_launch_dependents();
  griddep_wait();

  Piece<T, V> xr[CH];
  Piece<S, V> rr[CH];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = (c * TH + tid) * V;
      if (e < p.n) {
        xr[c].load(x + row * p.ldx + e);
        if (residual) rr[c].load(residual + row * p.ldr + e);
      }
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + sub;
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
  if (row < p.t) fetch(row);
  for (; row < p.t; row += step) {
    const int m = p.groups ? p.groups[row] : static_cast<int>(row) / p.per;
    if (m < 0 || m >= p.count) {  // padding
      if (row + step < p.t) fetch(row + step);
      continue;
    }
    float v[CH][V];
    float mean = 0.f, scale = 1.f;
    const auto statistics = [&](int norm) {
      mean = 0.f, scale = 1.f;
      if (norm == OIDNX_NORM_NONE) return;
      if (norm == OIDNX_NORM_LAYER) {
        float a = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < V; ++i) a += v[c][i];
        mean = row_sum<TH>(a, parts, flip) * inv_n;
      }
      float a = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if ((c * TH + tid) * V < p.n) {
#pragma unroll
          for (int i = 0; i < V; ++i) a = fmaf(v[c][i] - mean, v[c][i] - mean, a);
        }
      }
      scale = inverse_root(fmaf(row_sum<TH>(a, parts, flip), inv_n, p.eps));
    };
    const auto normalise = [&](int which, int c, int e) {
      if (p.norm[which] == OIDNX_NORM_NONE) return;
#pragma unroll
      for (int i = 0; i < V; ++i) v[c][i] = (v[c][i] - mean) * scale;
      float f[V];
      Piece<T, V> w;
      if (p.weight[which]) {
        w.load_const(static_cast<const T*>(p.weight[which]) + e);
        w.unpack(f);
#pragma unroll
        for (int i = 0; i < V; ++i) v[c][i] *= f[i];
      }
      if (p.bias[which]) {
        w.load_const(static_cast<const T*>(p.bias[which]) + e);
        w.unpack(f);
#pragma unroll
        for (int i = 0; i < V; ++i) v[c][i] += f[i];
      }
    };

#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if ((c * TH + tid) * V < p.n) {
        xr[c].unpack(v[c]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[c][i] = 0.f;
      }
    }
    statistics(p.norm[0]);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = (c * TH + tid) * V;
      if (e < p.n) {
        normalise(0, c, e);
        if (p.gate) {
          Piece<T, V> g;
          float f[V];
          g.load_const(static_cast<const T*>(p.gate) + m * p.ldg + e);
          g.unpack(f);
#pragma unroll
          for (int i = 0; i < V; ++i) v[c][i] *= gate_of(f[i], p.gate_act);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) v[c][i] *= p.beta;
        if (residual) {
          float f[V];
          rr[c].unpack(f);
#pragma unroll
          for (int i = 0; i < V; ++i) v[c][i] = fmaf(p.alpha, f[i], v[c][i]);
        }
        if (p.sum) {
          Piece<S, V> out;
          out.pack(v[c]);
          out.store(static_cast<S*>(p.sum) + row * p.ld_sum + e);
        }
      }
    }
    if (row + step < p.t) fetch(row + step);
    if (!p.y) continue;
    statistics(p.norm[1]);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = (c * TH + tid) * V;
      if (e < p.n) {
        normalise(1, c, e);
        Piece<T, V> w;
        float f[V];
        if (p.scale) {
          w.load_const(static_cast<const T*>(p.scale) + m * p.lds + e);
          w.unpack(f);
#pragma unroll
          for (int i = 0; i < V; ++i) v[c][i] = fmaf(v[c][i], f[i], v[c][i]);
        }
        if (p.shift) {
          w.load_const(static_cast<const T*>(p.shift) + m * p.ldh + e);
          w.unpack(f);
#pragma unroll
          for (int i = 0; i < V; ++i) v[c][i] += f[i];
        }
        w.pack(v[c]);
        w.store(static_cast<T*>(p.y) + row * p.ldy + e);
      }
    }
  }
}

// Rows of any length: a CTA a row, the values made again from x and the residual
// for each sum over them.  (A value is written by the thread that read it last, so
// outputs may be their inputs here too.)
constexpr int kLongThreads = 512;
template <typename T, typename S> __global__ void __launch_bounds__(kLongThreads) block_norm_long_kernel(const BlockParams p) {
  __shared__ __align__(16) float parts[2][kMostThreads / 32];
  const float inv_n = 1.f / static_cast<float>(p.n);
  int flip = 0;
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t row = blockIdx.x; row < p.t; row += gridDim.x) {
    const int m = p.groups ? p.groups[row] : static_cast<int>(row) / p.per;
    if (m < 0 || m >= p.count) continue;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const S* residual = p.residual ? static_cast<const S*>(p.residual) + row * p.ldr : nullptr;
    float mean[2] = {0.f, 0.f}, scale[2] = {1.f, 1.f};
    const auto normed = [&](int which, float v, int e) {
      if (p.norm[which] == OIDNX_NORM_NONE) return v;
      v = (v - mean[which]) * scale[which];
      if (p.weight[which]) v *= to_f32<T>(static_cast<const T*>(p.weight[which])[e]);
      if (p.bias[which]) v += to_f32<T>(static_cast<const T*>(p.bias[which])[e]);
      return v;
    };
    const auto total = [&](int e) {
      float v = normed(0, to_f32<T>(x[e]), e);
      if (p.gate) v *= gate_of(to_f32<T>(static_cast<const T*>(p.gate)[m * p.ldg + e]), p.gate_act);
      v *= p.beta;
      return residual ? fmaf(p.alpha, to_f32<S>(residual[e]), v) : v;
    };
    for (int which = 0; which < (p.y ? 2 : 1); ++which) {
      if (p.norm[which] == OIDNX_NORM_NONE) continue;
      for (int power = p.norm[which] == OIDNX_NORM_LAYER ? 1 : 2; power <= 2; ++power) {
        // sums of up to 2^30 / 512 values a thread: in parts of 256, so that small ones are not lost
        float sum = 0.f, part = 0.f;
        int k = 0;
        for (int e = threadIdx.x; e < p.n; e += kLongThreads) {
          const float v = which ? total(e) : to_f32<T>(x[e]);
          const float c = v - mean[which];
          part = power == 1 ? part + v : fmaf(c, c, part);
          if ((++k & 255) == 0) sum += part, part = 0.f;
        }
        const float all = row_sum<kLongThreads>(sum + part, parts, flip) * inv_n;
        if (power == 1) mean[which] = all;
        else scale[which] = inverse_root(all + p.eps);
      }
    }
    for (int e = threadIdx.x; e < p.n; e += kLongThreads) {
      float v = total(e);
      if (p.sum) static_cast<S*>(p.sum)[row * p.ld_sum + e] = from_f32<S>(v);
      if (!p.y) continue;
      v = normed(1, v, e);
      if (p.scale) v = fmaf(v, to_f32<T>(static_cast<const T*>(p.scale)[m * p.lds + e]), v);
      if (p.shift) v += to_f32<T>(static_cast<const T*>(p.shift)[m * p.ldh + e]);
      static_cast<T*>(p.y)[row * p.ldy + e] = from_f32<T>(v);
    }
  }
}

template <typename T, typename S, int V, int CH, int TH>
cudaError_t launch_rows(const BlockParams& p, int device, int sms, cudaStream_t stream) {
  constexpr int threads = TH < 128 ? 128 : TH, rows = threads / TH;
  const int64_t ctas = (static_cast<int64_t>(p.t) + rows - 1) / rows;
  const int64_t most = static_cast<int64_t>(sms) * (2048 / threads);
  static Kernel handle;
  return handle.launch(block_norm_kernel<T, S, V, CH, TH>, device, dim3(static_cast<unsigned>(std::min(ctas, most))), threads,
                       0, 1, stream, p);
}

template <typename T, typename S>
cudaError_t launch_t(const BlockParams& p, bool vector, int device, int sms, cudaStream_t stream) {
  const int n = p.n;
  if (vector) {
    if (n <= 256) return launch_rows<T, S, 8, 1, 32>(p, device, sms, stream);
    if (n <= 512) return launch_rows<T, S, 8, 2, 32>(p, device, sms, stream);
    if (n <= 1024) return launch_rows<T, S, 8, 4, 32>(p, device, sms, stream);
    if (n <= 4096 && p.t <= sms) return launch_rows<T, S, 8, 1, 512>(p, device, sms, stream);
    if (n <= 2048) return launch_rows<T, S, 8, 2, 128>(p, device, sms, stream);
    if (n <= 4096) return launch_rows<T, S, 8, 4, 128>(p, device, sms, stream);
    if (n <= 8192) return launch_rows<T, S, 8, 2, 512>(p, device, sms, stream);
    if (n <= 16384) return launch_rows<T, S, 8, 4, 512>(p, device, sms, stream);
  } else {
    if (n <= 256) return launch_rows<T, S, 1, 8, 32>(p, device, sms, stream);
    if (n <= 1024) return launch_rows<T, S, 1, 32, 32>(p, device, sms, stream);
    if (n <= 4096) return launch_rows<T, S, 1, 32, 128>(p, device, sms, stream);
    if (n <= 16384) return launch_rows<T, S, 1, 32, 512>(p, device, sms, stream);
  }
  static Kernel handle;
  return handle.launch(block_norm_long_kernel<T, S>, device, dim3(std::min(p.t, 4 * sms)), kLongThreads, 0, 1, stream, p);
}

}  // namespace

cudaError_t launch_block_norm(const BlockParams& p, bool vector, int precision, int sum_precision, int device, int sms,
                              cudaStream_t stream) {
  const bool wide = sum_precision == OIDNX_PRECISION_FP32;
  if (precision == OIDNX_PRECISION_FP32) return launch_t<float, float>(p, vector, device, sms, stream);
  if (precision == OIDNX_PRECISION_BF16)
    return wide ? launch_t<__nv_bfloat16, float>(p, vector, device, sms, stream)
                : launch_t<__nv_bfloat16, __nv_bfloat16>(p, vector, device, sms, stream);
  return wide ? launch_t<__half, float>(p, vector, device, sms, stream)
              : launch_t<__half, __half>(p, vector, device, sms, stream);
}

}  // namespace oidnx
