// Shared declarations of the token operators (linear layer, query/key norm
// with rotation, window attention): launch parameters, type helpers and the
// launchers that token_host.cpp chooses from.
#pragma once

#include <atomic>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/oidnx.h"
#include "internal.h"

namespace oidnx {

// ---------------------------------------------------------------- types
template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two consecutive 16-bit values <-> one 32-bit word.
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// The 16 bytes of a vector load as fp32 values (8 of 16 bits or 4 of 32), and back.
template <typename T> struct Vec16 {
  static constexpr int N = 16 / sizeof(T);
  static __device__ __forceinline__ void unpack(uint4 r, float (&v)[N]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack2<T>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
      else w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// ---------------------------------------------------------------- linear
// y[i][j] = act(sum_k x[i][k] w[j][k] + bias[j]) + residual[i][j]; row strides
// in elements.
struct LinearParams {
  const void* x;
  const void* w;
  const void* bias;      // [n] or null
  const void* residual;  // or null
  void* y;
  int64_t ldx, ldw, ldr, ldy;
  int m, n, k, act;
  int* status;
};

// Matrices of k values a row to be copied to rows that start on 16 bytes.
struct AlignParams {
  struct Matrix {
    const void* from;
    void* to;
    int64_t ld, ld_to, rows;
  } matrix[2];
  int k;
};

// Launch of a tensor-core form; maps that a form does not use are zero.
struct LinearTcLaunch {
  LinearParams p;
  CUtensorMap map_x, map_w, map_r, map_y;
  int device, sms;
  int bn;       // columns per tile: 64 or 128 (pair: 128 or 256); split form: tokens per tile
  int pair;     // CTA pairs on tiles of 256 rows
  int gather;   // split form: x and w through plain loads
  int tma_out;  // y and residual through TMA
  int split;    // split form: CTAs of a cluster along K
};

// A kernel of the token operators, launched through the driver's call: a
// single-token step is bound by the host, and the runtime's launch (symbol
// look-up, configuration) is most of what this library adds to it.
struct Kernel {
  std::atomic<CUfunction> fn[64] = {};  // by device

  template <typename... KArgs, typename... Args>
  cudaError_t launch(void (*kernel)(KArgs...), int device, dim3 grid, int threads, int smem, int cluster,
                     cudaStream_t stream, const Args&... args) {
    CUfunction f = fn[device].load(std::memory_order_acquire);
    if (!f) {
      const cudaError_t e = find(reinterpret_cast<const void*>(kernel), smem, device, &f);
      if (e != cudaSuccess) return e;
    }
    void* params[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    static_assert(sizeof...(KArgs) == sizeof...(Args), "one value a parameter");
    static_assert((std::is_same<KArgs, Args>::value && ...), "of its type");
    return launch_found(f, grid, threads, smem, cluster, stream, params);
  }
  // Clusters that the device holds at once (by its GPCs: 15 of eight CTAs of one
  // an SM, not 152 / 8).
  template <typename K> int clusters(K kernel, int device, int threads, int smem, int cluster) {
    return count_clusters(reinterpret_cast<const void*>(kernel), device, threads, smem, cluster);
  }

 private:
  std::atomic<int> held[4][64] = {};  // by log2 of the cluster, device
  int count_clusters(const void* kernel, int device, int threads, int smem, int cluster);
  cudaError_t find(const void* kernel, int smem, int device, CUfunction* f);
  static cudaError_t launch_found(CUfunction f, dim3 grid, int threads, int smem, int cluster, cudaStream_t stream,
                                  void** params);
};

// ---------------------------------------------------------------- norm and rotation
// Index 0 = queries, 1 = keys, 2 = values; strides in elements.
struct NormParams {
  const void* in[3];
  void* out[3];
  int64_t in_t[3], in_h[3], out_t[3], out_h[3];
  int heads[3];
  const void* weight[2];
  float eps;
  const float* cos_t;
  const float* sin_t;
  int64_t table_rows;
  const int* positions;
  const int* slots;  // or null: row t
  int64_t cache_rows;
  int t, d, rot, interleaved;
  int wide;  // vector form: 16-byte loads of 16-bit values (else 8-byte)
};

// ---------------------------------------------------------------- attention
// Strides in elements: batch, token, head.
struct AttnParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;         // [b][hq][tq] or null
  const int* q_lens;  // [b] or null: tq
  const int* kv_lens; // [b] or null: cap
  int64_t q_s[3], k_s[3], v_s[3], o_s[3];
  int b, tq, cap, hq, hk, d;
  int window;  // 0: none
  int sinks;
  int held_sinks;  // min(sinks, cap): the slots that the ring leaves alone
  float scale;
  int* status;
  int group, per, pairs;  // for prompts: heads a key head, queries a row tile, pairs of row tiles
};

__device__ __forceinline__ int attn_q_len(const AttnParams& p, int b) {
  const int n = p.q_lens ? p.q_lens[b] : p.tq;
  return n < 0 ? 0 : n > p.tq ? p.tq : n;
}
__device__ __forceinline__ int attn_kv_len(const AttnParams& p, int b) {
  const int n = p.kv_lens ? p.kv_lens[b] : p.cap;
  return n < 0 ? 0 : min(n, 1 << 30);
}
// First position after the sinks whose key the cache still holds when n keys
// have been written: the ring keeps the last cap - held_sinks of them.
__device__ __forceinline__ int attn_ring_begin(const AttnParams& p, int n) {
  const int b = n - (p.cap - p.held_sinks);
  return b > p.held_sinks ? b : p.held_sinks;
}
// Cache slot of a held position.
__device__ __forceinline__ int attn_slot(const AttnParams& p, int pos) {
  if (pos < p.cap) return pos;
  return p.held_sinks + (pos - p.held_sinks) % (p.cap - p.held_sinks);
}

cudaError_t launch_linear_tc(const LinearTcLaunch& L, bool bf16, cudaStream_t stream);
cudaError_t launch_align_rows(const AlignParams& p, int count, int device, int sms, cudaStream_t stream);
cudaError_t launch_linear_split(const LinearTcLaunch& L, bool bf16, cudaStream_t stream);
cudaError_t launch_norm_vec(const NormParams& p, int precision, int device, int sms, cudaStream_t stream);
cudaError_t launch_norm_any(const NormParams& p, int precision, int device, cudaStream_t stream);
cudaError_t launch_attn_token(const AttnParams& p, bool bf16, int split, int device, cudaStream_t stream);
// CTAs in clusters of `split` that the device holds at once.
int attn_token_slots(const AttnParams& p, bool bf16, int split, int device);
struct AttnLaunch {
  AttnParams p;
  CUtensorMap map_q, map_k, map_v, map_o;
  int device;
  unsigned grid;
};
cudaError_t launch_attn_prompt(const AttnLaunch& L, bool bf16, cudaStream_t stream);    // heads of over 64 values
cudaError_t launch_attn_prompt64(const AttnLaunch& L, bool bf16, cudaStream_t stream);  // of up to 64
cudaError_t launch_attn_any(const AttnParams& p, int precision, int device, cudaStream_t stream);

}  // namespace oidnx
