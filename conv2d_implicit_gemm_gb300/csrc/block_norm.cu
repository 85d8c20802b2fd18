// Norm after a branch, gate, residual, and the norm before the next branch, in
// one pass:
//
//   s = alpha residual + beta g(gate) post(x);  y = pre(s) (1 + scale) + shift
//
// A row's values stay in registers between their one read and the two writes, in fp32
// (but for rows of over 16384, which are read again for each sum).  Means come first,
// then the squares of what is left of the values, so that the squares do not cancel; a
// value less its mean is off by the mean's own rounding, 2^-24 of it.  The bound is memory.
#include <algorithm>
#include <type_traits>

#include "token_math.cuh"
#include "token_pairs.cuh"
#include "token_warp.cuh"
#include "token.h"

namespace oidnx {
namespace {

constexpr int kMostThreads = 512;

__device__ __forceinline__ float gate_of(float g, int act) {
  if (act == OIDNX_GATE_TANH) return tanhf(g);
  if (act == OIDNX_GATE_SIGMOID) return 1.f / (1.f + expf(-g));
  return g;
}

// A thread's E values of a row: pieces of 8 a team apart (V = 8), or single ones.  They
// are fetched as words, zeros past the row, and worked on in pairs.
template <int V, int E> struct Mine {
  static constexpr int PAIRS = E / 2, N = E / V;
  int first, step, count;  // pieces first, first + step, ..; those within the row
  bool full;               // single ones, all of the warp's within it
  __device__ __forceinline__ Mine(int first, int step, int n) : first(first), step(step) {
    count = first < n ? min((n - first + step - 1) / step, N) : 0;
    full = V == 1 && (first | (min(step, 32) - 1)) + step * (N - 1) < n;
  }
  template <typename U> static constexpr int kWords = V == 8 ? E * static_cast<int>(sizeof(U)) / 4 : E;

  // (words past the row are left alone)
  template <typename U, int W> __device__ __forceinline__ void fetch(const U* p, uint32_t (&w)[W]) const {
    if (full) fetch_part<true>(p, w);
    else fetch_part<false>(p, w);
  }
  template <bool ALL, typename U, int W> __device__ __forceinline__ void fetch_part(const U* p, uint32_t (&w)[W]) const {
    static_assert(W == kWords<U>, "");
    p += first;
#pragma unroll
    for (int c = 0; c < N; ++c, p += step) {
      if (ALL || c < count) {
        if constexpr (V == 8) {
          constexpr int Q = sizeof(U) / 2;
#pragma unroll
          for (int k = 0; k < Q; ++k) {
            const uint4 q = reinterpret_cast<const uint4*>(p)[k];
            w[(c * Q + k) * 4] = q.x, w[(c * Q + k) * 4 + 1] = q.y, w[(c * Q + k) * 4 + 2] = q.z, w[(c * Q + k) * 4 + 3] = q.w;
          }
        } else if constexpr (sizeof(U) == 2) {
          w[c] = *reinterpret_cast<const uint16_t*>(p);
        } else {
          w[c] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
    }
  }
  template <typename U, int W> static __device__ __forceinline__ void pairs(const uint32_t (&w)[W], uint64_t (&v)[PAIRS]) {
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      if constexpr (sizeof(U) == 4) {
        v[i] = f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      } else if constexpr (V == 1) {
        v[i] = f2(unpack2<U>(w[2 * i]).x, unpack2<U>(w[2 * i + 1]).x);
      } else {
        const float2 u = unpack2<U>(w[i]);
        v[i] = f2(u.x, u.y);
      }
    }
  }
  template <typename U> __device__ __forceinline__ void load(const U* p, uint64_t (&v)[PAIRS]) const {
    uint32_t w[kWords<U>] = {};
    fetch(p, w);
    pairs<U>(w, v);
  }
  // (whole: fp32 rows that start on 32 bytes)
  template <typename U> __device__ __forceinline__ void store(U* p, const uint64_t (&v)[PAIRS], bool whole = false) const {
    uint32_t w[E * sizeof(U) / 4];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const float2 u = f2_of(v[i]);
      if constexpr (sizeof(U) == 4) w[2 * i] = __float_as_uint(u.x), w[2 * i + 1] = __float_as_uint(u.y);
      else w[i] = pack2<U>(u.x, u.y);
    }
    if constexpr (V == 8 && sizeof(U) == 4) {
      if (whole) {
        p += first;
#pragma unroll
        for (int c = 0; c < N; ++c, p += step)
          if (c < count)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[c * 8]), "r"(w[c * 8 + 1]),
                         "r"(w[c * 8 + 2]), "r"(w[c * 8 + 3]), "r"(w[c * 8 + 4]), "r"(w[c * 8 + 5]), "r"(w[c * 8 + 6]),
                         "r"(w[c * 8 + 7])
                         : "memory");
        return;
      }
    }
    if (full) store_part<true>(p, w);
    else store_part<false>(p, w);
  }
  template <bool ALL, typename U, int W> __device__ __forceinline__ void store_part(U* p, const uint32_t (&w)[W]) const {
    p += first;
#pragma unroll
    for (int c = 0; c < N; ++c, p += step) {
      if (ALL || c < count) {
        if constexpr (V == 8) {
          constexpr int Q = sizeof(U) / 2;
#pragma unroll
          for (int k = 0; k < Q; ++k)
            reinterpret_cast<uint4*>(p)[k] =
                make_uint4(w[(c * Q + k) * 4], w[(c * Q + k) * 4 + 1], w[(c * Q + k) * 4 + 2], w[(c * Q + k) * 4 + 3]);
        } else if constexpr (sizeof(U) == 2) {
          *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(c % 2 ? w[c / 2] >> 16 : w[c / 2]);
        } else {
          *reinterpret_cast<uint32_t*>(p) = w[c];
        }
      }
    }
  }
  // zeros in the places past the row
  __device__ __forceinline__ void clear(uint64_t (&v)[PAIRS]) const {
    if (full) return;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      if constexpr (V == 8) {
        if (2 * i / V >= count) v[i] = 0;
      } else {
        float2 u = f2_of(v[i]);
        u.x = 2 * i < count ? u.x : 0.f, u.y = 2 * i + 1 < count ? u.y : 0.f;
        v[i] = f2(u.x, u.y);
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

// A row a value at a time, made again from x and the residual for each sum over it, its
// factors one after the other: the thread's pieces of V values from `first` on, `step`
// apart, below `end`.  sum_of adds over the row's threads.  (A value is written by the
// thread that read it last, so outputs may be their inputs here too.)
template <typename T, typename S, int V, typename Sum>
__device__ __forceinline__ void by_values(const BlockParams& p, int64_t row, int m, int first, int step, int end, const Sum& sum_of) {
  const float inv_n = 1.f / static_cast<float>(p.n);
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
      for (int at = first; at < end; at += step) {
        for (int e = at; e < at + V; ++e) {
          const float v = which ? total(e) : to_f32<T>(x[e]);
          const float c = v - mean[which];
          part = power == 1 ? part + v : fmaf(c, c, part);
          if ((++k & 255) == 0) sum += part, part = 0.f;
        }
      }
      const float all = sum_of(sum + part) * inv_n;
      if (power == 1) mean[which] = all;
      else scale[which] = inverse_root(all + p.eps);
    }
  }
  for (int at = first; at < end; at += step) {
    for (int e = at; e < at + V; ++e) {
      float v = total(e);
      if (p.sum) static_cast<S*>(p.sum)[row * p.ld_sum + e] = from_f32<S>(v);
      if (!p.y) continue;
      v = normed(1, v, e);
      if (p.scale) v *= 1.f + to_f32<T>(static_cast<const T*>(p.scale)[m * p.lds + e]);
      if (p.shift) v += to_f32<T>(static_cast<const T*>(p.shift)[m * p.ldh + e]);
      static_cast<T*>(p.y)[row * p.ldy + e] = from_f32<T>(v);
    }
  }
}

// Few rows, or long ones: a CTA a row of up to 512 x E values.
template <typename T, typename S, int V, int E>
__global__ void __launch_bounds__(kMostThreads) block_norm_kernel(const BlockParams p) {
  constexpr int TH = kMostThreads, PAIRS = E / 2;
  __shared__ __align__(16) float parts[2][kMostThreads / 32];
  const Mine<V, E> own(threadIdx.x * V, TH * V, p.n);
  const float inv_n = 1.f / static_cast<float>(p.n);
  int flip = 0;
  griddep_launch_dependents();
  griddep_wait();

  for (int64_t row = blockIdx.x; row < p.t; row += gridDim.x) {
    const int m = p.groups ? p.groups[row] : static_cast<int>(row) / p.per;
    if (m < 0 || m >= p.count) continue;  // padding
    uint32_t rw[Mine<V, E>::template kWords<S>] = {};
    uint64_t v[PAIRS], f[PAIRS];
    own.load(static_cast<const T*>(p.x) + row * p.ldx, v);
    if (p.residual) own.fetch(static_cast<const S*>(p.residual) + row * p.ldr, rw);
    float mean, root;
    const auto statistics = [&](int norm) {  // of v, which is zero past the row
      mean = 0.f, root = 1.f;
      if (norm == OIDNX_NORM_NONE) return;
      uint64_t a = 0, b = 0;
      if (norm == OIDNX_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) a = add2(a, v[i]);
        const float2 u = f2_of(a);
        mean = row_sum<TH>(u.x + u.y, parts, flip) * inv_n;
        a = 0;
      }
      uint64_t c[PAIRS];
      const uint64_t less = f2(-mean, -mean);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) c[i] = add2(v[i], less);
      own.clear(c);
#pragma unroll
      for (int i = 0; i < PAIRS; i += 2) a = fma2(c[i], c[i], a), b = fma2(c[i + 1], c[i + 1], b);
      const float2 u = f2_of(add2(a, b));
      root = inverse_root(fmaf(row_sum<TH>(u.x + u.y, parts, flip), inv_n, p.eps));
    };
    const auto normalise = [&](int which) {
      if (p.norm[which] == OIDNX_NORM_NONE) return;
      statistics(p.norm[which]);
      const uint64_t roots = f2(root, root), shifts = f2(-mean * root, -mean * root);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) v[i] = fma2(v[i], roots, shifts);
      if (p.weight[which]) {
        own.load(static_cast<const T*>(p.weight[which]), f);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) v[i] = mul2(v[i], f[i]);
      }
      if (p.bias[which]) {
        own.load(static_cast<const T*>(p.bias[which]), f);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) v[i] = add2(v[i], f[i]);
      }
      own.clear(v);
    };
    normalise(0);
    const uint64_t beta = f2(p.beta, p.beta), alpha = f2(p.alpha, p.alpha);
    if (p.gate) {
      own.load(static_cast<const T*>(p.gate) + m * p.ldg, f);
      if (p.gate_act != OIDNX_GATE_PLAIN) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          const float2 u = f2_of(f[i]);
          f[i] = f2(gate_of(u.x, p.gate_act), gate_of(u.y, p.gate_act));
        }
      }
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) v[i] = mul2(v[i], f[i]);
    }
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) v[i] = mul2(v[i], beta);
    if (p.residual) {
      Mine<V, E>::template pairs<S>(rw, f);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) v[i] = fma2(f[i], alpha, v[i]);
    }
    if (p.sum) own.store(static_cast<S*>(p.sum) + row * p.ld_sum, v);
    if (!p.y) continue;
    normalise(1);
    if (p.scale) {
      own.load(static_cast<const T*>(p.scale) + m * p.lds, f);
      const uint64_t one = f2(1.f, 1.f);  // (not v + v scale: an infinite v under a negative scale)
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) v[i] = mul2(v[i], add2(f[i], one));
    }
    if (p.shift) {
      own.load(static_cast<const T*>(p.shift) + m * p.ldh, f);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) v[i] = add2(v[i], f[i]);
    }
    own.store(static_cast<T*>(p.y) + row * p.ldy, v);
  }
}

// Many rows of up to 8192 values: teams of 8 or 16 lanes of a warp or of whole warps
// take consecutive rows, 16 values a thread.  Rows come through a ring in shared memory
// (cp.async, one row ahead or two), and what stands beside a row (weights, gate,
// modulation) is multiplied together once a group and stays in registers:
//
//   s = alpha r + a (x - mean) root + b,   a = beta g w_post,   b = beta g b_post
//   y = (s - mean) root c + d,             c = (1 + scale) w_pre, d = (1 + scale) b_pre + shift
//
// Where such a product is beyond fp32 (a gate of infinity; factors of 1e30 and 1e-30) the
// team's rows from there on go value by value, their factors one after the other as in the
// other kernels.
//
// A thread copies the pieces that it will read itself.  Rows that do not start on 16
// bytes are copied by each warp for itself, from the 16 bytes that its 512 values start
// in to the 16 that they end in (which are in their pages).
//
// 16384 rows of 4096 in bf16: 86 us, 6.2 TB/s, 92% of the measured copy rate (8192 of
// 8192 94, 131072 of 512 86, 262144 of 128 47); with an fp32 sum 126 us, 94%.  Odd
// widths, a value at a time: 16384 of 4095 144 us, 65536 of 1001 118; what bounds these
// is instructions.  All 128 registers are taken, so what can be made again from the row
// is (3 to 7% of an odd width).  Not kept: teams of powers of two in warps, their values
// apart by the team's width (101, 143, 219, and 140 for rows of 128 on a whole warp),
// rows side by side sharing a wait (105 to 127 us), what stands beside the rows in shared
// memory (124 and up), rows copied whole by one thread (178), a check of the team's width
// in one kernel for all (17% more), fp32 rows copied lane by lane (1% either way).
constexpr int kRingThreads = 512;
constexpr int kMostParts = 32;  // in fours a team: 8 teams of a warp, 3 of 5
struct RingParams : BlockParams {
  int team, stages;
  int x_bytes, stage_bytes;  // of a stage: x, then the residual
  bool whole_sum, whole_y;   // fp32 rows that start on 32 bytes
};
constexpr int kRingBytes = 144 * 1024;  // 8192 fp32 values and their residuals twice, and what stands beside rows

// Whether v is true for any of the barrier's threads.
__device__ __forceinline__ bool named_barrier_any(int id, int threads, bool v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n selp.s32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<int>(v))
      : "memory");
  return r != 0;
}

// Sum over a team, the same in all its threads.
template <int LANES>
__device__ __forceinline__ float sum_of_team(float v, int team, int mine, float (*parts)[kMostParts], int& flip) {
  const int warps = team / 32, slots = (warps + 3) & ~3;
  const uint32_t lanes = LANES < 32 ? ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1)) : 0xFFFFFFFFu;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(lanes, v, o);
  if (LANES < 32 || warps == 1) return v;
  float* to = parts[flip] + mine * slots;
  flip ^= 1;
  if ((threadIdx.x & 31) == 0) to[(threadIdx.x - mine * team) >> 5] = v;
  __syncwarp();
  named_barrier_sync(1 + mine, team);
  float4 q = *reinterpret_cast<const float4*>(to);
  v = (q.x + q.y) + (q.z + q.w);
  for (int i = 4; i < warps; i += 4) {
    q = *reinterpret_cast<const float4*>(to + i);
    v += (q.x + q.y) + (q.z + q.w);
  }
  return v;
}

// The rows from `row` to `end` of a team value by value: outside the kernel, whose registers
// it would take, where rows are whole pieces (16384 x 4096 86 us, within 92); within it for
// single values, which lose more by the call (65536 x 1001 118 us, 124).
template <typename T, typename S, int V, int LANES>
__device__ __forceinline__ void rows_by_values(const RingParams& p, int row, int end, int first, int team, int mine,
                                               float (*parts)[kMostParts], int flip) {
  for (; row < end; ++row) {
    const int m = p.groups ? p.groups[row] : row / p.per;
    if (m >= 0 && m < p.count)
      by_values<T, S, V>(p, row, m, first, LANES * V, min(first + 16 * LANES, p.n),
                         [&](float v) { return sum_of_team<LANES>(v, team, mine, parts, flip); });
  }
}

template <typename T, typename S, int V, int LANES>
__device__ __noinline__ void rows_apart(const RingParams& p, int row, int end, int first, int team, int mine,
                                        float (*parts)[kMostParts], int flip) {
  rows_by_values<T, S, V, LANES>(p, row, end, first, team, mine, parts, flip);
}

// Teams of LANES threads, or of warps, each with 16 x 32 consecutive values.
template <typename T, typename S, int V, int LANES>
__global__ void __launch_bounds__(kRingThreads, 1) block_norm_ring_kernel(const __grid_constant__ RingParams p) {
  constexpr int PAIRS = 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float parts[2][kMostParts];
  const int team = LANES < 32 ? LANES : p.team, mine = threadIdx.x / team, tid = threadIdx.x - mine * team;
  // the team's lanes of its warp
  const uint32_t lanes = LANES < 32 ? ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1)) : 0xFFFFFFFFu;
  if constexpr (LANES == 32) {  // (those of no warp stay zero)
    if (threadIdx.x < 2 * kMostParts) parts[0][threadIdx.x] = 0.f;
    __syncthreads();
  }
  uint8_t* ring = smem + mine * p.stages * p.stage_bytes;
  const int64_t teams = static_cast<int64_t>(gridDim.x) * (blockDim.x / team);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + mine;
  const int begin = static_cast<int>(p.t * at / teams), end = static_cast<int>(p.t * (at + 1) / teams);
  griddep_launch_dependents();
  griddep_wait();

  const Mine<V, 16> own(tid / LANES * (LANES * 16) + tid % LANES * V, LANES * V, p.n);
  // bytes of a row's first 16 that stand before it
  const auto skip = [](const auto* q, int row, int64_t ld) {
    const uint32_t start = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q));
    return V == 8 ? 0u : (start + row * static_cast<uint32_t>(ld * sizeof(*q))) & 15u;
  };
  const uint32_t warp = V == 8 ? 0u : tid / LANES;
  const T* x_next = static_cast<const T*>(p.x) + begin * p.ldx;  // the row that is fetched next
  const S* r_next = static_cast<const S*>(p.residual) + (p.residual ? begin * p.ldr : 0);
  const auto copy_row = [&](uint32_t to, const auto* row) {
    constexpr int size = sizeof(*row);
    if constexpr (V == 8) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (c < own.count) {
#pragma unroll
          for (int k = 0; k < size / 2; ++k)
            cp_async16(to + (own.first + c * own.step) * size + 16 * k,
                       reinterpret_cast<const uint8_t*>(row + own.first + c * own.step) + 16 * k, 16u);
        }
    } else {
      // (a warp's part starts 16 bytes further on than the last one's, which its first 16 bytes end)
      const uint32_t before = reinterpret_cast<uintptr_t>(row) & 15u;
      const uint32_t most = before + min(static_cast<uint32_t>(p.n), (warp + 1) * 16 * LANES) * size;
      const uint8_t* from = reinterpret_cast<const uint8_t*>(row) - before;
      for (uint32_t k = warp * 16 * LANES * size + tid % LANES * 16; k < most; k += LANES * 16)
        cp_async16(to + k + warp * 16, from + k, 16u);
    }
  };
  const auto fetch = [&](int row, int stage) {
    if (row < end) {
      const uint32_t to = smem_u32(ring + stage * p.stage_bytes);
      copy_row(to, x_next);
      x_next += p.ldx;
      if (p.residual) {
        copy_row(to + p.x_bytes, r_next);
        r_next += p.ldr;
      }
    }
    cp_async_commit();
  };
  for (int s = 0; s + 1 < p.stages; ++s) fetch(begin + s, s);

  const float inv_n = 1.f / static_cast<float>(p.n);
  int flip = 0;
  const auto team_sum = [&](float v) { return sum_of_team<LANES>(v, team, mine, parts, flip); };
  uint64_t v[PAIRS];
  float mean = 0.f, root = 1.f;
  const auto statistics = [&](int norm) {  // of v, which is zero past the row
    mean = 0.f, root = 1.f;
    if (norm == OIDNX_NORM_NONE) return;
    uint64_t c[PAIRS], a = 0, b = 0;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) c[i] = v[i];
    if (norm == OIDNX_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < PAIRS; i += 2) a = add2(a, v[i]), b = add2(b, v[i + 1]);
      const float2 u = f2_of(add2(a, b));
      mean = team_sum(u.x + u.y) * inv_n;
      a = b = 0;
      const uint64_t less = f2(-mean, -mean);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) c[i] = add2(v[i], less);
      own.clear(c);
    }
#pragma unroll
    for (int i = 0; i < PAIRS; i += 2) a = fma2(c[i], c[i], a), b = fma2(c[i + 1], c[i + 1], b);
    const float2 u = f2_of(add2(a, b));
    root = inverse_root(fmaf(team_sum(u.x + u.y), inv_n, p.eps));
  };

  uint64_t ca[PAIRS], cb[PAIRS], cc[PAIRS], cd[PAIRS];
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) ca[i] = cb[i] = cc[i] = cd[i] = 0;
  const auto read = [&](const void* q, int64_t offset, uint64_t (&f)[PAIRS], float none) {
    if (q) {
      own.load(static_cast<const T*>(q) + offset, f);
    } else {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) f[i] = f2(none, none);
      own.clear(f);
    }
  };
  int group = -1, group_end = begin;  // rows of one group, where they follow one another
  bool kept = false;
  S* sum_row = static_cast<S*>(p.sum) + (p.sum ? begin * p.ld_sum : 0);
  T* y_row = static_cast<T*>(p.y) + (p.y ? begin * p.ldy : 0);
  int stage = 0;
#pragma unroll 1
  for (int row = begin; row < end; ++row) {
    if (row >= group_end) {
      const int m = p.groups ? p.groups[row] : row / p.per;
      group_end = p.groups ? row + 1 : static_cast<int>(min(static_cast<int64_t>(m + 1) * p.per, static_cast<int64_t>(end)));
      kept = m >= 0 && m < p.count;  // else padding
      if (kept && m != group) {
        group = m;
        uint64_t f[PAIRS], g[PAIRS];
        const uint64_t beta = f2(p.beta, p.beta);
        read(p.gate, m * p.ldg, g, 1.f);
        if (p.gate && p.gate_act != OIDNX_GATE_PLAIN) {
#pragma unroll
          for (int i = 0; i < PAIRS; ++i) {
            const float2 u = f2_of(g[i]);
            g[i] = f2(gate_of(u.x, p.gate_act), gate_of(u.y, p.gate_act));
          }
          own.clear(g);
        }
        bool lost = false;  // a gate's product with beta, below the normal values
        if (fabsf(p.beta) < 1.f && p.beta != 0.f) {
          constexpr float least = 1.17549435e-38f;
#pragma unroll
          for (int i = 0; i < PAIRS; ++i) {
            const float2 u = f2_of(g[i]);
            lost |= (u.x != 0.f && fabsf(u.x * p.beta) < least) || (u.y != 0.f && fabsf(u.y * p.beta) < least);
          }
        }
        read(p.weight[0], 0, f, 1.f);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) g[i] = mul2(g[i], beta), ca[i] = mul2(f[i], g[i]);
        read(p.bias[0], 0, f, 0.f);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) cb[i] = mul2(f[i], g[i]);
        read(p.scale, m * p.lds, g, 0.f);
        read(p.weight[1], 0, f, 1.f);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) cc[i] = fma2(f[i], g[i], f[i]);
        read(p.bias[1], 0, f, 0.f);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) cd[i] = fma2(f[i], g[i], f[i]);
        read(p.shift, m * p.ldh, g, 0.f);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) cd[i] = add2(cd[i], g[i]);
        uint64_t none[2] = {0, 0};  // 0, or NaN where a product is infinite or none
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          none[0] = fma2(ca[i], 0, fma2(cb[i], 0, none[0]));
          none[1] = fma2(cc[i], 0, fma2(cd[i], 0, none[1]));
        }
        const float2 u = f2_of(add2(none[0], none[1]));
        lost = __any_sync(lanes, lost || u.x + u.y != 0.f);
        if (LANES == 32 && team > 32) {
          __syncwarp();
          lost = named_barrier_any(1 + mine, team, lost);
        }
        if (lost) {
          if constexpr (V == 1) rows_by_values<T, S, V, LANES>(p, row, end, own.first, team, mine, parts, flip);
          else rows_apart<T, S, V, LANES>(p, row, end, own.first, team, mine, parts, flip);
          cp_async_wait<0>();
          return;
        }
      }
    }
    // stages is 2 or 3, and stages - 1 rows are in flight: this one is the oldest
    if (p.stages == 2) cp_async_wait<0>();
    else cp_async_wait<1>();
    if constexpr (V == 1) __syncwarp(lanes);  // its lanes have copied its part together
    fetch(row + p.stages - 1, (stage == 0 ? p.stages : stage) - 1);  // over the last row, which every reader is done with
    const uint8_t* from = ring + stage * p.stage_bytes + warp * 16;
    if (kept) {
      own.load(reinterpret_cast<const T*>(from + skip(static_cast<const T*>(p.x), row, p.ldx)), v);
      statistics(p.norm[0]);
      const uint64_t roots = f2(root, root), shifts = f2(-mean * root, -mean * root);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) v[i] = fma2(fma2(v[i], roots, shifts), ca[i], cb[i]);
      if (p.residual) {
        uint64_t r[PAIRS];
        own.load(reinterpret_cast<const S*>(from + p.x_bytes + skip(static_cast<const S*>(p.residual), row, p.ldr)), r);
        const uint64_t alpha = f2(p.alpha, p.alpha);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) v[i] = fma2(r[i], alpha, v[i]);
      }
      if (p.sum) own.store(sum_row, v, p.whole_sum);
      if (p.y) {
        statistics(p.norm[1]);
      }
    }
    if (kept && p.y) {
      const uint64_t roots = f2(root, root), shifts = f2(-mean * root, -mean * root);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) v[i] = fma2(fma2(v[i], roots, shifts), cc[i], cd[i]);
      own.store(y_row, v, p.whole_y);
    }
    sum_row += p.ld_sum, y_row += p.ldy;
    if (++stage == p.stages) stage = 0;
  }
}

// Rows of any length: a CTA a row, a value at a time.
constexpr int kLongThreads = 512;
template <typename T, typename S> __global__ void __launch_bounds__(kLongThreads, 3) block_norm_long_kernel(const BlockParams p) {
  __shared__ __align__(16) float parts[2][kMostThreads / 32];
  int flip = 0;
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t row = blockIdx.x; row < p.t; row += gridDim.x) {
    const int m = p.groups ? p.groups[row] : static_cast<int>(row) / p.per;
    if (m < 0 || m >= p.count) continue;
    by_values<T, S, 1>(p, row, m, threadIdx.x, kLongThreads, p.n, [&](float v) { return row_sum<kLongThreads>(v, parts, flip); });
  }
}

template <typename T, typename S, int V, int E>
cudaError_t launch_rows(const BlockParams& p, int device, int sms, cudaStream_t stream) {
  static Kernel handle;
  return handle.launch(block_norm_kernel<T, S, V, E>, device, dim3(std::min(p.t, 4 * sms)), kMostThreads, 0, 1, stream, p);
}

template <typename T, typename S, int V, int LANES>
cudaError_t launch_teams(const BlockParams& p, int device, int sms, cudaStream_t stream) {
  RingParams q;
  static_cast<BlockParams&>(q) = p;
  q.team = LANES < 32 ? LANES : (p.n + 511) / 512 * 32;
  // two CTAs an SM, or one where that holds more teams
  const int ctas = kRingThreads / q.team > kRingThreads / 2 / q.team * 2 ? 1 : 2, teams = kRingThreads / ctas / q.team;
  const int beside = V == 8 ? 0 : 15 + 16 * std::max(1, q.team / 32);  // before a row, and between its warps' parts
  const auto bytes = [&](int size) { return (p.n * size + beside + 15) / 16 * 16; };
  q.x_bytes = bytes(sizeof(T));
  q.stage_bytes = q.x_bytes + (p.residual ? bytes(sizeof(S)) : 0);
  // One row ahead, for one or two teams two while that is 64 KB at most: more in flight
  // slows the writes down (us with 2 and 3 stages: 131072 rows of 512 87, 98, 32768 of 2048
  // 89, 97, with an fp32 sum 16384 of 4096 126, 143; but 16384 of 4096 93, 86 and 8192 of
  // 8192 96, 93).
  const int all = teams * ctas;
  q.stages = all <= 2 && 2 * all * q.stage_bytes <= 64 * 1024 ? 3 : 2;
  const auto whole = [](const void* q, int64_t ld) { return (reinterpret_cast<uintptr_t>(q) | ld * sizeof(float)) % 32 == 0; };
  q.whole_sum = whole(p.sum, p.ld_sum), q.whole_y = whole(p.y, p.ldy);
  const int64_t most = static_cast<int64_t>(sms) * ctas, want = (static_cast<int64_t>(p.t) + teams - 1) / teams;
  static Kernel handle(kRingBytes);
  return handle.launch(block_norm_ring_kernel<T, S, V, LANES>, device, dim3(static_cast<unsigned>(std::min(most, want))),
                       teams * q.team, teams * q.stages * q.stage_bytes, 1, stream, q);
}

template <typename T, typename S, int V>
cudaError_t launch_ring(const BlockParams& p, int device, int sms, cudaStream_t stream) {
  if (p.n <= 128) return launch_teams<T, S, V, 8>(p, device, sms, stream);
  if (p.n <= 256) return launch_teams<T, S, V, 16>(p, device, sms, stream);
  return launch_teams<T, S, V, 32>(p, device, sms, stream);
}

template <typename T, typename S>
cudaError_t launch_t(const BlockParams& p, bool vector, int device, int sms, cudaStream_t stream) {
  const int n = p.n;
  // Rows of a CTA each start sooner, teams keep what stands beside the rows: us, bf16,
  // 153, 300 and 608 rows of 1024 values 3.3, 3.4, 6.2 and 3.4, 3.6, 3.5; of 4096 3.6,
  // 4.8, 9.0 and 4.0, 5.5, 7.8; 153 and 300 rows of 8192 9.2, 10.2 and 7.2, 8.2, of 128
  // 3.3, 3.4 and 3.1, 3.1.
  if (p.t > (n > 256 && n <= kMostThreads * 8 ? 2 : 1) * sms && n <= kRingThreads * 16)
    return vector ? launch_ring<T, S, 8>(p, device, sms, stream) : launch_ring<T, S, 1>(p, device, sms, stream);
  if (n <= kMostThreads * 8)
    return vector ? launch_rows<T, S, 8, 8>(p, device, sms, stream) : launch_rows<T, S, 1, 8>(p, device, sms, stream);
  if (n <= kMostThreads * 16 && vector) return launch_rows<T, S, 8, 16>(p, device, sms, stream);
  if (n <= kMostThreads * 32)
    return vector ? launch_rows<T, S, 8, 32>(p, device, sms, stream) : launch_rows<T, S, 1, 32>(p, device, sms, stream);
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
