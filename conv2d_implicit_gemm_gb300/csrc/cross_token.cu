// Attention to an encoder's states for few queries (single tokens above all):
// bound by the bytes of keys and values.
//
// The rows of one key head (queries x heads of its group, 16 or 32 a tile) go
// through warp-level products m16n8k16, so that each key is read once for all of
// them.  A CTA's warps take the 16-key chunks of its part of the keys in
// turns; each copies its own (cp.async, three in flight) and keeps its own running
// maximum, sum and output.  Warps are joined in shared memory.  Keys are divided
// over the CTAs of a cluster, joined over its shared memory, or, where that leaves
// SMs idle, over as many CTAs as the device holds, whose parts a second kernel
// joins; the order is always the same.
//
// The weights are rounded to the storage type before their product with the values, as
// both operands of a product have one type (their sum is taken before the rounding): the
// outputs' error against 64 bits is 1.1 to 1.4 times that of a form in 32 bits throughout,
// of one rounding of the output alone.
//
// 64 streams of one token, 20 heads of 64, up to 1500 keys: 44 us, 5.4 TB/s, 80% of the
// measured copy rate (full ones 80 us, 6.1 TB/s).  One token over 20000 keys, 8 key heads
// of 128: 20 us in 19 parts a head, of which the memory's share is 12, the start 4 and the
// join 3 (eight CTAs a head in clusters: 21.9; sixteen do not fit side by side: 30.8); one
// key head 10.2 us in 38 parts, 20.6 in a cluster.
#include <algorithm>

#include "cross.h"
#include "token_math.cuh"
#include "token_warp.cuh"

namespace oidnx {
namespace {

constexpr int kChunk = 16;  // keys of one step of a warp
constexpr int kStages = 3;  // chunks in flight and at work
constexpr int kMostSplit = 8;  // CTAs of a cluster

template <int DP, int MT> struct Tok {
  static constexpr int kWarps = DP == 256 ? 4 : 8;        // as many rings as shared memory holds
  static constexpr int kRow = DP * 2;                     // bytes of one key in shared memory
  static constexpr int kHalf = kChunk * kRow;             // bytes of the chunk's keys (or values)
  static constexpr int kPieces = DP / 8;                  // 16-byte pieces of a key
  // two CTAs an SM where registers and shared memory allow it: one starts while the other is at work
  static constexpr int kCtas = DP == 64 && MT == 1 ? 2 : 1;
  static constexpr int kWarpBytes = kStages * 2 * kHalf;  // a warp's ring
  static constexpr int kRows = 16 * MT;
  // the joined parts reuse the rings: per warp [rows][DP] fp32 and, behind all, [rows] maxima and sums
  static constexpr int kPart = kRows * DP * 4;
  static constexpr int kRing = kWarps * (kWarpBytes > kPart ? kWarpBytes : kPart);
  static constexpr int kSmem = kRing + (kWarps + 1) * kRows * 8 + 128;
};
static_assert(Tok<64, 2>::kSmem <= 227 * 1024 && Tok<128, 2>::kSmem <= 227 * 1024 && Tok<256, 1>::kSmem <= 227 * 1024, "");

// Powers of two by which the largest weight of a row stands above 1: fp16 ends
// 2^24 below 1, and many small weights next to a large one would be lost to the
// output but not to their sum.  2^15 is the largest power of two that fp16 holds.
template <typename T> constexpr float kLift = std::is_same<T, __half>::value ? 15.f : 0.f;

template <typename T, int DP, int MT>
__global__ void __launch_bounds__(Tok<DP, MT>::kWarps * 32, Tok<DP, MT>::kCtas)
    cross_token_kernel(const CrossParams p, const int split, const int parts, float* work) {
  using C = Tok<DP, MT>;
  constexpr int kWarps = C::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int ways = split * parts;
  const unsigned units = static_cast<unsigned>(p.b) * p.hk, cta = blockIdx.x / ways, tile = cta / units;
  const int unit = cta - tile * units, part = blockIdx.x - cta * ways;
  const int b = unit / p.hk, kvh = unit - b * p.hk;
  const int group = p.group;
  const int row0 = tile * C::kRows;  // of queries x group
  const int rows_all = p.tq * group;
  griddep_launch_dependents();
  griddep_wait();

  const int n = cross_kv_len(p, b), nq = cross_q_len(p, b);
  const int total = row0 < nq * group ? n : 0;
  const int chunks = (total + kChunk - 1) / kChunk;
  const int c_begin = static_cast<int>(static_cast<int64_t>(chunks) * part / ways);
  const int c_end = static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / ways);

  uint8_t* ring = smem + warp * (C::kRing / kWarps);
  const uint32_t ring_s = smem_u32(ring);
  const T* kb = static_cast<const T*>(p.k) + b * p.k_s[0] + kvh * p.k_s[2];
  const T* vb = static_cast<const T*>(p.v) + b * p.v_s[0] + kvh * p.v_s[2];
  const uint8_t* mask = p.mask ? p.mask + b * p.mask_s : nullptr;

  // chunk c -> ring stage; keys past the end and head values past d become zeros
  constexpr int PER = 32 / (C::kPieces < 32 ? C::kPieces : 32);  // keys per pass of the warp
  const int piece = lane % C::kPieces, sub = lane / C::kPieces;
  auto load = [&](int c, int stage) {
    const uint32_t at = ring_s + stage * 2 * C::kHalf;
#pragma unroll
    for (int r = 0; r < kChunk; r += PER) {
      const int key = c * kChunk + r + sub;
      const bool go = key < total && piece * 8 < p.d;
      const int64_t sl = go ? key : 0;
      const uint32_t dst = at + (r + sub) * C::kRow + ((piece ^ ((r + sub) & 7)) << 4);
      const int off = go ? piece * 8 : 0;
      cp_async16(dst, kb + sl * p.k_s[1] + off, go ? 16u : 0u);
      cp_async16(dst + C::kHalf, vb + sl * p.v_s[1] + off, go ? 16u : 0u);
    }
  };
  // which of the chunk's keys are seen: lane l looks at key l
  auto look = [&](int c) -> int {
    const int key = c * kChunk + lane;
    return lane < kChunk && key < total && (!mask || mask[key]);
  };
  int next = c_begin + warp;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (next < c_end) load(next, s);
    next += kWarps;
    cp_async_commit();
  }
  int seen = c_begin + warp < c_end ? look(c_begin + warp) : 0;

  // this thread's rows of each 16-row tile: lane / 4 and + 8
  bool asks[MT][2];
  uint32_t qf[MT][DP / 16][4];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = row0 + t * 16 + h * 8 + lane / 4;
      const int i = r / group, g = r - i * group;
      asks[t][h] = i < nq;
      const T* q = static_cast<const T*>(p.q) + b * p.q_s[0] + i * p.q_s[1] + (kvh * group + g) * p.q_s[2];
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int c = k * 16 + s * 8 + (lane % 4) * 2;
          qf[t][k][s * 2 + h] = asks[t][h] && c < p.d ? *reinterpret_cast<const uint32_t*>(q + c) : 0u;
        }
    }
  }

  float o[MT][DP / 8][4];
  float top[MT][2], sum[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
    top[t][0] = top[t][1] = -INFINITY;
    sum[t][0] = sum[t][1] = 0.f;
  }
  const float scale = p.scale * 1.4426950408889634f;

  int stage = 0;
  for (int c = c_begin + warp; c < c_end; c += kWarps) {
    cp_async_wait<kStages - 2>();
    const uint32_t bits = __ballot_sync(0xFFFFFFFFu, seen);
    {
      int s = stage + kStages - 1;
      if (s >= kStages) s -= kStages;
      if (next < c_end) load(next, s);
      next += kWarps;
      cp_async_commit();
    }
    seen = c + kWarps < c_end ? look(c + kWarps) : 0;
    const uint32_t kt = ring_s + stage * 2 * C::kHalf, vt = kt + C::kHalf;
    if (++stage == kStages) stage = 0;
    const bool whole = bits == 0xFFFFu;
    __syncwarp();
    if (!whole) {  // values that no row sees: whatever they hold, as zeros they add nothing
      uint8_t* v8 = ring + (vt - ring_s);
#pragma unroll 1
      for (int e = lane; e < kChunk * C::kPieces; e += 32)
        if (!(bits >> (e / C::kPieces) & 1u)) reinterpret_cast<uint4*>(v8)[e] = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
    }

    float sc[MT][2][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][h][e] = 0.f;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) {
      // matrices: keys 0-7 at k, k + 8; keys 8-15 at k, k + 8
      const int row = (lane & 7) + ((lane >> 4) << 3), pc = 2 * k + ((lane >> 3) & 1);
      uint32_t f[4];
      ldsm4(kt + row * C::kRow + ((pc ^ (row & 7)) << 4), f);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        mma16<T>(sc[t][0], qf[t][k], f[0], f[1]);
        mma16<T>(sc[t][1], qf[t][k], f[2], f[3]);
      }
    }

    uint32_t pf[MT][4];
    bool changed = false;
    float old[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float s[4] = {sc[t][0][2 * h] * scale, sc[t][0][2 * h + 1] * scale, sc[t][1][2 * h] * scale,
                      sc[t][1][2 * h + 1] * scale};
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(bits >> ((e >> 1) * 8 + (lane % 4) * 2 + (e & 1)) & 1u)) s[e] = -INFINITY;
        }
        float m = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        m = fmaxf(m, top[t][h]);
        const float base = m == -INFINITY ? 0.f : m;
        old[t][h] = exp2_fast(top[t][h] - base);
        changed |= m != top[t][h];
        top[t][h] = m;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = exp2_fast(s[e] - (base - kLift<T>));
        sum[t][h] = fmaf(sum[t][h], old[t][h], (s[0] + s[1]) + (s[2] + s[3]));
        pf[t][h] = pack2<T>(s[0], s[1]);
        pf[t][2 + h] = pack2<T>(s[2], s[3]);
      }
    }
    if (__any_sync(0xFFFFFFFFu, changed)) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          o[t][i][0] *= old[t][0];
          o[t][i][1] *= old[t][0];
          o[t][i][2] *= old[t][1];
          o[t][i][3] *= old[t][1];
        }
    }
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int row = lane & 15, pc = 2 * i + (lane >> 4);
      uint32_t f[4];
      ldsm4_t(vt + row * C::kRow + ((pc ^ (row & 7)) << 4), f);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        mma16<T>(o[t][2 * i], pf[t], f[0], f[1]);
        mma16<T>(o[t][2 * i + 1], pf[t], f[2], f[3]);
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();
  __syncthreads();

  // join the warps: parts [warp][row][DP], statistics [warp][row] behind the rings
  float2* stats = reinterpret_cast<float2*>(smem + C::kRing);  // (maximum, sum); [kWarps]: the CTA's
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s = sum[t][h];
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      const int r = t * 16 + h * 8 + lane / 4;
      const bool row_ok = asks[t][h];  // rows without a query see nothing
      if (lane % 4 == 0) stats[warp * C::kRows + r] = row_ok ? make_float2(top[t][h], s) : make_float2(-INFINITY, 0.f);
      float* to = reinterpret_cast<float*>(ring) + r * DP + (lane % 4) * 2;
#pragma unroll
      for (int i = 0; i < DP / 8; ++i)
        *reinterpret_cast<float2*>(to + i * 8) =
            row_ok ? make_float2(o[t][i][2 * h], o[t][i][2 * h + 1]) : make_float2(0.f, 0.f);
    }
  __syncthreads();
  const int rows = min(C::kRows, rows_all - row0);
  float* part_o = reinterpret_cast<float*>(smem);  // the first warp's part becomes the CTA's
  for (int e = threadIdx.x; e < rows * (DP / 4); e += kWarps * 32) {
    const int r = e / (DP / 4), c = e % (DP / 4);
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stats[w * C::kRows + r].x);
    const float base = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 st = stats[w * C::kRows + r];
      const float f = exp2_fast(st.x - base);
      const float4 v = *reinterpret_cast<const float4*>(smem + w * (C::kRing / kWarps) + (r * DP + c * 4) * 4);
      l = fmaf(st.y, f, l);
      acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
    }
    if (parts > 1) {  // [unit][row][part]
      float* to = work + ((static_cast<int64_t>(unit) * rows_all + row0 + r) * parts + part) * cross_part_floats(p.d);
      if (c * 4 < p.d) *reinterpret_cast<float4*>(to + kPartValues + c * 4) = acc;
      if (c == 0) *reinterpret_cast<float2*>(to) = make_float2(m, l);
      continue;
    }
    *reinterpret_cast<float4*>(part_o + r * DP + c * 4) = acc;
    if (c == 0) stats[kWarps * C::kRows + r] = make_float2(m, l);
  }
  if (parts > 1) return;
  if (split > 1) cluster_sync();
  else __syncthreads();

  // join the CTAs: each writes its share of the rows' values, eight at a time
  const int items = rows * (p.d / 8);
  for (int e = rank * kWarps * 32 + threadIdx.x; e < items; e += split * kWarps * 32) {
    const int r = e / (p.d / 8), c = e % (p.d / 8);
    const float* at = part_o + r * DP + c * 8;
    const float2* st_at = &stats[kWarps * C::kRows + r];
    // every part's loads before the first use (a remote load takes 0.7 us)
    float m = -INFINITY;
    float2 st[kMostSplit];
#pragma unroll
    for (int s = 0; s < kMostSplit; ++s) {
      st[s] = make_float2(-INFINITY, 0.f);
      if (s >= split) continue;
      if (split > 1) {
        const uint32_t sa = map_to_rank(st_at, s);
        st[s].x = ld_cluster_f32(sa), st[s].y = ld_cluster_f32(sa + 4);
      } else {
        st[s] = *st_at;
      }
    }
#pragma unroll
    for (int s = 0; s < kMostSplit; ++s) m = fmaxf(m, st[s].x);
    const float base = m == -INFINITY ? 0.f : m;
    float acc[8] = {}, l = 0.f;
    float4 u[kMostSplit], v[kMostSplit];
#pragma unroll
    for (int s = 0; s < kMostSplit; ++s) {
      u[s] = v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s >= split) continue;
      if (split > 1) {
        const uint32_t oa = map_to_rank(at, s);
        u[s] = ld_cluster_f4(oa), v[s] = ld_cluster_f4(oa + 16);
      } else {
        u[s] = *reinterpret_cast<const float4*>(at), v[s] = *reinterpret_cast<const float4*>(at + 4);
      }
    }
#pragma unroll
    for (int s = 0; s < kMostSplit; ++s) {
      const float f = exp2_fast(st[s].x - base);
      l = fmaf(st[s].y, f, l);
      acc[0] = fmaf(u[s].x, f, acc[0]), acc[1] = fmaf(u[s].y, f, acc[1]);
      acc[2] = fmaf(u[s].z, f, acc[2]), acc[3] = fmaf(u[s].w, f, acc[3]);
      acc[4] = fmaf(v[s].x, f, acc[4]), acc[5] = fmaf(v[s].y, f, acc[5]);
      acc[6] = fmaf(v[s].z, f, acc[6]), acc[7] = fmaf(v[s].w, f, acc[7]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing seen: zeros
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= inv;
    const int i = (row0 + r) / group, h = kvh * group + (row0 + r) % group;
    *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + b * p.o_s[0] + i * p.o_s[1] + h * p.o_s[2] + c * 8) =
        Vec16<T>::pack(acc);
    if (p.lse && c == 0)
      p.lse[(static_cast<int64_t>(b) * p.hq + h) * p.tq + i] =
          l == 0.f ? -INFINITY : (m - kLift<T> + log2f(l)) * 0.69314718055994531f;
  }
  if (split > 1) cluster_sync();  // a part stays until everyone has read it
}

// The parts of a row, joined by a CTA: eight values a thread, as many threads for a
// piece as there are parts to share among them, so that all loads are in flight.
constexpr int kJoinThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) cross_join_kernel(const CrossParams p, const int parts, const float* work) {
  __shared__ float top[kJoinThreads / 32];
  __shared__ __align__(16) float sums[kJoinThreads][12];  // l and eight values
  const int tid = threadIdx.x;
  const int rows = p.tq * p.group, unit = blockIdx.x / rows, row = blockIdx.x - unit * rows;
  const int size = cross_part_floats(p.d), pieces = p.d / 8, sharing = kJoinThreads / pieces;
  const float* at = work + static_cast<int64_t>(blockIdx.x) * parts * size;
  griddep_launch_dependents();
  griddep_wait();
  float m = -INFINITY;
  for (int s = tid; s < parts; s += kJoinThreads) m = fmaxf(m, at[s * size]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
  if ((tid & 31) == 0) top[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) m = fmaxf(m, top[i]);
  const float base = m == -INFINITY ? 0.f : m;
  const int c = tid % pieces, first = tid / pieces;
  float acc[8] = {}, l = 0.f;
  if (first < sharing) {
#pragma unroll 4
    for (int s = first; s < parts; s += sharing) {
      const float2 st = *reinterpret_cast<const float2*>(at + s * size);
      const float4 u = *reinterpret_cast<const float4*>(at + s * size + kPartValues + c * 8);
      const float4 v = *reinterpret_cast<const float4*>(at + s * size + kPartValues + 4 + c * 8);
      const float f = exp2_fast(st.x - base);
      l = fmaf(st.y, f, l);
      acc[0] = fmaf(u.x, f, acc[0]), acc[1] = fmaf(u.y, f, acc[1]);
      acc[2] = fmaf(u.z, f, acc[2]), acc[3] = fmaf(u.w, f, acc[3]);
      acc[4] = fmaf(v.x, f, acc[4]), acc[5] = fmaf(v.y, f, acc[5]);
      acc[6] = fmaf(v.z, f, acc[6]), acc[7] = fmaf(v.w, f, acc[7]);
    }
  }
  sums[tid][0] = l;
  *reinterpret_cast<float4*>(&sums[tid][4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  *reinterpret_cast<float4*>(&sums[tid][8]) = make_float4(acc[4], acc[5], acc[6], acc[7]);
  __syncthreads();
  if (tid >= pieces) return;
  for (int i = 1; i < sharing; ++i) {
    const float* other = sums[tid + i * pieces];
    l += other[0];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += other[4 + k];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] *= inv;
  const int b = unit / p.hk, i = row / p.group, h = (unit - b * p.hk) * p.group + row - i * p.group;
  *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + b * p.o_s[0] + i * p.o_s[1] + h * p.o_s[2] + c * 8) = Vec16<T>::pack(acc);
  if (p.lse && tid == 0)
    p.lse[(static_cast<int64_t>(b) * p.hq + h) * p.tq + i] =
        l == 0.f ? -INFINITY : (m - kLift<T> + log2f(l)) * 0.69314718055994531f;
}

// slots: only count the CTAs that the device holds at once.
template <typename T, int DP, int MT>
cudaError_t launch(const CrossParams& p, int split, int parts, float* work, int device, cudaStream_t stream, int* slots) {
  using C = Tok<DP, MT>;
  auto kernel = cross_token_kernel<T, DP, MT>;
  static Kernel handle;
  if (slots) {
    *slots = handle.clusters(kernel, device, C::kWarps * 32, C::kSmem, split) * split;
    return cudaSuccess;
  }
  const int64_t ctas = static_cast<int64_t>(p.b) * p.hk * split * parts * ((p.tq * p.group + C::kRows - 1) / C::kRows);
  return handle.launch(kernel, device, dim3(static_cast<unsigned>(ctas)), C::kWarps * 32, C::kSmem, split, stream, p, split, parts, work);
}

template <typename T>
cudaError_t launch_t(const CrossParams& p, int split, int parts, float* work, int device, cudaStream_t stream, int* slots) {
  const bool two = p.tq * p.group > 16;
  if (p.d <= 64)
    return two ? launch<T, 64, 2>(p, split, parts, work, device, stream, slots)
               : launch<T, 64, 1>(p, split, parts, work, device, stream, slots);
  if (p.d <= 128)
    return two ? launch<T, 128, 2>(p, split, parts, work, device, stream, slots)
               : launch<T, 128, 1>(p, split, parts, work, device, stream, slots);
  return launch<T, 256, 1>(p, split, parts, work, device, stream, slots);
}

template <typename T> cudaError_t launch_both(const CrossTokenLaunch& L, cudaStream_t stream) {
  const cudaError_t e = launch_t<T>(L.p, L.split, L.parts, L.work, L.device, stream, nullptr);
  if (e != cudaSuccess || L.parts == 1) return e;
  static Kernel handle;
  const int64_t rows = static_cast<int64_t>(L.p.b) * L.p.hk * L.p.tq * L.p.group;
  return handle.launch(cross_join_kernel<T>, L.device, dim3(static_cast<unsigned>(rows)), kJoinThreads, 0, 1, stream, L.p,
                       L.parts, static_cast<const float*>(L.work));
}

}  // namespace

cudaError_t launch_cross_token(const CrossTokenLaunch& L, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_both<__nv_bfloat16>(L, stream) : launch_both<__half>(L, stream);
}

int cross_token_slots(const CrossParams& p, bool bf16, int split, int device) {
  int slots = 0;
  bf16 ? launch_t<__nv_bfloat16>(p, split, 1, nullptr, device, nullptr, &slots)
       : launch_t<__half>(p, split, 1, nullptr, device, nullptr, &slots);
  return slots;
}

}  // namespace oidnx
