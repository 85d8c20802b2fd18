// Window attention for few queries (single tokens above all): bound by the
// bytes of the cache.
//
// The query rows of one key head (queries x heads of its group, 16 or 32 of
// them) go through warp-level products m16n8k16, which are far from being
// the limit here; every key is read once for all of them.  The visible keys
// (sinks, then the window, one wrap of the ring) are numbered through and cut
// into chunks of 16; the CTAs of a cluster take contiguous parts, the eight
// warps of a CTA take turns.  A warp copies its own chunks (cp.async, three
// in flight) and keeps its own running maximum, sum and output, so that no
// barrier stands in the loop; warps are joined in shared memory at the end and
// CTAs over the cluster, always in the same order.
//
// 64 ragged streams of one token, 8 key heads of 128, window 4096: 133 us, 5.95
// TB/s, 88% of the measured copy rate.  One stream over 4100 slots: 11.6 us, where
// its 17 MB take 2.5 at that rate: the launch, the lengths, two rounds of the ring
// and the joining are latency, and eight CTAs a key head leave 88 of 152 SMs idle.
// 32768 slots, a CTA's 56 GB/s being the bound: 43 us with 1, 2 or 8 key heads.
#include <type_traits>

#include "token_math.cuh"
#include "token_warp.cuh"
#include "token.h"

namespace oidnx {
namespace {

constexpr int kWarps = 8;
constexpr int kChunk = 16;   // keys of one step of a warp
constexpr int kStages = 3;

template <int DP, int MT> struct Tok {
  static constexpr int kRow = DP * 2;                    // bytes of one key in shared memory
  static constexpr int kHalf = kChunk * kRow;            // bytes of the chunk's keys (or values)
  static constexpr int kWarpBytes = kStages * 2 * kHalf; // a warp's ring
  static constexpr int kRows = 16 * MT;
  // the joined parts reuse the rings: per warp [rows][DP] fp32 and, behind all, [rows] maxima and sums
  static constexpr int kPart = kRows * DP * 4;
  static constexpr int kRing = kWarps * (kWarpBytes > kPart ? kWarpBytes : kPart);
  static constexpr int kSmem = kRing + (kWarps + 1) * kRows * 8 + 128;
};

// Powers of two by which the largest weight of a row stands above 1: weights go
// into the second product in the storage type, and fp16 ends 2^24 below 1, so
// relative to 1 many small weights next to a large one would be lost to the
// output but not to their sum.  2^15 is the largest power of two that fp16 holds.
template <typename T> constexpr float kLift = std::is_same<T, __half>::value ? 15.f : 0.f;
// Whether a pair of 16-bit values holds an infinity or a NaN.
template <typename T> __device__ __forceinline__ bool not_finite2(uint32_t w) {
  constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}

// The visible keys of one sequence, numbered through: [0, sinks) and then the
// positions from `begin` on.
struct Keys {
  int sinks, begin, total;
  int slot0;  // slot of position `begin`
};
template <typename T, int DP, int MT>
__global__ void __launch_bounds__(kWarps * 32, 1) attn_token_kernel(const AttnParams p, const int split) {
  using C = Tok<DP, MT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / split;
  const int b = unit / p.hk, kvh = unit % p.hk;
  const int group = p.hq / p.hk;
  const int row0 = blockIdx.y * C::kRows;           // of queries x group
  const int rows_all = p.tq * group;
  griddep_launch_dependents();
  griddep_wait();

  const int n = attn_kv_len(p, b), nq = attn_q_len(p, b);
  const int pq = n - nq;  // position of query 0
  // queries of this row tile
  const int i_first = row0 / group, i_last = min(min(row0 + C::kRows, rows_all) - 1, nq * group - 1) / group;
  const int p_first = max(pq + i_first, 0), p_last = min(pq + i_last, n - 1);
  const bool any = row0 < nq * group && p_last >= 0;
  Keys K;
  K.sinks = any ? min(min(p.held_sinks, n), p_last + 1) : 0;
  K.begin = attn_ring_begin(p, n);
  if (p.window > 0) K.begin = max(K.begin, p_first - p.window + 1);
  K.total = any ? K.sinks + max(p_last + 1 - K.begin, 0) : 0;
  K.slot0 = K.begin < n ? attn_slot(p, K.begin) : 0;
  const int chunks = (K.total + kChunk - 1) / kChunk;
  const int c_begin = static_cast<int>(static_cast<int64_t>(chunks) * part / split);
  const int c_end = static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / split);

  // this thread's rows of each 16-row tile: lane / 4 and + 8
  int pos[MT][2];
  uint32_t qf[MT][DP / 16][4];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = row0 + t * 16 + h * 8 + lane / 4;
      const int i = r / group, g = r - i * group;
      pos[t][h] = i < nq ? pq + i : -1;
      const T* q = static_cast<const T*>(p.q) + b * p.q_s[0] + i * p.q_s[1] + (kvh * group + g) * p.q_s[2];
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int c = k * 16 + s * 8 + (lane % 4) * 2;
          qf[t][k][s * 2 + h] = pos[t][h] >= 0 && c < p.d ? *reinterpret_cast<const uint32_t*>(q + c) : 0u;
        }
    }
  }

  uint8_t* ring = smem + warp * (C::kRing / kWarps);
  const uint32_t ring_s = smem_u32(ring);
  const T* kb = static_cast<const T*>(p.k) + b * p.k_s[0] + kvh * p.k_s[2];
  const T* vb = static_cast<const T*>(p.v) + b * p.v_s[0] + kvh * p.v_s[2];

  // chunk c of the numbering -> ring stage; keys past the end and head values past d become zeros
  constexpr int PIECES = DP / 8;          // 16-byte pieces of a key
  constexpr int PER = 32 / PIECES;        // keys per pass of the warp
  const int piece = lane % PIECES, sub = lane / PIECES;
  auto load = [&](int c, int stage) {
    const uint32_t at = ring_s + stage * 2 * C::kHalf;
#pragma unroll
    for (int r = 0; r < kChunk; r += PER) {
      const int key = c * kChunk + r + sub;
      int slot = key;
      if (key >= K.sinks) {
        slot = K.slot0 + (key - K.sinks);
        if (slot >= p.cap) slot -= p.cap - p.held_sinks;
      }
      const bool go = key < K.total && piece * 8 < p.d;
      const int64_t sl = go ? slot : 0;
      const uint32_t dst = at + (r + sub) * C::kRow + ((piece ^ ((r + sub) & 7)) << 4);
      const int off = go ? piece * 8 : 0;
      cp_async16(dst, kb + sl * p.k_s[1] + off, go ? 16u : 0u);
      cp_async16(dst + C::kHalf, vb + sl * p.v_s[1] + off, go ? 16u : 0u);
    }
  };

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

  int next = c_begin + warp;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (next < c_end) load(next, s);
    next += kWarps;
    cp_async_commit();
  }
  int stage = 0;
  for (int c = c_begin + warp; c < c_end; c += kWarps) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    {
      int s = stage + kStages - 1;
      if (s >= kStages) s -= kStages;
      if (next < c_end) load(next, s);
      next += kWarps;
      cp_async_commit();
    }
    const uint32_t kt = ring_s + stage * 2 * C::kHalf, vt = kt + C::kHalf;
    if (++stage == kStages) stage = 0;

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

    // does every row of the tile see every key of the chunk?
    const int key0 = c * kChunk;
    const int j0 = key0 < K.sinks ? key0 : K.begin + key0 - K.sinks;
    const int j_last = K.begin + key0 + kChunk - 1 - K.sinks;
    const bool whole = key0 + kChunk <= K.total && (i_first == i_last || (j_last <= p_first && key0 >= K.sinks &&
                       (p.window == 0 || j0 > p_last - p.window)));
    auto visible = [&](int t, int h, int key) {
      const int j = key < K.sinks ? key : K.begin + key - K.sinks;
      const int q = pos[t][h];
      return key < K.total && j <= q && (p.window == 0 || j > q - p.window || j < p.sinks);
    };
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
            if (!visible(t, h, key0 + (e >> 1) * 8 + (lane % 4) * 2 + (e & 1))) s[e] = -INFINITY;
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
    // A value that is no number must not reach rows that do not see its key
    // (0 x NaN): where some row does not see all, such chunks are added value
    // by value.
    bool odd = false;
    if (!whole) {
      const uint8_t* v8 = ring + (vt - ring_s);
      for (int e = lane; e < C::kHalf / 4; e += 32) odd |= not_finite2<T>(reinterpret_cast<const uint32_t*>(v8)[e]);
      odd = __any_sync(0xFFFFFFFFu, odd);
    }
    if (!odd) {
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
    } else {
      const uint8_t* v8 = ring + (vt - ring_s);
#pragma unroll 1
      for (int key = 0; key < kChunk; ++key) {
        const int from = (lane & ~3) | ((key & 7) >> 1);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t pair = __shfl_sync(0xFFFFFFFFu, key < 8 ? pf[t][h] : pf[t][2 + h], from);
            const float2 w2 = unpack2<T>(pair);
            const float w = key & 1 ? w2.y : w2.x;
            if (visible(t, h, key0 + key)) {
#pragma unroll
              for (int i = 0; i < DP / 8; ++i) {
                const float2 v = unpack2<T>(*reinterpret_cast<const uint32_t*>(
                    v8 + key * C::kRow + ((i ^ (key & 7)) << 4) + (lane % 4) * 4));
                o[t][i][2 * h] = fmaf(w, v.x, o[t][i][2 * h]);
                o[t][i][2 * h + 1] = fmaf(w, v.y, o[t][i][2 * h + 1]);
              }
            }
          }
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
      // rows without a position (padding, before the first key) see nothing
      const bool row_ok = pos[t][h] >= 0;
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
    *reinterpret_cast<float4*>(part_o + r * DP + c * 4) = acc;
    if (c == 0) stats[kWarps * C::kRows + r] = make_float2(m, l);
  }
  if (split > 1) cluster_sync();
  else __syncthreads();

  // join the CTAs: each writes its share of the rows' values, eight at a time
  const int items = rows * (p.d / 8);
  for (int e = part * kWarps * 32 + threadIdx.x; e < items; e += split * kWarps * 32) {
    const int r = e / (p.d / 8), c = e % (p.d / 8);
    const float* at = part_o + r * DP + c * 8;
    const float2* st_at = &stats[kWarps * C::kRows + r];
    // every part's loads before the first use (a remote load takes 0.7 us)
    float2 st[8];
    float4 u[8], v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      st[s] = make_float2(-INFINITY, 0.f);
      u[s] = v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s >= split) continue;
      if (split > 1) {
        const uint32_t sa = map_to_rank(st_at, s), oa = map_to_rank(at, s);
        st[s].x = ld_cluster_f32(sa), st[s].y = ld_cluster_f32(sa + 4);
        u[s] = ld_cluster_f4(oa), v[s] = ld_cluster_f4(oa + 16);
      } else {
        st[s] = *st_at;
        u[s] = *reinterpret_cast<const float4*>(at), v[s] = *reinterpret_cast<const float4*>(at + 4);
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int s = 0; s < 8; ++s) m = fmaxf(m, st[s].x);
    const float base = m == -INFINITY ? 0.f : m;
    float acc[8] = {}, l = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
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

// slots: only count the CTAs that the device holds at once.
template <typename T, int DP, int MT>
cudaError_t launch(const AttnParams& p, int split, int device, cudaStream_t stream, int* slots) {
  using C = Tok<DP, MT>;
  auto kernel = attn_token_kernel<T, DP, MT>;
  static Kernel handle;
  if (slots) {
    *slots = handle.clusters(kernel, device, kWarps * 32, C::kSmem, split) * split;
    return cudaSuccess;
  }
  return handle.launch(kernel, device, dim3(p.b * p.hk * split, (p.tq * (p.hq / p.hk) + C::kRows - 1) / C::kRows),
                       kWarps * 32, C::kSmem, split, stream, p, split);
}

template <typename T>
cudaError_t launch_t(const AttnParams& p, int split, int device, cudaStream_t stream, int* slots) {
  const bool two = p.tq * (p.hq / p.hk) > 16;
  if (p.d <= 64)
    return two ? launch<T, 64, 2>(p, split, device, stream, slots) : launch<T, 64, 1>(p, split, device, stream, slots);
  return two ? launch<T, 128, 2>(p, split, device, stream, slots) : launch<T, 128, 1>(p, split, device, stream, slots);
}

}  // namespace

cudaError_t launch_attn_token(const AttnParams& p, bool bf16, int split, int device, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(p, split, device, stream, nullptr)
              : launch_t<__half>(p, split, device, stream, nullptr);
}

int attn_token_slots(const AttnParams& p, bool bf16, int split, int device) {
  int slots = 0;
  bf16 ? launch_t<__nv_bfloat16>(p, split, device, nullptr, &slots) : launch_t<__half>(p, split, device, nullptr, &slots);
  return slots;
}

}  // namespace oidnx
