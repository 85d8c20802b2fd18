// What the prompt forms of window attention share: a CTA's plan over row and
// key tiles, and small helpers.
#pragma once

#include <type_traits>

#include "attn_row.cuh"
#include "token_ptx.cuh"
#include "token.h"

namespace oidnx {

constexpr int kTileKeys = 128;
constexpr int kHalf = kTileKeys / 2;

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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Value operand: rows of 64 values (128 bytes, swizzled) a key, 8 keys 1024
// bytes apart, 64-value blocks 16384 bytes apart; values contiguous (N-major).
// An operand's descriptors differ in their start address only (16-byte units in
// the low bits, which do not overflow), so the issuing thread adds constants.
__device__ __forceinline__ uint64_t value_desc(uint32_t saddr) {
  return smem_desc_sw128(saddr) | (static_cast<uint64_t>(16384u >> 4) << 16);
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(src))
               : "memory");
}

// sum + 0 v of pairs: zeros of either sign while every v is a number.
template <typename T> __device__ __forceinline__ uint32_t add_nulls(uint32_t sum, uint32_t v) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0u), "r"(sum));
  else
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0u), "r"(sum));
  return r;
}

// One warp: looks over the values of a tile that some row does not see whole.
// Clears what is no number past the last key; true where a key has such a value.
template <typename T, int DB> __device__ __forceinline__ bool look_over(uint8_t* V, int count, int lane) {
  const int pieces = (count + 15) / 16 * 16 * 8;  // of a 64-value block
  // 0 x v is NaN where v is none: a sum of them tells in one instruction a pair
  uint32_t sum[2] = {0u, 0u};
#pragma unroll 8
  for (int e = lane; e < pieces * DB; e += 32) {
    const int block = e / pieces;  // any order of a row's pieces will do
    const uint4 v = *reinterpret_cast<const uint4*>(V + block * 16384 + (e - block * pieces) * 16);
    sum[0] = add_nulls<T>(add_nulls<T>(sum[0], v.x), v.y);
    sum[1] = add_nulls<T>(add_nulls<T>(sum[1], v.z), v.w);
  }
  bool found = false;
  if (__any_sync(0xFFFFFFFFu, (sum[0] | sum[1]) & 0x7FFF7FFFu)) {
    for (int e = lane; e < pieces * DB; e += 32) {
      const int block = e / pieces, r = (e - block * pieces) / 8;
      uint4* at = reinterpret_cast<uint4*>(V + block * 16384 + (e - block * pieces) * 16);
      const uint4 v = *at;
      if ((add_nulls<T>(add_nulls<T>(0u, v.x), v.y) | add_nulls<T>(add_nulls<T>(0u, v.z), v.w)) & 0x7FFF7FFFu) {
        if (r >= count) *at = make_uint4(0u, 0u, 0u, 0u);
        else found = true;
      }
    }
  }
  return found;
}

// Powers of two by which weights stand above what the running maximum says: fp16
// ends 2^24 below 1, and many small weights next to a large one would be lost to
// the output but not to their sum.  With the 2^8 that a weight may be above 1
// before the maximum follows, 2^15 is the largest power of two that fp16 holds.
template <typename T> constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;

struct Tile {
  int slot, pos, count;
};

__device__ __forceinline__ int keys_of_half(int count, int h) { return min(max(count - h * kHalf, 0), kHalf); }

// The lowest n of 32 bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// What a CTA works on; every role computes the same.
struct Plan {
  int b, kvh, group, per;  // per: queries of a row tile
  int n, nq, pq;           // keys written, queries, position of query 0
  int i00, min0, max0, min1, max1;  // first query; first and last position of each row tile (last < first: no row)
  int sinks, n_sinks;                  // keys and tiles of the sinks' run
  int begin, slot0, len_a, n_a, len_b; // the window: up to the ring's end, and from its start on
  int tiles;
  int plain_lo, plain_hi;  // tiles of 128 keys that every row of both row tiles sees whole, as far as they are in one run

  __device__ __forceinline__ bool plain(int j) const { return j >= plain_lo && j < plain_hi; }
  __device__ __forceinline__ Tile tile(const AttnParams& p, int j) const {
    Tile t;
    if (j < n_sinks) {
      t.slot = t.pos = j * kTileKeys;
      t.count = min(kTileKeys, sinks - t.pos);
    } else if (j < n_sinks + n_a) {
      const int o = (j - n_sinks) * kTileKeys;
      t.slot = slot0 + o, t.pos = begin + o, t.count = min(kTileKeys, len_a - o);
    } else {
      const int o = (j - n_sinks - n_a) * kTileKeys;
      t.slot = p.held_sinks + o, t.pos = begin + len_a + o, t.count = min(kTileKeys, len_b - o);
    }
    return t;
  }
  // query index, and whether row tile t has a row that sees anything
  __device__ __forceinline__ int i0(int t) const { return i00 + t * per; }
  __device__ __forceinline__ bool active(int t) const { return t ? max1 >= min1 : max0 >= min0; }
  // Does some row of tile t see some key of the tile; does every row see every key?
  __device__ __forceinline__ bool seen(const AttnParams& p, int t, const Tile& k) const {
    const int lo = t ? min1 : min0, hi = t ? max1 : max0;
    return hi >= lo && k.pos <= hi && (p.window == 0 || k.pos + k.count - 1 > lo - p.window || k.pos < p.sinks);
  }
  __device__ __forceinline__ bool whole(const AttnParams& p, int t, const Tile& k) const {
    const int lo = t ? min1 : min0, hi = t ? max1 : max0;
    return k.count == kTileKeys && k.pos + k.count - 1 <= lo &&
           (p.window == 0 || k.pos > hi - p.window || k.pos + k.count <= p.sinks);
  }
  __device__ __forceinline__ bool looked_over(const AttnParams& p, const Tile& k) const {
    return (seen(p, 0, k) && !whole(p, 0, k)) || (seen(p, 1, k) && !whole(p, 1, k));
  }
};

__device__ __forceinline__ Plan make_plan(const AttnParams& p) {
  Plan w;
  // row tiles from the last to the first (causal: the longest first), the heads of one next to each other
  const unsigned heads = p.b * p.hk, from_last = blockIdx.x / heads, unit = blockIdx.x - from_last * heads;
  const int rows = p.pairs - 1 - static_cast<int>(from_last);
  w.b = unit / static_cast<unsigned>(p.hk), w.kvh = unit - w.b * p.hk;
  w.group = p.group;
  w.per = p.per;
  w.n = attn_kv_len(p, w.b), w.nq = attn_q_len(p, w.b);
  w.pq = w.n - w.nq;
  w.i00 = 2 * rows * w.per;
  // a tile without queries, or all before the first key: last < first
  w.min0 = max(w.pq + w.i00, 0);
  w.max0 = w.pq + min(w.i00 + w.per, w.nq) - 1;
  w.min1 = max(w.pq + w.i00 + w.per, 0);
  w.max1 = w.pq + min(w.i00 + 2 * w.per, w.nq) - 1;
  const bool on0 = w.active(0), on1 = w.active(1);
  const int lo = on0 ? w.min0 : w.min1, hi = on1 ? w.max1 : on0 ? w.max0 : -1;
  w.sinks = w.n_sinks = w.begin = w.slot0 = w.len_a = w.n_a = w.len_b = w.tiles = w.plain_lo = w.plain_hi = 0;
  if (hi < 0) return w;
  w.sinks = min(min(p.held_sinks, w.n), hi + 1);
  w.begin = attn_ring_begin(p, w.n);
  if (p.window > 0) w.begin = max(w.begin, lo - p.window + 1);
  int len = max(hi + 1 - w.begin, 0);
  if (len == 0) w.begin = 0;
  w.slot0 = len ? attn_slot(p, w.begin) : 0;
  if (len && w.begin == w.sinks && w.slot0 == w.sinks) {  // one run from the first key on
    w.begin = w.slot0 = 0;
    len += w.sinks;
    w.sinks = 0;
  }
  w.len_a = min(len, p.cap - w.slot0);
  w.len_b = len - w.len_a;
  w.n_sinks = (w.sinks + kTileKeys - 1) / kTileKeys;
  w.n_a = (w.len_a + kTileKeys - 1) / kTileKeys;
  w.tiles = w.n_sinks + w.n_a + (w.len_b + kTileKeys - 1) / kTileKeys;
  // whole: the last key at or before the first row's position, the first key in
  // the last row's window
  const int past = p.window > 0 ? hi - p.window - w.begin : -1;
  const int room = lo + 1 - w.begin;
  w.plain_lo = w.n_sinks + (past >= 0 ? past / kTileKeys + 1 : 0);
  w.plain_hi = w.n_sinks + min(w.len_a, max(room, 0)) / kTileKeys;
  return w;
}

}  // namespace oidnx
