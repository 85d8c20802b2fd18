// Attention to an encoder's states: what its host side and its two forms share.
#pragma once

#include "token.h"

namespace oidnx {

// Strides in elements: sequence, token, head.
struct CrossParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;             // [b][hq][tq] or null
  const int* q_lens;      // [b] or null: tq
  const int* kv_lens;     // [b] or null: kv
  const uint8_t* mask;    // [b][kv] or null
  int64_t mask_s;
  int64_t q_s[3], k_s[3], v_s[3], o_s[3];
  int b, tq, kv, hq, hk, d;
  int group;              // query heads a key head
  float scale;            // not 0
  int* status;
};

__device__ __forceinline__ int cross_q_len(const CrossParams& p, int b) {
  const int n = p.q_lens ? p.q_lens[b] : p.tq;
  return n < 0 ? 0 : n > p.tq ? p.tq : n;
}
__device__ __forceinline__ int cross_kv_len(const CrossParams& p, int b) {
  const int n = p.kv_lens ? p.kv_lens[b] : p.kv;
  return n < 0 ? 0 : n > p.kv ? p.kv : n;
}

// Many queries: items of `tiles` row tiles of 128 rows (queries x the group's heads).
struct CrossTileLaunch {
  CrossParams p;
  CUtensorMap map_q, map_k, map_v, map_o;
  int per;      // queries of a row tile
  int tiles;    // row tiles of an item
  int blocks;   // items of a key head
  int items;
  int whole;    // items that single CTAs take; each of the rest is divided over a cluster
  int cluster;
  int grid;
  int device;
};
constexpr int cross_most_tiles(int d) { return d <= 64 ? 4 : d <= 128 ? 2 : 1; }
cudaError_t launch_cross_tile(const CrossTileLaunch& L, bool bf16, cudaStream_t stream);
// CTAs in clusters of `cluster` that the device holds at once.
int cross_tile_slots(int d, bool bf16, int cluster, int device);

// Few queries: a CTA for each part of a key head's keys.  A part of a row: maximum, sum, six
// floats that nobody reads, and from kPartValues on d values, on 16 bytes.
constexpr int kPartValues = 8;
__host__ __device__ constexpr int cross_part_floats(int d) { return kPartValues + d; }
struct CrossTokenLaunch {
  CrossParams p;
  int split;    // CTAs of a cluster along the keys
  int parts;    // clusters along the keys; over 1: through `work` and a second kernel
  float* work;  // over 1 part: [unit][row][part][cross_part_floats(d)]
  int device;
};
cudaError_t launch_cross_token(const CrossTokenLaunch& L, bool bf16, cudaStream_t stream);
int cross_token_slots(const CrossParams& p, bool bf16, int split, int device);

// Copies of heads of d values to heads of ld values (the rest zeros), or back.
struct HeadsCopy {
  const void* from;
  void* to;
  int64_t from_s[3], to_s[3];
  int n[3];
  int d, d_to;  // values read and written of a head
  int negate;
};
cudaError_t launch_heads_copy(const HeadsCopy* copies, int count, int device, int sms, cudaStream_t stream);

}  // namespace oidnx
