// Attention to an encoder's states for many queries, on the 5th-generation tensor
// cores.
//
// A CTA takes items: row tiles of 128 query rows of one key head (queries x the
// heads of its group, query-major), four of them for heads of up to 64 values, two
// up to 128, one up to 256, which share each tile of keys and values that the CTA
// loads.
//
//   S = Q K^T (tcgen05, accumulators in tensor memory), softmax in registers (one
//   thread a row), P in 16 bits over S in tensor memory, O += P V with P as the
//   tensor-memory operand and V read as it lies (values contiguous).
//
//  * Keys in units of 64: 64 columns of scores each, two units in turn for a row
//    tile (one where four row tiles fill the tensor memory), so that the tensor
//    cores make one's scores while the softmax warps are at another's.
//  * The running maximum that P is relative to follows the true one only when it
//    falls more than 2^8 behind, so O is rescaled rarely; P <= 2^8 (fp16: 2^15, to
//    keep the small ones) stays within 16 bits and the sums are fp32.
//  * P is rounded to the storage type, as both operands of a product have one type;
//    the sum of the weights is taken before the rounding.
//  * Which keys are seen does not depend on the row: scores of others are replaced,
//    and a warp clears their values in shared memory (0 x NaN) before the product.
//  * CTAs stay, and take the next item's queries under the last one's end.  What
//    does not fill a round of CTAs is divided: a cluster takes an item, each CTA a
//    part of its keys, and the parts are joined over distributed shared memory.
//
// Heads of over 64 values are bound by the tensor cores: for 64 keys the operands of a
// row tile's two products take 640 cycles through shared memory (its queries are read
// again for each unit), two tiles 1280 of some 1500, and a long run lowers the clock:
// 8160 queries and keys, 16 heads of 128, 361 us in a graph, 1510 TFLOP/s, and 388 in a
// long run of calls, at 1410; 398 without the last round divided, 392 of them with all of
// the softmax's arithmetic left out.  Stages handed back by the softmax warps instead of
// the issuing threads: 423.  2040 x 2040, 4 heads of 256: 39 us (47).
// Heads of up to 64 are bound by the chain from scores to weights to the next scores,
// four of which share an SM's issue slots: 8160 x 8160, 16 heads of 64, 326 us, 840
// TFLOP/s (276 without the softmax's arithmetic).  Four row tiles of 8160 queries to 77
// keys, 4 x 16 heads of 64: 38 us, of which 5 are a CTA's start and 3.7 each of seven
// items, 5.3 TB/s.  Not kept: weights in columns of their own, with the next scores made
// under the softmax, for three tiles (431 us); one issuing thread for four tiles (477);
// two tiles of two buffers (403); outputs sent off by a warp of their own (text 43); both
// units of a short text at once (no faster).
//
// Warps 4 t .. 4 t + 3: softmax of row tile t, rescaling, output; then a warp that
// loads (TMA), one or two that issue the products, one that clears values.
#include "attn_prompt.cuh"
#include "cross.h"

namespace oidnx {
namespace {

constexpr int kUnit = 64;  // keys

// DB: 64-value blocks of a head.
template <int DB> struct Shape {
  static constexpr int NT = DB == 1 ? 4 : DB == 2 ? 2 : 1;  // row tiles
  static constexpr int SB = DB == 1 ? 1 : 2;                // score buffers of a row tile
  static constexpr int UPS = DB == 4 ? 1 : 2;               // units of a stage
  static constexpr int NS = DB == 1 ? 3 : 2;                // stages of keys and of values
  static constexpr int QB = DB == 1 ? 2 : 1;                // buffers of queries; with two the output takes its own queries' place
  static constexpr int NM = DB == 4 ? 1 : 2;                // issuing warps
  static constexpr int TPW = NT / NM;                       // row tiles of one
  static constexpr bool kGives = TPW == 1;                  // it hands the stages back itself (commits); else the softmax warps do
  static constexpr int kBlock = UPS * kUnit * 128;          // bytes of a stage's 64-value block
  static constexpr int kStage = DB * kBlock;
  static constexpr int kQTile = DB * 16384;
  static constexpr int kSoftWarps = 4 * NT;
  static constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kLoadWarp + 1, kLookWarp = kMmaWarp + NM;
  static constexpr int kThreads = (kLookWarp + 1) * 32;
  static constexpr int kOut = 16384;  // a row tile's 64 values on their way out
  static constexpr int kSmem = QB * NT * kQTile + 2 * NS * kStage + (QB == 1 ? NT * kOut : 0) + 1024 + 512;
};
static_assert(Shape<1>::kSmem <= 227 * 1024 && Shape<2>::kSmem <= 227 * 1024 && Shape<4>::kSmem <= 227 * 1024, "");
// the parts of a divided item, [row][value] in fp32, take the operands' place (with two
// buffers of queries theirs alone: their statistics stand where values were)
template <int DB> constexpr int kParts = Shape<DB>::NT * 128 * DB * 64 * 4;
static_assert(kParts<1> <= Shape<1>::QB * Shape<1>::NT * Shape<1>::kQTile, "");
static_assert(kParts<2> <= 2 * Shape<2>::kQTile + 4 * Shape<2>::kStage && kParts<4> <= Shape<4>::kQTile + 4 * Shape<4>::kStage, "");

struct TileParams : CrossParams {
  int per;      // queries of a row tile
  int tiles;    // row tiles of an item
  int blocks;   // items of a key head
  int items, whole, cluster;
  int step_block, step_kvh, step_b;  // from an item to the grid's size behind it
};

// One item, or a part of its keys; every role computes the same.
struct Work {
  int b, kvh, i0;       // first query
  int n, nq;            // keys, queries of the sequence
  int u0, units;        // units of keys
  bool part;
};

// The items of a CTA: blockIdx.x and every gridDim.x-th from there, by steps (a
// division takes 400 cycles), then its part of a divided one.
template <int DB> struct Schedule {
  const TileParams& p;
  int next, block, kvh, b;
  int n, nq;  // of the next item's sequence, on their way
  bool tail;
  __device__ __forceinline__ Schedule(const TileParams& p_) : p(p_), next(blockIdx.x), tail(true) {
    if (next >= p.whole) {
      next = p.whole + blockIdx.x / p.cluster;
      tail = next < p.items;
    }
    locate();
  }
  __device__ __forceinline__ void locate() {
    const int unit = next / p.blocks;
    block = next - unit * p.blocks;
    b = unit / p.hk, kvh = unit - b * p.hk;
    if (b >= p.b) b = 0;  // (no item: its lengths are not used)
  }
  __device__ __forceinline__ void lengths() { n = cross_kv_len(p, b), nq = cross_q_len(p, b); }
  __device__ __forceinline__ bool take(Work& w) {
    const bool whole = next < p.whole;
    if (!whole && !tail) return false;
    w.b = b, w.kvh = kvh, w.i0 = block * p.tiles * p.per;
    w.n = n, w.nq = nq;
    w.u0 = 0;
    w.units = w.i0 < nq ? (n + kUnit - 1) / kUnit : 0;
    w.part = !whole && p.cluster > 1;
    if (w.part) {  // whole stages of them
      constexpr int KT = Shape<DB>::UPS * kUnit;
      const int part = blockIdx.x % p.cluster;
      const int64_t tiles = w.i0 < nq ? (n + KT - 1) / KT : 0;
      w.u0 = static_cast<int>(tiles * part / p.cluster) * Shape<DB>::UPS;
      w.units = min(static_cast<int>(tiles * (part + 1) / p.cluster) * Shape<DB>::UPS, w.units) - w.u0;
    }
    if (!whole) {
      tail = false;
      return true;
    }
    next += gridDim.x;
    if (next < p.whole) {
      block += p.step_block;
      kvh += p.step_kvh, b += p.step_b;
      if (block >= p.blocks) block -= p.blocks, ++kvh;
      if (kvh >= p.hk) kvh -= p.hk, ++b;
    } else {
      next = p.whole + blockIdx.x / p.cluster;
      tail = next < p.items;
      locate();
    }
    lengths();
    return true;
  }
};

__device__ __forceinline__ uint64_t block_desc(uint32_t saddr, uint32_t block) {  // value operand, as value_desc
  return smem_desc_sw128(saddr) | (static_cast<uint64_t>(block >> 4) << 16);
}

template <typename T, int DB>
__global__ void __launch_bounds__(Shape<DB>::kThreads, 1)
    cross_tile_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                      const __grid_constant__ TileParams p) {
  using C = Shape<DB>;
  constexpr int NT = C::NT, SB = C::SB, UPS = C::UPS, NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  constexpr int QB = C::QB;
  uint8_t* Q = smem_raw + pad;  // [QB][NT]
  uint8_t* Ks = Q + QB * NT * C::kQTile;
  uint8_t* Vs = Ks + NS * C::kStage;
  uint8_t* Out = Vs + NS * C::kStage;  // [NT], where it has a place of its own
  // [NT][128]: maximum and sum of a part, once nothing comes or goes any more
  float2* stats = reinterpret_cast<float2*>(QB == 1 ? Out : Vs);
  uint64_t* qfull = reinterpret_cast<uint64_t*>(Out + (QB == 1 ? NT * C::kOut : 0));  // [QB][NT]
  uint64_t* qempty = qfull + QB * NT;
  uint64_t* kfull = qempty + QB * NT;  // [NS]
  uint64_t* kempty = kfull + NS;
  uint64_t* vfull = kempty + NS;
  uint64_t* vempty = vfull + NS;
  uint64_t* vclean = vempty + NS;
  uint64_t* sfull = vclean + NS;       // [NT][SB]
  uint64_t* pfull = sfull + NT * SB;   // the same
  uint64_t* odone = pfull + NT * SB;   // [NT]
  uint64_t* plast = odone + NT;        // [NT]
  uint32_t* slot = reinterpret_cast<uint32_t*>(plast + NT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], p.tiles);
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], p.tiles + 1);  // and the clearing warp
      mbar_init(&vclean[s], 32);
    }
    for (int t = 0; t < QB * NT; ++t) {
      mbar_init(&qfull[t], 1);
      mbar_init(&qempty[t], 1);
    }
    for (int t = 0; t < NT; ++t) {
      mbar_init(&odone[t], 1);
      mbar_init(&plast[t], 1);
    }
    for (int c = 0; c < NT * SB; ++c) {
      mbar_init(&sfull[c], 1);
      mbar_init(&pfull[c], 128);
    }
    fence_mbarrier_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(slot, 512);
  if (warp == C::kLoadWarp && lane < 4) prefetch_tmap(lane == 0 ? &map_k : lane == 1 ? &map_q : lane == 2 ? &map_v : &map_o);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  Work w;
  Schedule<DB> work(p);
  griddep_launch_dependents();
  griddep_wait();
  work.lengths();
  const int kd = (p.d + 15) / 16;  // blocks of 16 values of a head
  // columns: S (then P) of the row tiles' buffers, O of the row tiles
  const auto s_col = [tmem](int t, int c) { return tmem + (t * SB + c) * 64; };
  const auto o_col = [tmem](int t) { return tmem + NT * SB * 64 + t * 64 * DB; };
  // a stage's use count gives its phase: tile g of all that the CTA takes is in stage g % NS
  const bool masked = p.mask != nullptr;
  bool ok = true;
  // of a softmax thread, after its last item
  float top = -INFINITY, sum = 0.f;
  bool valid = false;

  if (warp == C::kLoadWarp) {
    if (lane == 0) {
      const uint64_t pol = l2_evict_normal();
      const int q_bytes = p.per * p.group * 128;
      int s = 0, ph = 0, round = 0;
      const auto queries = [&](const Work& q) {  // the round'th item's
        const int at = round % QB * NT, phase = round / QB & 1;
        for (int t = 0; t < p.tiles && ok; ++t) {
          ok = mbar_wait_soon(&qempty[at + t], phase ^ 1, p.status, kErrTimeoutProducer);
          if (!ok) break;
          mbar_arrive_expect_tx(&qfull[at + t], DB * q_bytes);
#pragma unroll
          for (int d = 0; d < DB; ++d)
            tma_load_4d(Q + (at + t) * C::kQTile + d * 16384, &map_q, &qfull[at + t], d * 64, q.kvh * p.group, q.i0 + t * p.per,
                        p.q_s[0] ? q.b : 0, pol);
        }
        ++round;
      };
      const auto next_with_keys = [&](Work& q) {
        while (work.take(q))
          if (q.units > 0) return true;
        return false;
      };
      bool more = next_with_keys(w), first = true;
      while (ok && more) {
        const int tiles = (w.units + UPS - 1) / UPS;
        Work after;
        bool another = false;
        for (int j = 0; j < tiles && ok; ++j) {
          const int key = (w.u0 + j * UPS) * kUnit;
          ok = mbar_wait_soon(&kempty[s], ph ^ 1, p.status, kErrTimeoutProducer);
          if (!ok) break;
          mbar_arrive_expect_tx(&kfull[s], C::kStage);
#pragma unroll
          for (int d = 0; d < DB; ++d)
            tma_load_4d(Ks + s * C::kStage + d * C::kBlock, &map_k, &kfull[s], d * 64, key, p.k_s[2] ? w.kvh : 0,
                        p.k_s[0] ? w.b : 0, pol);
          if ((QB == 1 || first) && j == 0) queries(w);
          if (!ok) break;
          ok = mbar_wait_soon(&vempty[s], ph ^ 1, p.status, kErrTimeoutProducer);
          if (!ok) break;
          mbar_arrive_expect_tx(&vfull[s], C::kStage);
#pragma unroll
          for (int d = 0; d < DB; ++d)
            tma_load_4d(Vs + s * C::kStage + d * C::kBlock, &map_v, &vfull[s], d * 64, key, p.v_s[2] ? w.kvh : 0,
                        p.v_s[0] ? w.b : 0, pol);
          if (++s == NS) s = 0, ph ^= 1;
        }
        if (!ok) break;
        another = next_with_keys(after);
        if (QB == 2 && another) queries(after);
        w = after, more = another, first = false;
      }
    }
  } else if (warp >= C::kMmaWarp && warp < C::kLookWarp) {
    // The thread only issues: a commit covers all its earlier products, so the
    // scores of unit u + SB landing tells that P V of unit u is done.
    const int t0 = (warp - C::kMmaWarp) * C::TPW, t1 = min(t0 + C::TPW, p.tiles);
    if (t0 < t1 && elect_one()) {
      constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
      const uint32_t id_s = idesc_16(bf, 128, kUnit), id_pv = idesc_16(bf, 128, kd * 16, true);
      const uint64_t q0 = smem_desc_sw128(smem_u32(Q)), k0 = smem_desc_sw128(smem_u32(Ks));
      const uint64_t v0 = block_desc(smem_u32(Vs), C::kBlock);
      int g = 0;             // tiles before this item, and their stages and phases
      int round = 0;
      uint32_t phase = 0;    // of the weights' barriers, a bit each
      uint32_t clean = 0;    // of the cleared stages'
      const auto stage_of = [](int g) { return g % NS; };
      const auto phase_of = [](int g) { return (g / NS) & 1; };
      const auto score = [&](int t, int u, int keys, int stage, uint32_t to) {  // S of unit u
        const uint32_t id = keys == kUnit ? id_s : idesc_16(bf, 128, (keys + 15) / 16 * 16);
        const uint64_t qd = q0 + (round % QB * NT + t) * (C::kQTile >> 4);
        const uint64_t kt = k0 + stage * (C::kStage >> 4) + (u % UPS) * (kUnit * 128 >> 4);
#pragma unroll
        for (int i = 0; i < 4 * DB; ++i)
          if (i < kd)
            mma_f16_ss(to, qd + (((i >> 2) * 16384 + (i & 3) * 32) >> 4),
                       kt + (((i >> 2) * C::kBlock + (i & 3) * 32) >> 4), id, i > 0);
      };
      while (ok && work.take(w)) {
        if (w.units <= 0) continue;
        const int U = w.units;
        const int left = w.n - w.u0 * kUnit;  // keys from the first unit on
        for (int u = 0; u < SB && u < U && ok; ++u) {
          if (u % UPS == 0) ok = mbar_wait_soon(&kfull[stage_of(g + u / UPS)], phase_of(g + u / UPS), p.status, kErrTimeoutMma);
          for (int t = t0; t < t1 && ok; ++t) {
            if (u == 0) ok = mbar_wait_soon(&qfull[round % QB * NT + t], round / QB & 1, p.status, kErrTimeoutMma);
            if (!ok) break;
            tc_fence_after();
            score(t, u, min(left - u * kUnit, kUnit), stage_of(g + u / UPS), s_col(t, u % SB));
            mma_commit(&sfull[t * SB + u % SB]);
            if (C::kGives && (u % UPS == UPS - 1 || u == U - 1)) mma_commit(&kempty[stage_of(g + u / UPS)]);
          }
        }
        for (int u = 0; u < U && ok; ++u) {
          const int gu = g + u / UPS, s = stage_of(gu), nu = u + SB;
          if (u % UPS == 0) {
            ok = mbar_wait_soon(&vfull[s], phase_of(gu), p.status, kErrTimeoutMma);
            if (ok && (masked || (w.n < p.kv && (u + UPS) * kUnit > left))) {
              ok = mbar_wait_soon(&vclean[s], clean >> s & 1, p.status, kErrTimeoutMma);
              clean ^= 1u << s;
            }
          }
          const int gn = g + nu / UPS;
          if (ok && nu < U && nu % UPS == 0) ok = mbar_wait_soon(&kfull[stage_of(gn)], phase_of(gn), p.status, kErrTimeoutMma);
          const uint64_t vt = v0 + s * (C::kStage >> 4) + (u % UPS) * (kUnit * 128 >> 4);
          const int steps = (min(left - u * kUnit, kUnit) + 15) / 16;
          // the row tile whose weights are there first
          const int turn = C::TPW == 2 && t1 - t0 == 2 && !mbar_test_wait(&pfull[t0 * SB + u % SB], phase >> (t0 * SB + u % SB) & 1) &&
                           mbar_test_wait(&pfull[(t0 + 1) * SB + u % SB], phase >> ((t0 + 1) * SB + u % SB) & 1);
          for (int k = t0; k < t1 && ok; ++k) {
            const int t = turn ? t0 + t1 - 1 - k : k;
            const int c = t * SB + u % SB;
            ok = mbar_wait_soon(&pfull[c], phase >> c & 1, p.status, kErrTimeoutMma);
            if (!ok) break;
            phase ^= 1u << c;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < kUnit / 16; ++i)
              if (i < steps) mma_ts(o_col(t), s_col(t, u % SB) + i * 8, vt + i * (2048 >> 4), id_pv, u > 0 || i > 0);
            if (C::kGives && (u % UPS == UPS - 1 || u == U - 1)) mma_commit(&vempty[s]);
            if (nu < U) {
              score(t, nu, min(left - nu * kUnit, kUnit), stage_of(gn), s_col(t, nu % SB));
              mma_commit(&sfull[t * SB + nu % SB]);
              if (C::kGives && (nu % UPS == UPS - 1 || nu == U - 1)) mma_commit(&kempty[stage_of(gn)]);
            } else if (SB > 1 && u + 2 == U) {
              mma_commit(&plast[t]);
            }
            if (u + 1 == U) mma_commit(&odone[t]);
          }
        }
        g += (U + UPS - 1) / UPS;
        ++round;
      }
    }
  } else if (warp == C::kLookWarp) {
    // Clears the values that no row sees; every tile is waited for and handed back,
    // so that the phases stay in step
    int s = 0, ph = 0;
    while (ok && work.take(w)) {
      if (w.units <= 0) continue;
      const int tiles = (w.units + UPS - 1) / UPS;
      for (int j = 0; j < tiles; ++j) {
        const int key = (w.u0 + j * UPS) * kUnit;
        uint32_t bits[UPS * 2];
        bool all = true;
#pragma unroll
        for (int k = 0; k < UPS * 2; ++k) {
          const int at = key + k * 32 + lane;
          bits[k] = __ballot_sync(0xFFFFFFFFu, at < w.n && (!masked || p.mask[w.b * p.mask_s + at]));
          all = all && bits[k] == 0xFFFFFFFFu;
        }
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_soon(&vfull[s], ph, p.status, kErrTimeoutProducer));
        if (!ok) break;
        if (masked || (w.n < p.kv && key + UPS * kUnit > w.n)) {
          if (!all) {
            for (int r = 0; r < UPS * kUnit; r += 4) {  // four rows of a 64-value block at a time
              const int row = r + lane / 8;
              uint32_t word = bits[0];
#pragma unroll
              for (int k = 1; k < UPS * 2; ++k) word = row / 32 == k ? bits[k] : word;
              if (!(word >> (row & 31) & 1u)) {
#pragma unroll
                for (int d = 0; d < DB; ++d)
                  *reinterpret_cast<uint4*>(Vs + s * C::kStage + d * C::kBlock + row * 128 + (lane & 7) * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
              }
            }
            fence_proxy_async_smem();
          }
          mbar_arrive(&vclean[s]);
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&vempty[s]);
        __syncwarp();
        if (++s == NS) s = 0, ph ^= 1;
      }
    }
  } else if ((warp >> 2) < p.tiles) {
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the tile = lane of tensor memory
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c = p.scale * 1.4426950408889634f;  // scores to powers of two
    const int query = t * p.per + r / p.group, head = r % p.group;  // of the row, from the item's first
    const bool row_used = r < p.per * p.group;
    uint32_t phase = 0;  // of each buffer's scores
    int g = 0, last_phase = 0, done_phase = 0;
    int round = 0;  // items with keys
    bool more = work.take(w);
    while (ok && more) {
      const int i = w.i0 + query;
      valid = row_used && i < w.nq;
      const int U = max(w.units, 0);
      top = -INFINITY;  // what P is relative to
      sum = 0.f;
      const uint8_t* mask = masked ? p.mask + w.b * p.mask_s : nullptr;
      int first = 0, second = 0;  // mask bytes of the next unit's keys
      const auto look = [&](int u) {
        const int at = (w.u0 + u) * kUnit + lane;
        first = at < w.n ? mask[at] : 0;
        second = at + 32 < w.n ? mask[at + 32] : 0;
      };
      if (masked && U > 0) look(0);
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        const int keys = min(w.n - (w.u0 + u) * kUnit, kUnit);
        const int buf = u % SB;
        uint32_t bits[2] = {below(keys), below(keys - 32)};  // which are seen
        if (masked) {
          bits[0] = __ballot_sync(0xFFFFFFFFu, first), bits[1] = __ballot_sync(0xFFFFFFFFu, second);
          if (u + 1 < U) look(u + 1);
        }
        const uint32_t sc = s_col(t, buf) + lanes;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_soon(&sfull[t * SB + buf], phase >> buf & 1, p.status, kErrTimeoutEpilogue));
        if (!ok) break;
        phase ^= 1u << buf;
        tc_fence_after();
        if ((warp & 3) == 0) {  // (whole warps: what follows reads tensor memory)
          if constexpr (!C::kGives) {
            mbar_arrive_if(lane == 0 && (u % UPS == UPS - 1 || u == U - 1), &kempty[(g + u / UPS) % NS]);
            const int before = u - SB;  // its values have been read
            if (before >= 0) mbar_arrive_if(lane == 0 && before % UPS == UPS - 1, &vempty[(g + before / UPS) % NS]);
          }
          if constexpr (QB == 1) mbar_arrive_if(lane == 0 && u == U - 1, &qempty[t]);
        }
        const auto hide = [](uint32_t seen, uint32_t (&s)[32]) {
#pragma unroll
          for (int e = 0; e < 32; ++e) s[e] = seen >> e & 1u ? s[e] : 0xFF800000u;
        };
        const bool hidden = (bits[0] & bits[1]) != 0xFFFFFFFFu;
        const auto largest = [](const uint32_t (&s)[32]) {
          float m2[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            m2[q] = fmaxf(__uint_as_float(s[16 * q]), __uint_as_float(s[16 * q + 1]));
#pragma unroll
            for (int e = 2; e < 16; e += 2) m2[q] = max3(m2[q], __uint_as_float(s[16 * q + e]), __uint_as_float(s[16 * q + e + 1]));
          }
          return fmaxf(m2[0], m2[1]);
        };
        // With four row tiles registers hold 32 scores at a time: the second half is
        // looked over, let go and read again.
        constexpr int HELD = SB == 1 ? 1 : 2;
        uint32_t raw[HELD][32];
        float m = -INFINITY;
        if constexpr (HELD == 2) {
          tmem_ld32_nowait(sc, raw[0]);
          tmem_ld32_nowait(sc + 32, raw[1]);
          tmem_wait_ld();
          if (hidden) hide(bits[0], raw[0]), hide(bits[1], raw[1]);
          m = fmaxf(largest(raw[0]), largest(raw[1]));
        } else {
          if (keys > 32) {
            tmem_ld32_nowait(sc + 32, raw[0]);
            tmem_wait_ld();
            if (hidden) hide(bits[1], raw[0]);
            m = largest(raw[0]);
          }
          tmem_ld32_nowait(sc, raw[0]);
          tmem_wait_ld();
          if (hidden) hide(bits[0], raw[0]);
          m = fmaxf(m, largest(raw[0]));
        }
        // (lanes without a query hold whatever shared memory held, and must not
        // decide for the others)
        const bool rise = valid && (m - top) * c > 8.f;
        if (__any_sync(0xFFFFFFFFu, rise)) {
          const float up = fmaxf(m, top);
          const float f = up == -INFINITY ? 1.f : exp2_fast((top - up) * c);
          top = up;
          sum *= f;
          if (u > 0) {
            // P V of unit u - 1 must be done.  With one buffer these scores were
            // committed behind it; with two the next ones are, or it is the last but
            // one and has a commit of its own.
            if constexpr (SB > 1) {
              ok = __all_sync(0xFFFFFFFFu, u + 1 < U ? mbar_wait_soon(&sfull[t * SB + (buf ^ 1)], phase >> (buf ^ 1) & 1, p.status,
                                                                      kErrTimeoutEpilogue)
                                                     : mbar_wait_soon(&plast[t], last_phase, p.status, kErrTimeoutEpilogue));
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll 1
            for (int x = 0; x < kd * 16; x += 16) {
              uint32_t o[16];
              tmem_ld16_nowait(o_col(t) + lanes + x, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_col(t) + lanes + x, o);
            }
          }
        }
        const float base = top == -INFINITY ? 0.f : top * c - kLift<T>;
        const uint64_t c2 = f2(c, c), b2 = f2(-base, -base);
        uint64_t acc[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        const auto weigh = [&](int q, const uint32_t (&s)[32]) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = f2_of(fma2(f2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, b2));
            const float a = exp2_fast(x.x), b = exp2_fast(x.y);
            acc[(e >> 1) & 1] = add2(acc[(e >> 1) & 1], f2(a, b));
            pk[e / 2] = pack2<T>(a, b);
          }
          tmem_st16(sc + q * 16, pk);
        };
        if constexpr (HELD == 2) {
          weigh(0, raw[0]);
          if (keys > 32) weigh(1, raw[1]);
        } else {
          weigh(0, raw[0]);
          if (keys > 32) {
            tmem_ld32_nowait(sc + 32, raw[0]);
            tmem_wait_ld();
            if (hidden) hide(bits[1], raw[0]);
            weigh(1, raw[0]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&pfull[t * SB + buf]);
        const float2 a = f2_of(add2(acc[0], acc[1]));
        sum += a.x + a.y;
        if (QB == 2 && u == 0 && round > 0) {  // the last item's output has left its buffer by now
          if (r == 0) {
            bulk_wait_read<0>();
            mbar_arrive(&qempty[(round - 1) % QB * NT + t]);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      // while the last product runs: the statistics out, the next item
      const bool some = valid && !(sum == 0.f);
      const bool part = w.part;
      const int b = w.b, kvh = w.kvh, i0 = w.i0;
      if (!part && p.lse && row_used && i < p.tq) {
        const float base = top == -INFINITY ? 0.f : top * c - kLift<T>;
        p.lse[(static_cast<int64_t>(w.b) * p.hq + w.kvh * p.group + head) * p.tq + i] =
            some ? (base + log2f(sum)) * 0.69314718055994531f : -INFINITY;
      }
      if (U == 0 && !part) {  // nothing is seen
        if (row_used && i < p.tq) {
          T* to = static_cast<T*>(p.o) + w.b * p.o_s[0] + i * p.o_s[1] + (w.kvh * p.group + head) * p.o_s[2];
          for (int x = 0; x < p.d; x += 8) *reinterpret_cast<uint4*>(to + x) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }
      more = work.take(w);
      if (U > 0) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_soon(&odone[t], done_phase, p.status, kErrTimeoutEpilogue));
        if (!ok) break;
        done_phase ^= 1;
        if (SB > 1 && U > 1) last_phase ^= 1;
        tc_fence_after();
        if constexpr (!C::kGives) {
          if ((warp & 3) == 0) {
            for (int u = max(U - SB, 0); u < U; ++u)
              mbar_arrive_if(lane == 0 && (u % UPS == UPS - 1 || u == U - 1), &vempty[(g + u / UPS) % NS]);
          }
          g += (U + UPS - 1) / UPS;
        }
      }
      if (part) break;  // joined below; always a CTA's last
      if (U == 0) continue;
      const float inv = some ? 1.f / sum : 0.f;
      uint8_t* out = QB == 1 ? Out + t * C::kOut : Q + (round % QB * NT + t) * C::kQTile;
      ++round;
#pragma unroll 1
      for (int d = 0; d * 64 < p.d; ++d) {
        if (QB == 1) {
          if (r == 0) bulk_wait_read<0>();  // the last store has read the buffer
          __syncwarp();
          named_barrier_sync(1 + t, 128);
        }
#pragma unroll 1
        for (int x = 0; x < 64; x += 32) {
          uint32_t o[32];
          tmem_ld32_nowait(o_col(t) + lanes + d * 64 + x, o);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[q * 8 + e]) * inv;
            const uint4 z = Vec16<T>::pack(v);
            *reinterpret_cast<uint4*>(out + r * 128 + (((x / 8 + q) ^ (r & 7)) << 4)) = some ? z : make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();  // (the barrier takes whole warps)
        named_barrier_sync(1 + t, 128);
        if (r == 0 && i0 + t * p.per < p.tq) {
          tma_store_4d(&map_o, out, d * 64, kvh * p.group, i0 + t * p.per, b);
          bulk_commit();
        }
        __syncwarp();
      }
      tc_fence_before();  // (the next item's products overwrite what was read)
    }
    if (r == 0) bulk_wait_read<0>();  // the tile must outlive the store's reads
  }

  __syncwarp();
  // ---- a divided item: each CTA's part to its shared memory, joined over the cluster
  if (p.cluster > 1 && p.whole + static_cast<int>(blockIdx.x) / p.cluster < p.items) {
    Schedule<DB> again(p);
    again.lengths();
    while (again.next < p.whole) again.take(w);
    again.take(w);
    tc_fence_before();
    __syncthreads();  // every row tile's products are done: the operands' memory is free
    tc_fence_after();
    float* parts = reinterpret_cast<float*>(Q);
    constexpr int kPieces = DB * 16;  // of four values
    if (warp < 4 * p.tiles) {
      const int t = warp >> 2, r = threadIdx.x & 127;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      stats[t * 128 + r] = valid ? make_float2(top, sum) : make_float2(-INFINITY, 0.f);
#pragma unroll 1
      for (int x = 0; x < kd * 16; x += 16) {
        uint32_t o[16];
        if (w.units > 0) {
          tmem_ld16_nowait(o_col(t) + lanes + x, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 v = w.units > 0 && valid ? make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]) : make_uint4(0u, 0u, 0u, 0u);
          const int piece = (x / 4 + q) ^ (r & 7);
          *reinterpret_cast<uint4*>(parts + ((t * 128 + r) * kPieces + piece) * 4) = v;
        }
      }
    }
    cluster_sync();
    const int rank = static_cast<int>(cluster_ctarank());
    const float c = p.scale * 1.4426950408889634f;
    const int rows = p.tiles * 128, pieces = p.d / 8;
    for (int e = rank * C::kThreads + threadIdx.x; e < rows * pieces; e += p.cluster * C::kThreads) {
      const int row = e / pieces, col = e - row * pieces;
      const int t = row >> 7, r = row & 127, i = w.i0 + t * p.per + r / p.group;
      if (r >= p.per * p.group || i >= p.tq) continue;
      // the sums are relative to each part's maximum
      float2 st[8];
      float m = -INFINITY;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        st[s] = make_float2(-INFINITY, 0.f);
        if (s >= p.cluster) continue;
        const uint32_t sa = map_to_rank(&stats[row], s);
        st[s].x = ld_cluster_f32(sa), st[s].y = ld_cluster_f32(sa + 4);
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) m = fmaxf(m, st[s].x);
      const float at = m == -INFINITY ? 0.f : m;
      float acc[8] = {}, l = 0.f;
#pragma unroll
      for (int s2 = 0; s2 < 8; s2 += 2) {  // two parts' loads at a time, as registers allow
        float4 a[2], b[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          a[k] = b[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (s2 + k >= p.cluster) continue;
          a[k] = ld_cluster_f4(map_to_rank(parts + (row * kPieces + ((2 * col) ^ (r & 7))) * 4, s2 + k));
          b[k] = ld_cluster_f4(map_to_rank(parts + (row * kPieces + ((2 * col + 1) ^ (r & 7))) * 4, s2 + k));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 q = st[s2 + k];
          if (q.y == 0.f) continue;  // (a part that saw nothing)
          const float f = q.x == -INFINITY ? 1.f : exp2_fast((q.x - at) * c);
          l = fmaf(q.y, f, l);
          acc[0] = fmaf(a[k].x, f, acc[0]), acc[1] = fmaf(a[k].y, f, acc[1]);
          acc[2] = fmaf(a[k].z, f, acc[2]), acc[3] = fmaf(a[k].w, f, acc[3]);
          acc[4] = fmaf(b[k].x, f, acc[4]), acc[5] = fmaf(b[k].y, f, acc[5]);
          acc[6] = fmaf(b[k].z, f, acc[6]), acc[7] = fmaf(b[k].w, f, acc[7]);
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] *= inv;
      const int h = w.kvh * p.group + r % p.group;
      *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + w.b * p.o_s[0] + i * p.o_s[1] + h * p.o_s[2] + col * 8) =
          Vec16<T>::pack(acc);
      if (p.lse && col == 0) {
        const float base = m == -INFINITY ? 0.f : m * c - kLift<T>;
        p.lse[(static_cast<int64_t>(w.b) * p.hq + h) * p.tq + i] =
            l == 0.f ? -INFINITY : (base + log2f(l)) * 0.69314718055994531f;
      }
    }
    cluster_sync();  // a part stays until everyone has read it
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int DB> cudaError_t launch(const CrossTileLaunch* L, int cluster, int device, cudaStream_t stream, int* slots) {
  using C = Shape<DB>;
  auto kernel = cross_tile_kernel<T, DB>;
  static Kernel handle;
  if (slots) {
    *slots = handle.clusters(kernel, device, C::kThreads, C::kSmem, cluster) * cluster;
    return cudaSuccess;
  }
  TileParams p;
  static_cast<CrossParams&>(p) = L->p;
  p.per = L->per, p.tiles = L->tiles, p.blocks = L->blocks, p.items = L->items, p.whole = L->whole, p.cluster = L->cluster;
  const int units = L->grid / p.blocks;
  p.step_block = L->grid - units * p.blocks, p.step_b = units / p.hk, p.step_kvh = units - p.step_b * p.hk;
  return handle.launch(kernel, device, dim3(L->grid), C::kThreads, C::kSmem, cluster, stream, L->map_q, L->map_k, L->map_v,
                       L->map_o, p);
}

template <typename T> cudaError_t launch_t(int d, const CrossTileLaunch* L, int cluster, int device, cudaStream_t stream, int* slots) {
  if (d <= 64) return launch<T, 1>(L, cluster, device, stream, slots);
  if (d <= 128) return launch<T, 2>(L, cluster, device, stream, slots);
  return launch<T, 4>(L, cluster, device, stream, slots);
}

}  // namespace

cudaError_t launch_cross_tile(const CrossTileLaunch& L, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(L.p.d, &L, L.cluster, L.device, stream, nullptr)
              : launch_t<__half>(L.p.d, &L, L.cluster, L.device, stream, nullptr);
}

int cross_tile_slots(int d, bool bf16, int cluster, int device) {
  int slots = 0;
  bf16 ? launch_t<__nv_bfloat16>(d, nullptr, cluster, device, nullptr, &slots)
       : launch_t<__half>(d, nullptr, cluster, device, nullptr, &slots);
  return slots;
}

}  // namespace oidnx
