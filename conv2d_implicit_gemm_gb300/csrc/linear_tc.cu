// Linear layer on the 5th-generation tensor cores: y = act(x w^T + bias) + residual.
//
//  * Output tiles of 128 x BN per CTA, or 256 x BN per CTA pair
//    (cta_group::2: each CTA holds its 128 rows of x and half of the tile's
//    rows of w, and the pair reads both), fp32 accumulators in tensor memory,
//    two of them, so that one tile's epilogue runs under the next tile's
//    products.  Persistent CTAs walk the tiles in groups of 8 row blocks, so
//    that the tiles in flight share their operands in L2.
//  * K in blocks of 64 values: one 128-byte swizzled TMA box per operand and
//    block.  (Matrices whose rows do not start on 16 bytes are laid out anew
//    before, by linear_align.cu.)
//  * Epilogue: eight warps, each 32 rows x half the columns, through 32 x 64
//    tiles of 16-bit values that TMA stores (and, for the residual, loads
//    first); outputs that TMA cannot store (rows off 16 bytes, or that end within
//    16 bytes) go row by row in 32-bit words, shifted where a row starts on an odd
//    place.
//  * The MMA warp overwrites the accumulator with its first product and adds
//    the others; products outside the matrix are zeros that TMA fills in.
// 8192 x 8192 x 4096, bf16, gelu_tanh: 295 us alone (1865 TFLOP/s, the tensor pipe
// active 90% of the time), 315 to 343 among others, where the power limit lowers
// the clock (the measured library rates are 1898 in a burst and 1702 sustained).
//  * Every wait is bounded.  A role that gives up records it and leaves its
//    loop; its own loads were issued before that wait of two seconds and have
//    landed, and the other roles give up in turn, so the block ends together.
#include <climits>
#include <type_traits>

#include "token_ptx.cuh"
#include "token.h"
#include "token_math.cuh"

namespace oidnx {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kFirstEpi = 4;  // warp 0 loads, warp 1 multiplies, 2 and 3 rest
constexpr int kLinThreads = (kFirstEpi + kEpiWarps) * 32;
constexpr int kStageOut = 4096;  // bytes of staging per epilogue warp, on 1024
constexpr int kRoomMore = 128;   // the same of rows in words of their own (32 x 33)
constexpr int kKB = 64;          // values of one K block: one 128-byte row of a tile
constexpr int kRowGroup = 8;     // row blocks walked together

template <int CG, int BN> struct Shape {
  static constexpr int kA = 128 * 128;              // bytes of a CTA's x block
  static constexpr int kB = BN / CG * 128;          // bytes of its w block
  static constexpr int kStage = kA + kB;
  static constexpr int kRoom = 227 * 1024 - 2048 - kEpiWarps * (kStageOut + kRoomMore);
  static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
  static constexpr int kSmem = kStages * kStage + kEpiWarps * (kStageOut + kRoomMore) + 2048;
  static constexpr int kCols = 2 * BN < 32 ? 32 : 2 * BN;
};

struct TcArgs {
  LinearParams p;
  int tiles_m, tiles_n;
  int tma_out;  // y (and the residual) go through TMA
};

// Walk step -> tile: groups of kRowGroup row blocks, column by column.
__device__ __forceinline__ void tile_of(const TcArgs& a, int t, int* tm, int* tn) {
  const int per = kRowGroup * a.tiles_n;
  const int g = t / per, i = t - g * per;
  const int rows = min(kRowGroup, a.tiles_m - g * kRowGroup);
  *tn = i / rows;
  *tm = g * kRowGroup + i - *tn * rows;
}

// Bias of 32 columns from c0 on (zeros outside), for every lane.
template <typename T>
__device__ __forceinline__ void add_bias(const LinearParams& p, int c0, float (&v)[32]) {
  if (!p.bias) return;
  const T* b = static_cast<const T*>(p.bias) + c0;
  if (c0 + 32 <= p.n && (reinterpret_cast<uintptr_t>(b) & 15) == 0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[8];
      Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4*>(b) + q), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * q + i] += f[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c0 + i < p.n) v[i] += to_f32<T>(b[i]);
  }
}

// One lane: once the store before has left the staging tile, the residual's
// tile into it.
template <int W>
__device__ __forceinline__ void fetch_residual(const LinearParams& p, const CUtensorMap* map_r, uint8_t* stage,
                                               uint64_t* bar, int r0, int c0) {
  bulk_wait_read<0>();
  if (!p.residual) return;
  mbar_arrive_expect_tx(bar, 32 * W * 2);
  tma_load_2d(stage, map_r, bar, c0, r0, l2_evict_first());
}

// Columns [c0, c0 + COLS) of 32 rows from r0 on (the first tile's residual
// fetched by the caller), accumulators at `tmem` (lane
// = row), through the warp's staging tile.  `bar`/`phase`: residual loads.
template <typename T, int COLS>
__device__ __forceinline__ bool epilogue_tma(const TcArgs& a, const CUtensorMap* map_y, const CUtensorMap* map_r,
                                             uint32_t tmem, int r0, int c0, uint8_t* stage, uint64_t* bar,
                                             uint32_t* phase, int lane) {
  const LinearParams& p = a.p;
  constexpr int W = COLS < 64 ? COLS : 64;  // columns of one staging tile
#pragma unroll 1
  for (int c = 0; c < COLS; c += W) {
    if (c0 + c >= p.n) break;
    if (c > 0) {
      if (lane == 0) fetch_residual<W>(p, map_r, stage, bar, r0, c0 + c);
      __syncwarp();
    }
    if (p.residual) {
      const bool landed = mbar_wait_bounded(bar, *phase, p.status, kErrTimeoutEpilogue);
      *phase ^= 1;
      if (!__all_sync(0xFFFFFFFFu, landed)) return false;
    }
#pragma unroll
    for (int h = 0; h < W; h += 32) {
      uint32_t raw[32];
      tmem_ld32_nowait(tmem + c + h, raw);
      tmem_wait_ld();
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
      add_bias<T>(p, c0 + c + h, v);
      activate_all(v, p.act);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int piece = h / 8 + q;
        // 128-byte rows swizzled by row mod 8; 64-byte rows by (row / 2) mod 4
        uint4* at = reinterpret_cast<uint4*>(
            stage + lane * (W * 2) + ((W == 64 ? piece ^ (lane & 7) : piece ^ ((lane >> 1) & 3)) << 4));
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[8 * q + i];
        if (p.residual) {
          float f[8];
          Vec16<T>::unpack(*at, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += f[i];
        }
        *at = Vec16<T>::pack(o);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map_y, stage, c0 + c, r0);
      bulk_commit();
    }
  }
  return true;
}

// Outputs that TMA cannot store: tiles of 32 rows x W columns through shared
// memory, each row in words as its own alignment asks for (2040 x 1001 x 1000 with
// residual 14.7 us, 2040 x 1000 x 1000 through TMA 13.6; by single 16-bit values 18.8).
// Rows on 16 bytes that end within 16 (1001 values of 1008): 14.4.  With s = 1 where the
// row starts on an odd 16-bit place (0 else), word l holds columns 2 l - s and
// 2 l - s + 1, so that a warp reads and writes whole words; column 0 of s = 1 and
// a last column that no pair takes go alone, one lane a row.
template <typename T, int W> struct Ragged {
  static constexpr int kLanes = W / 2;          // lanes a row
  static constexpr int kRows = 32 / kLanes;     // rows at a time
  static constexpr int kSteps = 32 / kRows;
  static constexpr int kWords = W / 2 + 1;      // of a row (odd: no bank conflicts either way)

  const char* base;  // of the tile
  int64_t ld;
  int rows, cols;    // inside the matrix

  __device__ __forceinline__ Ragged(const void* x, int64_t row, int m, int n, int r0, int c0)
      : base(static_cast<const char*>(x) + 2 * (r0 * row + c0)), ld(row), rows(min(32, m - r0)), cols(min(W, n - c0)) {}
  __device__ __forceinline__ int shift(int r) const {
    return ((reinterpret_cast<uintptr_t>(base) >> 1) + static_cast<uint32_t>(ld) * r) & 1;
  }
  __device__ __forceinline__ bool first_alone(int r) const { return r < rows && cols > 0 && shift(r); }
  __device__ __forceinline__ bool last_alone(int r) const { return r < rows && cols > 0 && ((cols ^ shift(r)) & 1); }
  // Is word l of row r a pair inside the tile?
  __device__ __forceinline__ bool pair(int r, int l) const {
    const int c = 2 * l - shift(r);
    return r < rows && c >= 0 && c + 1 < cols;
  }
  __device__ __forceinline__ char* at(int r, int c) const { return const_cast<char*>(base) + 2 * (r * ld + c); }

  // From the matrix to registers, on to shared memory, and back from there.
  struct Values {
    uint32_t z[kSteps];
    uint16_t first, last;
  };
  __device__ __forceinline__ void load(Values& v, int lane) const {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = i * kRows + lane / kLanes, l = lane % kLanes;
      v.z[i] = pair(r, l) ? *reinterpret_cast<const uint32_t*>(at(r, 2 * l - shift(r))) : 0u;
    }
    v.first = first_alone(lane) ? *reinterpret_cast<const uint16_t*>(at(lane, 0)) : 0;
    v.last = last_alone(lane) ? *reinterpret_cast<const uint16_t*>(at(lane, cols - 1)) : 0;
  }
  __device__ __forceinline__ void put(const Values& v, uint32_t* tile, int lane) const {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) tile[(i * kRows + lane / kLanes) * kWords + lane % kLanes] = v.z[i];
    __syncwarp();
    uint16_t* half = reinterpret_cast<uint16_t*>(tile + lane * kWords);
    if (first_alone(lane)) half[1] = v.first;
    if (last_alone(lane)) half[cols - 1 + shift(lane)] = v.last;
  }
  __device__ __forceinline__ void store(const uint32_t* tile, int lane) const {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = i * kRows + lane / kLanes, l = lane % kLanes;
      if (pair(r, l)) *reinterpret_cast<uint32_t*>(at(r, 2 * l - shift(r))) = tile[r * kWords + l];
    }
    const uint16_t* half = reinterpret_cast<const uint16_t*>(tile + lane * kWords);
    if (first_alone(lane)) *reinterpret_cast<uint16_t*>(at(lane, 0)) = half[1];
    if (last_alone(lane)) *reinterpret_cast<uint16_t*>(at(lane, cols - 1)) = half[cols - 1 + shift(lane)];
  }
};

// The epilogue for them.  z: the first tile's residual; each next one is loaded
// a tile ahead (y may be the residual, so the compiler keeps a load behind every
// earlier store, but another tile's values are not written before).
template <typename T, int COLS, int W>
__device__ __forceinline__ void epilogue_any(const TcArgs& a, uint32_t tmem, int r0, int c0, uint8_t* stage, int lane,
                                             typename Ragged<T, W>::Values& z) {
  using R = Ragged<T, W>;
  const LinearParams& p = a.p;
  uint32_t* tile = reinterpret_cast<uint32_t*>(stage);
  uint32_t* row = tile + lane * R::kWords;
#pragma unroll 1
  for (int c = 0; c < COLS; c += W) {
    if (c0 + c >= p.n) break;
    const R y(p.y, p.ldy, p.m, p.n, r0, c0 + c), res(p.residual, p.ldr, p.m, p.n, r0, c0 + c);
    if (p.residual) {
      res.put(z, tile, lane);
      if (c + W < COLS) R(p.residual, p.ldr, p.m, p.n, r0, c0 + c + W).load(z, lane);
      __syncwarp();
    }
    // words as they are, or each with the upper half of the one before
    const uint32_t pick_res = res.shift(lane) ? 0x5432u : 0x3210u, pick_y = y.shift(lane) ? 0x5432u : 0x7654u;
    uint32_t word = 0;  // the last whole one
#pragma unroll
    for (int h = 0; h < W; h += 32) {
      uint32_t raw[32];
      tmem_ld32_nowait(tmem + c + h, raw);
      tmem_wait_ld();
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
      add_bias<T>(p, c0 + c + h, v);
      activate_all(v, p.act);
      if (p.residual) {
        uint32_t now = row[h / 2];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t next = row[h / 2 + i + 1];
          const float2 f = unpack2<T>(__byte_perm(now, next, pick_res));
          v[2 * i] += f.x, v[2 * i + 1] += f.y;
          now = next;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t both = pack2<T>(v[2 * i], v[2 * i + 1]);
        row[h / 2 + i] = __byte_perm(word, both, pick_y);
        word = both;
      }
    }
    row[W / 2] = word >> 16;  // (the last column's, where the row is shifted)
    __syncwarp();
    y.store(tile, lane);
    __syncwarp();
  }
}

template <typename T, int CG, int BN>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_y,
                     const TcArgs a) {
  using S = Shape<CG, BN>;
  constexpr int NS = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;  // every tile starts on 1024 bytes
  uint8_t* staging = stages + NS * S::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * (kStageOut + kRoomMore));
  uint64_t* empty = full + NS;
  uint64_t* tfull = empty + NS;    // [2]
  uint64_t* tempty = tfull + 2;    // [2]
  uint64_t* rbar = tempty + 2;     // [kEpiWarps] residual tiles
  uint32_t* slot = reinterpret_cast<uint32_t*>(rbar + kEpiWarps);
  const LinearParams& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const int kb = (p.k + kKB - 1) / kKB;
  const int tiles = a.tiles_m * a.tiles_n;
  const int walker = blockIdx.x / CG, walkers = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], CG * kEpiWarps);
    }
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&rbar[w], 1);
    fence_mbarrier_init();
  }
  if (warp == 1) {
    if (CG == 2) tmem_alloc_pair(slot, S::kCols);
    else tmem_alloc(slot, S::kCols);
  }
  tc_fence_before();
  if (CG == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&map_x);
      prefetch_tmap(&map_w);
      const uint64_t pol = l2_evict_normal();
      uint32_t s = 0, ph = 0;
      bool ok = true;
      for (int t = walker; t < tiles && ok; t += walkers) {
        int tm, tn;
        tile_of(a, t, &tm, &tn);
        const int row = (tm * CG + static_cast<int>(rank)) * 128;
        const int col = tn * BN + static_cast<int>(rank) * (BN / CG);
        for (int k = 0; k < kb; ++k) {
          ok = mbar_wait_bounded(&empty[s], ph ^ 1, p.status, kErrTimeoutProducer);
          if (!ok) break;
          uint8_t* A = stages + s * S::kStage;
          if (CG == 2) {
            const uint32_t bar = map_to_rank(&full[s], 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * S::kStage);
            tma_load_2d_pair(A, &map_x, bar, k * kKB, row, pol);
            tma_load_2d_pair(A + S::kA, &map_w, bar, k * kKB, col, pol);
          } else {
            mbar_arrive_expect_tx(&full[s], S::kStage);
            tma_load_2d(A, &map_x, &full[s], k * kKB, row, pol);
            tma_load_2d(A + S::kA, &map_w, &full[s], k * kKB, col, pol);
          }
          if (++s == NS) s = 0, ph ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_16(std::is_same<T, __nv_bfloat16>::value, 128 * CG, BN);
      uint32_t s = 0, ph = 0;
      int n = 0;
      bool ok = true;
      for (int t = walker; t < tiles && ok; t += walkers, ++n) {
        const int b = n & 1;
        ok = mbar_wait_bounded(&tempty[b], ((n >> 1) & 1) ^ 1, p.status, kErrTimeoutMma);
        tc_fence_after();
        const uint32_t d = tmem + b * BN;
        for (int k = 0; k < kb && ok; ++k) {
          ok = mbar_wait_bounded(&full[s], ph, p.status, kErrTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = smem_desc_sw128(smem_u32(stages + s * S::kStage));
          const uint64_t bd = smem_desc_sw128(smem_u32(stages + s * S::kStage + S::kA));
#pragma unroll
          for (int i = 0; i < kKB / 16; ++i) {
            if (CG == 2) mma_f16_ss_pair(d, ad + 2 * i, bd + 2 * i, idesc, k > 0 || i > 0);
            else mma_f16_ss(d, ad + 2 * i, bd + 2 * i, idesc, k > 0 || i > 0);
          }
          if (CG == 2) mma_commit_pair(&empty[s]);
          else mma_commit(&empty[s]);
          if (++s == NS) s = 0, ph ^= 1;
        }
        if (CG == 2) mma_commit_pair(&tfull[b]);
        else mma_commit(&tfull[b]);
      }
    }
  } else if (warp >= kFirstEpi) {
    const int e = warp - kFirstEpi;
    const int quarter = warp & 3, half = e >> 2;  // the TMEM lanes a warp may read; its columns
    uint8_t* stage = staging + e * (a.tma_out ? kStageOut : kStageOut + kRoomMore);
    uint32_t rphase = 0;
    int n = 0;
    for (int t = walker; t < tiles; t += walkers, ++n) {
      const int b = n & 1;
      int tm, tn;
      tile_of(a, t, &tm, &tn);
      const int r0 = (tm * CG + static_cast<int>(rank)) * 128 + quarter * 32;
      const int c0 = tn * BN + half * (BN / 2);
      // the epilogue's reads on their way while the products run
      // (64 columns and the next tile's residual would not fit the registers of 256:
      // 4000 x 3001 x 2000 69 us, with 32 59; 2040 x 1001 x 1000 in tiles of 128 columns
      // 15.2 with 64, 17.1 with 32)
      constexpr int W = BN == 128 ? 64 : 32;
      typename Ragged<T, W>::Values z;
      if (r0 < p.m && c0 < p.n) {
        if (a.tma_out && lane == 0)
          fetch_residual<BN / 2 < 64 ? BN / 2 : 64>(p, &map_r, stage, &rbar[e], r0, c0);
        if (p.bias && lane < BN / 2 / 32) prefetch_l1(static_cast<const T*>(p.bias) + min(c0 + lane * 32, p.n - 1));
        if (!a.tma_out && p.residual) Ragged<T, W>(p.residual, p.ldr, p.m, p.n, r0, c0).load(z, lane);
      }
      __syncwarp();
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&tfull[b], (n >> 1) & 1, p.status, kErrTimeoutEpilogue))) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * BN + half * (BN / 2);
      if (r0 < p.m) {
        if (a.tma_out) {
          if (!epilogue_tma<T, BN / 2>(a, &map_y, &map_r, acc, r0, c0, stage, &rbar[e], &rphase, lane)) break;
        } else {
          epilogue_any<T, BN / 2, W>(a, acc, r0, c0, stage, lane, z);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2) mbar_arrive_cluster(map_to_rank(&tempty[b], 0));
        else mbar_arrive(&tempty[b]);
      }
    }
    if (lane == 0) bulk_wait_read<0>();  // the staging tiles must outlive their stores
  }

  __syncwarp();
  tc_fence_before();
  if (CG == 2) cluster_sync();  // the pair's products read both CTAs' shared memory
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2) tmem_dealloc_pair(tmem, S::kCols);
    else tmem_dealloc(tmem, S::kCols);
  }
}

template <typename T, int CG, int BN>
cudaError_t launch(const LinearTcLaunch& L, cudaStream_t stream) {
  using S = Shape<CG, BN>;
  TcArgs a = {L.p, (L.p.m + 128 * CG - 1) / (128 * CG), (L.p.n + BN - 1) / BN, L.tma_out};
  auto kernel = linear_tc_kernel<T, CG, BN>;
  static Kernel handle;
  const long long tiles = static_cast<long long>(a.tiles_m) * a.tiles_n;
  if (tiles > INT_MAX) return cudaErrorInvalidValue;
  const int walkers = static_cast<int>(tiles < L.sms / CG ? tiles : L.sms / CG);
  return handle.launch(kernel, L.device, dim3(walkers * CG), kLinThreads, S::kSmem, CG,
                       stream, L.map_x, L.map_w, L.map_r, L.map_y, a);
}

template <typename T>
cudaError_t launch_t(const LinearTcLaunch& L, cudaStream_t stream) {
  if (L.pair) return L.bn == 256 ? launch<T, 2, 256>(L, stream) : launch<T, 2, 128>(L, stream);
  if (L.bn == 64) return launch<T, 1, 64>(L, stream);
  return launch<T, 1, 128>(L, stream);
}

}  // namespace

cudaError_t launch_linear_tc(const LinearTcLaunch& L, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(L, stream) : launch_t<__half>(L, stream);
}

}  // namespace oidnx
