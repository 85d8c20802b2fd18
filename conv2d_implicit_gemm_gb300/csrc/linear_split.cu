// Linear layer for few tokens: bound by the weight's bytes, so the weight is
// the operand with 128 rows and the tokens are the narrow one,
//   acc[j][i] = sum_k w[j][k] x[i][k],
// and K is split over the CTAs of a cluster, so that every SM streams weights
// however few output tiles there are.  Each CTA leaves its fp32 part of the
// 128 x BN tile in its shared memory; after a cluster barrier every CTA sums
// 128 / split rows over the parts (always in the same order) and applies the
// epilogue.
//
// 1 x 4096 x 4096: 9.3 us on the device, 10.2 with bias and residual (3.9 of them at
// any size: launch, first loads, joining; the rest streams the weight at 5.8 TB/s);
// 1 x 8192 x 8192: 23.6 us, 5.7 TB/s.  Rows that do not start on 16 bytes: 15.7 us for
// 1 x 4096 x 4095, their copies and shifts being two passes through shared memory.
#include <type_traits>

#include "linear_load.cuh"
#include "token_ptx.cuh"
#include "token.h"
#include "token_math.cuh"

namespace oidnx {
namespace {

// Warp 0 loads, warp 1 multiplies, warps 4-7 read the accumulator, all join the
// sums; gathered operands: warps 2, 3, 12 and 13 copy, warps 4-11 shift.
constexpr int kThreads = 256;
constexpr int kThreadsGather = 448;

template <int BN, bool GATHER> struct Split {
  static constexpr int kA = 128 * 128;
  static constexpr int kB = BN * 128;
  static constexpr int kStage = kA + kB;
  // two CTAs per SM; a gathering one's room holds blocks on their way as they
  // lie in memory as well
  static constexpr int kStages = GATHER ? 2 : 110 * 1024 / kStage;
  static constexpr int kRawStages = GATHER ? 3 : 0;
  static constexpr int kRaw = kRawStages * (128 + BN) * 144;
  static constexpr int kSmem = kStages * kStage + kRaw + 2048;
  static constexpr int kCols = BN < 32 ? 32 : BN;
  static_assert(kStages * kStage + kRaw >= 128 * BN * 4, "the parts reuse the stages");
};

template <typename T, int BN, bool GATHER>
__global__ void __launch_bounds__(GATHER ? kThreadsGather : kThreads, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                        const LinearParams p, const int split) {
  using S = Split<BN, GATHER>;
  constexpr int NS = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;
  uint8_t* raw = stages + NS * S::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(raw + S::kRaw);
  uint64_t* empty = full + NS;
  uint64_t* done = empty + NS;
  uint64_t* rawfull = done + 1;  // [RS]
  uint64_t* rawempty = rawfull + S::kRawStages;
  uint32_t* slot = reinterpret_cast<uint32_t*>(rawempty + S::kRawStages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int j0 = blockIdx.x / split * 128, i0 = blockIdx.y * BN;
  const int blocks = p.k > 0 ? (p.k + kKB - 1) / kKB : 1;
  const int first = static_cast<int>(static_cast<int64_t>(blocks) * part / split);
  const int last = static_cast<int>(static_cast<int64_t>(blocks) * (part + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], GATHER ? kPlaceThreads / 32 : 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    for (int r = 0; r < S::kRawStages; ++r) {
      mbar_init(&rawfull[r], 2 * kCopyThreads);
      mbar_init(&rawempty[r], kPlaceThreads / 32);
    }
    fence_mbarrier_init();
  }
  if (warp == 1) tmem_alloc(slot, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  griddep_launch_dependents();
  griddep_wait();

  float* sums = reinterpret_cast<float*>(stages);  // [BN][128], once every product has read the stages
  if (warp == 0) {
    if (!GATHER && lane == 0) {
      const uint64_t pol = l2_evict_normal();
      uint32_t s = 0, ph = 0;
      for (int k = first; k < last; ++k) {
        if (!mbar_wait_bounded(&empty[s], ph ^ 1, p.status, kErrTimeoutProducer)) break;
        uint8_t* A = stages + s * S::kStage;
        mbar_arrive_expect_tx(&full[s], S::kStage);
        tma_load_2d(A, &map_w, &full[s], k * kKB, j0, pol);
        tma_load_2d(A + S::kA, &map_x, &full[s], k * kKB, i0, pol);
        if (++s == NS) s = 0, ph ^= 1;
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_16(std::is_same<T, __nv_bfloat16>::value, 128, BN);
      uint32_t s = 0, ph = 0;
      for (int k = first; k < last; ++k) {
        if (!mbar_wait_bounded(&full[s], ph, p.status, kErrTimeoutMma)) break;
        tc_fence_after();
        const uint64_t ad = smem_desc_sw128(smem_u32(stages + s * S::kStage));
        const uint64_t bd = smem_desc_sw128(smem_u32(stages + s * S::kStage + S::kA));
#pragma unroll
        for (int i = 0; i < kKB / 16; ++i) mma_f16_ss(tmem, ad + 2 * i, bd + 2 * i, idesc, k > first || i > 0);
        mma_commit(&empty[s]);
        if (++s == NS) s = 0, ph ^= 1;
      }
      mma_commit(done);
    }
  } else if (warp < 4 || warp >= 12) {
    if constexpr (GATHER) {
      Gather<128, BN> g;
      g.matrices(p.w, p.ldw, p.n, p.x, p.ldx, p.m, p.k);
      g.a.r0 = j0, g.b.r0 = i0;
      int r = 0, ph = 0;
      for (int k = first; k < last; ++k) {
        if (!mbar_wait_bounded(&rawempty[r], ph ^ 1, p.status, kErrTimeoutProducer)) break;
        g.copy_block(raw + r * g.kStage, &rawfull[r], k * kKB, warp < 4 ? threadIdx.x - 64 : threadIdx.x - 384 + 64);
        if (++r == S::kRawStages) r = 0, ph ^= 1;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    if constexpr (GATHER) {
      Gather<128, BN> g;
      g.matrices(p.w, p.ldw, p.n, p.x, p.ldx, p.m, p.k);
      g.a.r0 = j0, g.b.r0 = i0;
      uint32_t s = 0, ph = 0, rs = 0, rph = 0;
      for (int k = first; k < last; ++k) {
        const bool ok = mbar_wait_bounded(&rawfull[rs], rph, p.status, kErrTimeoutProducer) &&
                        mbar_wait_bounded(&empty[s], ph ^ 1, p.status, kErrTimeoutProducer);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        uint8_t* A = stages + s * S::kStage;
        g.place(raw + rs * g.kStage, A, A + S::kA, p.k - k * kKB, threadIdx.x - 128);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]), mbar_arrive(&rawempty[rs]);
        if (++s == NS) s = 0, ph ^= 1;
        if (++rs == S::kRawStages) rs = 0, rph ^= 1;
      }
    }
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(done, 0, p.status, kErrTimeoutEpilogue));
    tc_fence_after();
    const int quarter = warp & 3;
    if (ok && warp < 8) {
#pragma unroll 1
      for (int c = 0; c < BN; c += 16) {
        if (i0 + c >= p.m) break;
        uint32_t raw[16];
        tmem_ld16_nowait(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, raw);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          // an empty range of K has issued no product: its part is zero
          sums[(c + i) * 128 + quarter * 32 + lane] = last > first ? __uint_as_float(raw[i]) : 0.f;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  if (split > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kCols);
  }

  // This CTA's rows of the tile, for all its tokens: four rows a thread, the
  // loads of two such pieces before the first store (y may be the residual).
  const int rows = 128 / split, r0 = part * rows;
  const int tokens = min(BN, p.m - i0);
  const int items = rows / 4 * tokens, threads = blockDim.x;
  uint32_t at[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) at[s] = split > 1 && s < split ? map_to_rank(sums, s) : smem_u32(sums);
  for (int e0 = threadIdx.x; e0 < items; e0 += 2 * threads) {
    float4 z[2];
    float res[2][4], bias[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = e0 + h * threads;
      if (e >= items) break;
      const int i = e / (rows / 4), r = r0 + e % (rows / 4) * 4, j = j0 + r;
      const uint32_t off = (i * 128 + r) * 4;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t row = i0 + i;
        bias[h][q] = p.bias && j + q < p.n ? to_f32<T>(static_cast<const T*>(p.bias)[j + q]) : 0.f;
        res[h][q] =
            p.residual && j + q < p.n ? to_f32<T>(static_cast<const T*>(p.residual)[row * p.ldr + j + q]) : 0.f;
      }
      if (split == 1) {
        z[h] = *reinterpret_cast<const float4*>(sums + i * 128 + r);
      } else {
        float4 v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) v[s] = s < split ? ld_cluster_f4(at[s] + off) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 4; w > 0; w >>= 1)
#pragma unroll
          for (int s = 0; s < w; ++s)
            v[s].x += v[s + w].x, v[s].y += v[s + w].y, v[s].z += v[s + w].z, v[s].w += v[s + w].w;
        z[h] = v[0];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = e0 + h * threads;
      if (e >= items) break;
      const int i = e / (rows / 4), j = j0 + r0 + e % (rows / 4) * 4;
      float f[4] = {z[h].x + bias[h][0], z[h].y + bias[h][1], z[h].z + bias[h][2], z[h].w + bias[h][3]};
      activate_all(f, p.act);
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] += res[h][q];
      T* y = static_cast<T*>(p.y) + static_cast<int64_t>(i0 + i) * p.ldy + j;
      if (j + 4 <= p.n && (reinterpret_cast<uintptr_t>(y) & 7) == 0) {
        *reinterpret_cast<uint2*>(y) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q < p.n) y[q] = from_f32<T>(f[q]);
      }
    }
  }
  if (split > 1) cluster_sync();  // a part stays until everyone has read it
}

template <typename T, int BN, bool GATHER>
cudaError_t launch(const LinearTcLaunch& L, cudaStream_t stream) {
  using S = Split<BN, GATHER>;
  auto kernel = linear_split_kernel<T, BN, GATHER>;
  static Kernel handle;
  return handle.launch(kernel, L.device, dim3((L.p.n + 127) / 128 * L.split, (L.p.m + BN - 1) / BN),
                       GATHER ? kThreadsGather : kThreads, S::kSmem, L.split, stream, L.map_x, L.map_w, L.p, L.split);
}

template <typename T>
cudaError_t launch_t(const LinearTcLaunch& L, cudaStream_t stream) {
  if (L.gather) return L.bn <= 16 ? launch<T, 16, true>(L, stream) : launch<T, 32, true>(L, stream);
  if (L.bn <= 16) return launch<T, 16, false>(L, stream);
  if (L.bn <= 32) return launch<T, 32, false>(L, stream);
  if (L.bn <= 64) return launch<T, 64, false>(L, stream);
  return launch<T, 128, false>(L, stream);
}

}  // namespace

cudaError_t launch_linear_split(const LinearTcLaunch& L, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_t<__nv_bfloat16>(L, stream) : launch_t<__half>(L, stream);
}

}  // namespace oidnx
