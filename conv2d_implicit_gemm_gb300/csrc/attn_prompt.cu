// Window attention for prompts on the 5th-generation tensor cores.
//
// A CTA takes two tiles of 128 query rows of one key head (queries x the heads
// of its group, query-major, so that keys and values are read once for the
// group) and walks the visible keys in tiles of 128: the sinks, then the
// window, in runs of consecutive cache slots.
//
//   S = Q K^T (tcgen05, accumulators in tensor memory), softmax in registers
//   (one thread a row), P in 16 bits over S in tensor memory, O += P V with P
//   as the tensor-memory operand and V read as it lies (values contiguous).
//
//  * Each key tile in two halves of 64, each with its own columns for S and P: the
//    tensor cores write one half's scores while the softmax warps are at the
//    other's, and the two row tiles' products alternate.
//  * The running maximum that P is relative to follows the true one only when
//    it falls more than 2^8 behind, so O is rescaled rarely; P <= 2^8 (fp16: 2^15,
//    to keep the small ones) stays within 16 bits and the sums are fp32, so
//    nothing is lost by it.
//  * P is rounded to the storage type, as both operands of a product have one
//    type; its error is that of the inputs' own rounding and averages out
//    over the keys.  The sum of the weights is taken before the rounding.
//  * Tiles that every row sees whole skip the mask.  In the others a value
//    that is no number must not reach rows that do not see it (0 x NaN):
//    a warp looks the tile's values over first, clears what lies past the
//    keys, and where a key itself holds such a value the CTA's rows are done
//    again one by one.
//
// Bound by shared memory and the softmax warps alike: some 3000 cycles a key tile,
// of which 2500 read operands (the queries again for each half of the keys;
// without three quarters of those products the whole takes 8% less) and 2800 are
// a softmax warp's own (without its exponentials alone nothing changes).  8192 tokens,
// window 2048, 16 heads of 128 over 4: 107 us, 1120 TFLOP/s of visible pairs, the
// tensor pipe active half of the time.  Whole key tiles, no half in advance: 128;
// sixteen softmax warps (two threads a row, exchanging maxima) 141; waits whose
// ready case goes through a loop (250 cycles instead of some 20, five of them a
// key tile in the issuing thread) 112.
//
// Warps 0-3 and 4-7: softmax of row tile 0 and 1, rescaling, output; warp 8
// loads (TMA), warps 9 and 10 issue the products of a row tile each (one thread
// for both was the bound), warp 11 looks values over.
#include "attn_prompt.cuh"

namespace oidnx {
namespace {

constexpr int kSoftWarps = 8;
constexpr int kThreads = (kSoftWarps + 4) * 32;
constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kLookWarp = kSoftWarps + 3;

constexpr int DB = 2;              // 64-value blocks of a head
constexpr int kTile = DB * 16384;  // 128 rows
constexpr int NS = 2;              // key tiles (and value tiles) in flight
constexpr int kSmem = (2 + 2 * NS) * kTile + 1024 + 512;

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                       const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* Q = smem_raw + pad;  // [2 row tiles]; the output tiles at the end
  uint8_t* Ks = Q + 2 * kTile;
  uint8_t* Vs = Ks + NS * kTile;
  uint64_t* qfull = reinterpret_cast<uint64_t*>(Vs + NS * kTile);  // [2]
  uint64_t* kfull = qfull + 2;    // [NS]
  uint64_t* kempty = kfull + NS;
  uint64_t* vfull = kempty + NS;
  uint64_t* vempty = vfull + NS;
  uint64_t* sfull = vempty + NS;  // [2 row tiles][2 halves of the keys]
  uint64_t* pfull = sfull + 4;    // the same
  uint64_t* pdone = pfull + 4;    // the same
  uint64_t* odone = pdone + 4;    // [2]
  uint64_t* vclean = odone + 2;   // [NS]
  uint32_t* slot = reinterpret_cast<uint32_t*>(vclean + NS);
  int* odd = reinterpret_cast<int*>(slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 4);  // both row tiles' halves
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 5);  // and the looking warp
      mbar_init(&vclean[s], 32);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&qfull[t], 1);
      mbar_init(&odone[t], 1);
    }
    for (int c = 0; c < 4; ++c) {
      mbar_init(&sfull[c], 1);
      mbar_init(&pfull[c], 128);
      mbar_init(&pdone[c], 1);
    }
    *odd = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  griddep_launch_dependents();
  griddep_wait();
  const Plan w = make_plan(p);
  const int kd = (p.d + 15) / 16;  // blocks of 16 values of a head
  // columns: S (then P) of the row tiles' halves, O of the row tiles
  const auto s_col = [tmem](int c) { return tmem + c * 64; };
  const auto o_col = [tmem](int t) { return tmem + 256 + t * 64 * DB; };

  if (warp >= kSoftWarps) {
    if (warp == kLoadWarp) {
      if (lane == 0) {
        const uint64_t pol = l2_evict_normal();
        const int q_bytes = w.per * w.group * 128;
        bool ok = true;
        for (int j = 0; j < w.tiles && ok; ++j) {
          const Tile k = w.tile(p, j);
          const int s = j % NS, ph = (j / NS) & 1;
          ok = mbar_wait_soon(&kempty[s], ph ^ 1, p.status, kErrTimeoutProducer);
          if (!ok) break;
          mbar_arrive_expect_tx(&kfull[s], kTile);
#pragma unroll
          for (int d = 0; d < DB; ++d)
            tma_load_4d(Ks + s * kTile + d * 16384, &map_k, &kfull[s], d * 64, k.slot, p.k_s[2] ? w.kvh : 0, p.k_s[0] ? w.b : 0, pol);
          if (j == 0) {
            for (int t = 0; t < 2; ++t) {
              if (!w.active(t)) continue;
              mbar_arrive_expect_tx(&qfull[t], DB * q_bytes);
#pragma unroll
              for (int d = 0; d < DB; ++d)
                tma_load_4d(Q + t * kTile + d * 16384, &map_q, &qfull[t], d * 64, w.kvh * w.group, w.i0(t), w.b, pol);
            }
          }
          ok = mbar_wait_soon(&vempty[s], ph ^ 1, p.status, kErrTimeoutProducer);
          if (!ok) break;
          mbar_arrive_expect_tx(&vfull[s], kTile);
#pragma unroll
          for (int d = 0; d < DB; ++d)
            tma_load_4d(Vs + s * kTile + d * 16384, &map_v, &vfull[s], d * 64, k.slot, p.v_s[2] ? w.kvh : 0, p.v_s[0] ? w.b : 0, pol);
        }
      }
    } else if (warp < kLookWarp) {
      // One warp a row tile.  Its thread only issues: a commit covers all the
      // thread's earlier products, so the scores of a half of key tile j landing
      // tells the softmax warps that its P V of the tile before is done too, and
      // they hand the stages back (keys of j, values of j - 1).  What a half has
      // no keys of the thread hands back itself, in step with the ring.
      const int t = warp - kMmaWarp;
      if (elect_one()) {
        constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
        const uint32_t id_s = idesc_16(bf, 128, kHalf), id_pv = idesc_16(bf, 128, kd * 16, true);
        const uint64_t qd = smem_desc_sw128(smem_u32(Q + t * kTile));
        const uint64_t kd0 = smem_desc_sw128(smem_u32(Ks)), vd0 = value_desc(smem_u32(Vs));
        const uint32_t o_at = o_col(t);
        uint32_t phase = 0;  // of each half's weights
        bool some = false;   // O holds something
        bool see[2] = {false, false};
        uint32_t clean = 0;  // phase of each stage's looked-over barrier
        bool ok = true;
        const auto score = [&](int h, uint64_t kt, int keys) {  // S of a half of the key tile at kt
          const uint32_t id = keys == kHalf ? id_s : idesc_16(bf, 128, (keys + 15) / 16 * 16);
#pragma unroll
          for (int i = 0; i < 4 * DB; ++i) {
            const uint32_t off = ((i >> 2) * 16384 + (i & 3) * 32) >> 4;
            if (i < kd) mma_f16_ss(s_col(2 * t + h), qd + off, kt + h * (kHalf * 128 >> 4) + off, id, i > 0);
          }
          mma_commit(&sfull[2 * t + h]);
        };
        if (w.tiles > 0) {
          const Tile k = w.tile(p, 0);
          const bool any = w.seen(p, t, k);
          ok = mbar_wait_soon(&kfull[0], 0, p.status, kErrTimeoutMma);
          if (ok && w.active(t)) ok = mbar_wait_soon(&qfull[t], 0, p.status, kErrTimeoutMma);
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int keys = keys_of_half(k.count, h);
            see[h] = any && keys > 0;
            if (ok && see[h]) score(h, kd0, keys);
            else mbar_arrive(&kempty[0]);
          }
        }
        int s = 0, ph = 0;
        for (int j = 0; j < w.tiles && ok; ++j) {
          const int s1 = s + 1 == NS ? 0 : s + 1, ph1 = s + 1 == NS ? ph ^ 1 : ph;
          const bool more = j + 1 < w.tiles;
          bool look = false, any1 = more && w.active(t);
          int count = kTileKeys, count1 = kTileKeys;
          if (!w.plain(j)) {
            const Tile k = w.tile(p, j);
            look = w.looked_over(p, k);
            count = k.count;
          }
          if (any1 && !w.plain(j + 1)) {
            const Tile k = w.tile(p, j + 1);
            any1 = w.seen(p, t, k);
            count1 = k.count;
          }
          ok = mbar_wait_soon(&vfull[s], ph, p.status, kErrTimeoutMma);
          if (ok && look) {
            ok = mbar_wait_soon(&vclean[s], clean >> s & 1, p.status, kErrTimeoutMma);
            clean ^= 1u << s;
          }
          if (ok && more) ok = mbar_wait_soon(&kfull[s1], ph1, p.status, kErrTimeoutMma);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (see[h]) {
              if (ok) ok = mbar_wait_soon(&pfull[2 * t + h], phase >> h & 1, p.status, kErrTimeoutMma);
              if (!ok) break;
              phase ^= 1u << h;
              tc_fence_after();
              const uint64_t vt = vd0 + s * (kTile >> 4) + h * (kHalf * 128 >> 4);
              const int steps = (keys_of_half(count, h) + 15) / 16;
#pragma unroll
              for (int i = 0; i < kHalf / 16; ++i)
                if (i < steps) mma_ts(o_at, s_col(2 * t + h) + i * 8, vt + i * (2048 >> 4), id_pv, some || i > 0);
              some = true;
              mma_commit(&pdone[2 * t + h]);
            }
            const int keys1 = keys_of_half(count1, h);
            see[h] = any1 && keys1 > 0;
            if (see[h]) {
              score(h, kd0 + s1 * (kTile >> 4), keys1);
            } else if (more) {
              mma_commit(&vempty[s]);
              mbar_arrive(&kempty[s1]);
            }
          }
          s = s1, ph = ph1;
        }
        mma_commit(&odone[t]);
      }
    } else {
      // look over the values of tiles that some row does not see whole; every
      // tile is waited for and handed back, so that the phases stay in step
      for (int j = 0; j < w.tiles; ++j) {
        const int s = j % NS;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_soon(&vfull[s], (j / NS) & 1, p.status, kErrTimeoutProducer))) break;
        const Tile k = w.tile(p, j);
        if (w.plain(j) || !w.looked_over(p, k)) {
          if (lane == 0) mbar_arrive(&vempty[s]);
          continue;
        }
        if (look_over<T, DB>(Vs + s * kTile, k.count, lane)) *odd = 1;
        fence_proxy_async_smem();
        mbar_arrive(&vclean[s]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&vempty[s]);
      }
    }
  } else {
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the tile = lane of tensor memory
    const int i = w.i0(t) + r / w.group;
    const bool valid = r < w.per * w.group && i < w.nq && w.pq + i >= 0;
    const int pos = valid ? w.pq + i : -1;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c = p.scale * 1.4426950408889634f;  // scores to powers of two
    float top = -INFINITY;  // what P is relative to
    float sum = 0.f;
    uint32_t phase = 0;  // of each half's scores
    int last = -1;       // the half whose weights went out last
    bool ok = true;
    const int tiles = w.active(t) ? w.tiles : 0;
    for (int j = 0; j < tiles && ok; ++j) {
      Tile k;
      k.count = kTileKeys;
      bool whole = true;
      if (!w.plain(j)) {
        k = w.tile(p, j);
        if (!w.seen(p, t, k)) continue;
        whole = w.whole(p, t, k);
      }
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int keys = keys_of_half(k.count, h);
        if (keys == 0) break;
        const uint32_t sc = s_col(2 * t + h) + lanes;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_soon(&sfull[2 * t + h], phase >> h & 1, p.status, kErrTimeoutEpilogue));
        if (!ok) break;
        phase ^= 1u << h;
        tc_fence_after();
        if ((warp & 3) == 0) {  // (whole warps: what follows reads tensor memory)
          mbar_arrive_if(lane == 0, &kempty[j % NS]);
          if (j > 0) mbar_arrive_if(lane == 0, &vempty[(j - 1) % NS]);
        }
        uint32_t raw[2][32];
        tmem_ld32_nowait(sc, raw[0]);
        tmem_ld32_nowait(sc + 32, raw[1]);
        tmem_wait_ld();
        if (!whole) {
          // columns lo .. hi, and the sinks
          const int hi = min(k.count - 1, pos - k.pos) - h * kHalf;
          const int lo = (p.window == 0 ? 0 : max(pos - p.window + 1 - k.pos, 0)) - h * kHalf;
          const int sk = min(p.sinks - k.pos - h * kHalf, hi + 1);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t bits = (below(hi + 1 - q * 32) & ~below(lo - q * 32)) | below(sk - q * 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) raw[q][e] = bits >> e & 1u ? raw[q][e] : 0xFF800000u;
          }
        }
        float m4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t* v = raw[q >> 1] + (q & 1) * 16;
          m4[q] = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
          for (int e = 2; e < 16; e += 2) m4[q] = max3(m4[q], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        }
        const float m = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
        // (lanes without a query hold whatever shared memory held, and must not
        // decide for the others)
        const bool rise = valid && (m - top) * c > 8.f;
        if (__any_sync(0xFFFFFFFFu, rise)) {
          const float up = fmaxf(m, top);
          const float f = up == -INFINITY ? 1.f : exp2_fast((top - up) * c);
          top = up;
          sum *= f;
          if (last >= 0) {  // the last P V must be done
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_soon(&pdone[2 * t + last], (phase >> last & 1) ^ 1 ^ (last == h), p.status,
                                                        kErrTimeoutEpilogue));
            if (!ok) break;
            tc_fence_after();
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
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q * 32 < keys) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = f2_of(fma2(f2(__uint_as_float(raw[q][e]), __uint_as_float(raw[q][e + 1])), c2, b2));
              const float u = exp2_fast(x.x), v = exp2_fast(x.y);
              acc[(e >> 1) & 1] = add2(acc[(e >> 1) & 1], f2(u, v));
              pk[e / 2] = pack2<T>(u, v);
            }
            tmem_st16(sc + q * 16, pk);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&pfull[2 * t + h]);
        const float2 a = f2_of(add2(acc[0], acc[1]));
        sum += a.x + a.y;
        last = h;
      }
    }
    // What follows writes over the queries: wait for the last product, or, where the
    // row tile saw no key tile (a prompt longer than the ring), for their load.
    if (tiles > 0 && ok) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_soon(last >= 0 ? &odone[t] : &qfull[t], 0, p.status, kErrTimeoutEpilogue));
      tc_fence_after();
    }
    // output: through the row tile's query tile, which no product reads any more
    const bool some = valid && last >= 0 && !(sum == 0.f);
    const float inv = some ? 1.f / sum : 0.f;
    uint8_t* out = Q + t * kTile;
#pragma unroll 1
    for (int x = 0; x < DB * 64; x += 32) {
      if (x >= p.d) break;
      uint32_t o[32];
      if (last >= 0) {
        tmem_ld32_nowait(o_col(t) + lanes + x, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = some ? __uint_as_float(o[q * 8 + e]) * inv : 0.f;
        const int pc = (x % 64) / 8 + q;
        *reinterpret_cast<uint4*>(out + (x / 64) * 16384 + r * 128 + ((pc ^ (r & 7)) << 4)) = Vec16<T>::pack(v);
      }
    }
    if (p.lse && r < w.per * w.group && i < p.tq) {
      const int h = w.kvh * w.group + r % w.group;
      p.lse[(static_cast<int64_t>(w.b) * p.hq + h) * p.tq + i] =
          some ? (top * c - kLift<T> + log2f(sum)) * 0.69314718055994531f : -INFINITY;
    }
    fence_proxy_async_smem();
    __syncwarp();  // (the barrier takes whole warps)
    named_barrier_sync(1 + t, 128);
    if (r == 0 && w.i0(t) < p.tq) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
        if (d * 64 < p.d) tma_store_4d(&map_o, out + d * 16384, d * 64, w.kvh * w.group, w.i0(t), w.b);
      bulk_commit();
      bulk_wait_read<0>();  // the tile must outlive the store's reads
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (*odd) {
    // a key's value is no number: every row again, on its own, over what the
    // stores have written
    bulk_wait_all();
    __syncthreads();
    for (int r = warp; r < 2 * w.per * w.group; r += kThreads / 32) {
      const int i = w.i00 + r / w.group;
      if (i < p.tq) attend_row<T, 2 * DB>(p, w.b, i, w.kvh * w.group + r % w.group, lane);
    }
  }
}

template <typename T> cudaError_t launch(const AttnLaunch& L, cudaStream_t stream) {
  static Kernel handle;
  return handle.launch(attn_prompt_kernel<T>, L.device, dim3(L.grid), kThreads, kSmem, 1, stream, L.map_q, L.map_k,
                       L.map_v, L.map_o, L.p);
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnLaunch& L, bool bf16, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(L, stream) : launch<__half>(L, stream);
}

}  // namespace oidnx
