// Window attention for prompts, heads of up to 64 values: the plan, operands and
// rules of attn_prompt.cu, with the halves of a key tile as chains of their own.
//
// Bound by a chain's latency: scores to weights to the next scores, some 2300
// cycles for 64 keys, of which the softmax warps take 1400.  Tensor memory has
// room for a chain per row tile and half of each key tile: 64 columns of scores
// and 64 of output each.  The halves of a row keep their own maximum, sum and
// output, sixteen softmax warps work at once, and the halves are joined at the
// end.  2 x 4096 causal, 8 heads of 64: 46 us (one chain a row tile: 54), 740
// TFLOP/s of visible pairs; the longest CTA's 32 key tiles are what remains.
//
// Warps 4 c .. 4 c + 3: softmax of chain c = 2 (row tile) + (half of the keys),
// one thread a row; warp 16 loads, 17 and 18 issue the products of a row tile's
// two chains each, 19 looks values over.
#include "attn_prompt.cuh"

namespace oidnx {
namespace {

constexpr int kSoftWarps = 16;
constexpr int kThreads = (kSoftWarps + 4) * 32;
constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kLookWarp = kSoftWarps + 3;
constexpr int kOperand = 16384;  // 128 rows of 64 values
constexpr int NS = 4;            // key tiles (and value tiles) in flight
constexpr int kSmem = (2 + 2 * NS) * kOperand + 1024 + 512 + 4 * 128 * 8;

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt64_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                         const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* Q = smem_raw + pad;  // [2 row tiles]; the output tiles at the end
  uint8_t* Ks = Q + 2 * kOperand;
  uint8_t* Vs = Ks + NS * kOperand;
  float2* stats = reinterpret_cast<float2*>(Vs + NS * kOperand);  // [chain][row]: maximum and sum, at the end
  uint64_t* qfull = reinterpret_cast<uint64_t*>(stats + 4 * 128);  // [2]
  uint64_t* kfull = qfull + 2;    // [NS]
  uint64_t* kempty = kfull + NS;
  uint64_t* vfull = kempty + NS;
  uint64_t* vempty = vfull + NS;
  uint64_t* sfull = vempty + NS;  // [4]
  uint64_t* pfull = sfull + 4;    // [4]
  uint64_t* odone = pfull + 4;    // [2]
  uint64_t* vclean = odone + 2;   // [NS]
  uint32_t* slot = reinterpret_cast<uint32_t*>(vclean + NS);
  int* odd = reinterpret_cast<int*>(slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 4);  // the chains
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 5);  // and the looking warp
      mbar_init(&vclean[s], 32);
    }
    for (int c = 0; c < 4; ++c) {
      mbar_init(&sfull[c], 1);
      mbar_init(&pfull[c], 128);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&qfull[t], 1);
      mbar_init(&odone[t], 1);
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
  // columns: S (then P) of the chains, O of the chains
  const auto s_col = [tmem](int c) { return tmem + c * 64; };
  const auto o_col = [tmem](int c) { return tmem + 256 + c * 64; };

  if (warp == kLoadWarp) {
    if (lane == 0) {
      const uint64_t pol = l2_evict_normal();
      bool ok = true;
      for (int j = 0; j < w.tiles && ok; ++j) {
        const Tile k = w.tile(p, j);
        const int s = j % NS, ph = (j / NS) & 1;
        ok = mbar_wait_soon(&kempty[s], ph ^ 1, p.status, kErrTimeoutProducer);
        if (!ok) break;
        mbar_arrive_expect_tx(&kfull[s], kOperand);
        tma_load_4d(Ks + s * kOperand, &map_k, &kfull[s], 0, k.slot, p.k_s[2] ? w.kvh : 0, p.k_s[0] ? w.b : 0, pol);
        if (j == 0) {
          for (int t = 0; t < 2; ++t) {
            if (!w.active(t)) continue;
            mbar_arrive_expect_tx(&qfull[t], w.per * w.group * 128);
            tma_load_4d(Q + t * kOperand, &map_q, &qfull[t], 0, w.kvh * w.group, w.i0(t), w.b, pol);
          }
        }
        ok = mbar_wait_soon(&vempty[s], ph ^ 1, p.status, kErrTimeoutProducer);
        if (!ok) break;
        mbar_arrive_expect_tx(&vfull[s], kOperand);
        tma_load_4d(Vs + s * kOperand, &map_v, &vfull[s], 0, k.slot, p.v_s[2] ? w.kvh : 0, p.v_s[0] ? w.b : 0, pol);
      }
    }
  } else if (warp == kLookWarp) {
    // every value tile is waited for and handed back, so that the phases stay in step
    for (int j = 0; j < w.tiles; ++j) {
      const int s = j % NS;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_soon(&vfull[s], (j / NS) & 1, p.status, kErrTimeoutProducer))) break;
      const Tile k = w.tile(p, j);
      if (!w.plain(j) && w.looked_over(p, k)) {
        if (look_over<T, 1>(Vs + s * kOperand, k.count, lane)) *odd = 1;
        fence_proxy_async_smem();
        mbar_arrive(&vclean[s]);
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&vempty[s]);
    }
  } else if (warp >= kMmaWarp) {
    // The scores of key tile j landing tells a chain's softmax warps that its P V
    // of the tile before is done too (a commit covers all the thread's earlier
    // products); they hand the stages back (keys of j, values of j - 1).  What a
    // chain has no keys of, the thread hands back itself, in step with the ring.
    const int t = warp - kMmaWarp;
    if (elect_one()) {
      constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
      const uint32_t id_s = idesc_16(bf, 128, kHalf), id_pv = idesc_16(bf, 128, kd * 16, true);
      const uint64_t qd = smem_desc_sw128(smem_u32(Q + t * kOperand));
      const uint64_t kd0 = smem_desc_sw128(smem_u32(Ks)), vd0 = value_desc(smem_u32(Vs));
      int n[2] = {0, 0};
      bool see[2] = {false, false};
      uint32_t clean = 0;  // phase of each stage's looked-over barrier
      bool ok = true;
      const auto score = [&](int h, uint64_t kt, int keys) {  // S of a half of the key tile at kt
        const uint32_t id = keys == kHalf ? id_s : idesc_16(bf, 128, (keys + 15) / 16 * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < kd) mma_f16_ss(s_col(2 * t + h), qd + i * 2, kt + h * (kHalf * 128 >> 4) + i * 2, id, i > 0);
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
            if (ok) ok = mbar_wait_soon(&pfull[2 * t + h], n[h] & 1, p.status, kErrTimeoutMma);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vt = vd0 + s * (kOperand >> 4) + h * (kHalf * 128 >> 4);
            const int steps = (keys_of_half(count, h) + 15) / 16;
#pragma unroll
            for (int i = 0; i < kHalf / 16; ++i)
              if (i < steps)
                mma_ts(o_col(2 * t + h), s_col(2 * t + h) + i * 8, vt + i * (2048 >> 4), id_pv, n[h] > 0 || i > 0);
            ++n[h];
          }
          const int keys1 = keys_of_half(count1, h);
          see[h] = any1 && keys1 > 0;
          if (see[h]) {
            score(h, kd0 + s1 * (kOperand >> 4), keys1);
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
    const int chain = warp >> 2, t = chain >> 1, h = chain & 1;
    const int r = threadIdx.x & 127;  // row of the tile = lane of tensor memory
    const int i = w.i0(t) + r / w.group;
    const bool valid = r < w.per * w.group && i < w.nq && w.pq + i >= 0;
    const int pos = valid ? w.pq + i : -1;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t sc = s_col(chain) + lanes, oc = o_col(chain) + lanes;
    const float c = p.scale * 1.4426950408889634f;  // scores to powers of two
    float top = -INFINITY;  // what P is relative to
    float sum = 0.f;
    int n = 0;
    bool ok = true;
    const int tiles = w.active(t) ? w.tiles : 0;
    for (int j = 0; j < tiles && ok; ++j) {
      Tile k;
      int keys = kHalf;
      bool whole = true;
      if (!w.plain(j)) {
        k = w.tile(p, j);
        keys = keys_of_half(k.count, h);
        if (keys == 0 || !w.seen(p, t, k)) continue;
        whole = w.whole(p, t, k);
      }
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_soon(&sfull[chain], n & 1, p.status, kErrTimeoutEpilogue));
      if (!ok) break;
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
        if (n > 0) {  // (the last P V is done: these scores were committed behind it)
#pragma unroll 1
          for (int x = 0; x < kd * 16; x += 16) {
            uint32_t o[16];
            tmem_ld16_nowait(oc + x, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(oc + x, o);
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
      mbar_arrive(&pfull[chain]);
      const float2 a = f2_of(add2(acc[0], acc[1]));
      sum += a.x + a.y;
      ++n;
    }
    // the halves' maxima and sums meet; each half writes 32 values of the row
    ok = __all_sync(0xFFFFFFFFu, mbar_wait_soon(&odone[t], 0, p.status, kErrTimeoutEpilogue));
    tc_fence_after();
    stats[chain * 128 + r] = make_float2(top, sum);
    __syncwarp();  // (the barrier takes whole warps)
    named_barrier_sync(1 + t, 256);
    const float2 a = stats[2 * t * 128 + r], b = stats[(2 * t + 1) * 128 + r];
    const bool has_a = !(a.y == 0.f), has_b = !(b.y == 0.f);
    const float both = fmaxf(a.x, b.x), at = both == -INFINITY ? 0.f : both;
    const float fa = has_a ? exp2_fast((a.x - at) * c) : 0.f, fb = has_b ? exp2_fast((b.x - at) * c) : 0.f;
    const float total = (has_a ? a.y * fa : 0.f) + (has_b ? b.y * fb : 0.f);
    const bool some = valid && (has_a || has_b);
    const float inv = some ? 1.f / total : 0.f;
    const float wa = fa * inv, wb = fb * inv;
    uint8_t* out = Q + t * kOperand;
    if (h * 32 < p.d) {
      uint32_t oa[32], ob[32];
      tmem_ld32_nowait(o_col(2 * t) + lanes + h * 32, oa);
      tmem_ld32_nowait(o_col(2 * t + 1) + lanes + h * 32, ob);
      tmem_wait_ld();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = some && has_a ? __uint_as_float(oa[q * 8 + e]) * wa : 0.f;
          v[e] = some && has_b ? fmaf(__uint_as_float(ob[q * 8 + e]), wb, x) : x;
        }
        const int piece = h * 4 + q;
        *reinterpret_cast<uint4*>(out + r * 128 + ((piece ^ (r & 7)) << 4)) = Vec16<T>::pack(v);
      }
    }
    if (p.lse && h == 0 && r < w.per * w.group && i < p.tq) {
      const int head = w.kvh * w.group + r % w.group;
      p.lse[(static_cast<int64_t>(w.b) * p.hq + head) * p.tq + i] =
          some ? (both * c - kLift<T> + log2f(total)) * 0.69314718055994531f : -INFINITY;
    }
    fence_proxy_async_smem();
    __syncwarp();
    named_barrier_sync(1 + t, 256);
    if (r == 0 && h == 0 && w.i0(t) < p.tq) {
      tma_store_4d(&map_o, out, 0, w.kvh * w.group, w.i0(t), w.b);
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
      if (i < p.tq) attend_row<T, 2>(p, w.b, i, w.kvh * w.group + r % w.group, lane);
    }
  }
}

template <typename T> cudaError_t launch(const AttnLaunch& L, cudaStream_t stream) {
  static Kernel handle;
  return handle.launch(attn_prompt64_kernel<T>, L.device, dim3(L.grid), kThreads, kSmem, 1, stream, L.map_q, L.map_k,
                       L.map_v, L.map_o, L.p);
}

}  // namespace

cudaError_t launch_attn_prompt64(const AttnLaunch& L, bool bf16, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(L, stream) : launch<__half>(L, stream);
}

}  // namespace oidnx
