// Entry points of a conditioned block's operators: argument checks and the choice
// of kernel, as in token_host.cpp.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <limits>

#include "cross.h"
#include "token_host.h"

using namespace oidnx;

namespace {

int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }

// ---------------------------------------------------------------- cross attention: choice of form
struct Dims {
  int n[3];  // sequences, tokens, heads
};

// Whether heads can be moved as they lie: in 16-byte pieces, by a tensor map, whose
// strides are positive and below 2^40 bytes.  Bits of `shared`: dimensions
// that may be shared (stride 0).
bool fits(const void* p, const int64_t* s, int d, unsigned shared) {
  bool ok = d % 8 == 0 && aligned(p, 16);
  for (int i = 0; i < 3; ++i)
    ok = ok && s[i] % 8 == 0 && s[i] < int64_t(1) << 38 && (s[i] > 0 || (s[i] == 0 && shared >> i & 1u));
  return ok;
}

int64_t bytes_of_copy(const int64_t* s, const Dims& n, int64_t ld, unsigned shared) {  // shared dimensions once
  int64_t all = 2 * ld;
  for (int i = 0; i < 3; ++i) all *= s[i] == 0 && shared >> i & 1u ? 1 : n.n[i];
  return all;
}

struct Tiles {
  int tiles = 1, blocks = 0, items = 0, whole = 0, cluster = 1, grid = 0;
  double cost = INFINITY;  // ns
};

// Bytes of queries, keys, values and output at 6.2 TB/s, ns.
double traffic_ns(const CrossParams& p) {
  return 2.0 * p.d * p.b * (2.0 * p.kv * p.hk + 2.0 * p.tq * p.hq) / 6200;
}

// Many queries: rounds of resident CTAs times an item's units of 64 keys, and its
// ends; what does not fill a round divided over clusters of 2 to 8, if they all fit.
// Measured, us a unit of one, two and four row tiles: heads of 64 values 0.85, 0.91,
// 1.30; of 128 0.60, 0.78; of 256 1.6.  8160 queries and keys, 16 heads of 128: 398 in
// four rounds, 363 with the last divided by two; 8 heads of 64 over 2040 keys: two row
// tiles 36, divided by two 27.
Tiles plan_tiles(const CrossParams& p, bool bf16, int device, int sms) {
  Tiles best;
  if (p.group > 128 || p.kv == 0) return best;
  const int per = 128 / p.group, most = cross_most_tiles(p.d);
  const int64_t row_tiles = (static_cast<int64_t>(p.tq) + per - 1) / per;
  const double units = std::max(1, (p.kv + 63) / 64);
  static const double unit_ns[3][3] = {{850, 910, 1300}, {600, 780, 0}, {1600, 0, 0}};
  const double start_ns = 3000, item_ns = 3000, join_ns = 4000;
  for (int tiles = 1, at = 0; tiles <= most; tiles *= 2, ++at) {
    const int64_t blocks = (row_tiles + tiles - 1) / tiles, items = blocks * p.b * p.hk;
    if (items > INT_MAX / 2) continue;
    const double unit = unit_ns[p.d <= 64 ? 0 : p.d <= 128 ? 1 : 2][at];
    for (int cluster = 1; cluster <= 8; cluster *= 2) {
      const int slots = cluster == 1 ? sms : cross_tile_slots(p.d, bf16, cluster, device);
      if (slots <= 0) continue;
      int64_t whole = items, rest = 0;
      if (cluster > 1) {
        whole = items / slots * slots, rest = items - whole;
        if (rest == 0 || rest > slots / cluster || units < 2 * cluster) continue;
      }
      const double rounds = std::ceil(static_cast<double>(whole) / slots);
      double cost = start_ns + rounds * (item_ns + units * unit);
      if (rest) cost += item_ns + join_ns + units / cluster * unit;
      cost = std::max(cost, start_ns + traffic_ns(p));
      if (cost < best.cost) {
        best.tiles = tiles, best.blocks = static_cast<int>(blocks), best.items = static_cast<int>(items);
        best.whole = static_cast<int>(whole), best.cluster = cluster;
        best.grid = static_cast<int>(whole ? std::min<int64_t>(slots, whole) : rest * cluster);
        best.cost = cost;
      }
    }
  }
  return best;
}

struct Parts {
  int split = 1, parts = 1;
  double cost = INFINITY;
};

// Few queries: rounds of resident CTAs times a CTA's keys, and its start.  Measured,
// us, 16 rows: heads of 64 values 4.3 + 3.7 a thousand keys, of 128 5.0 + 6.8, of 256
// 6.4 + 13.3; 32 rows 8.2 + 4.8 and 9.5 + 11.  Keys divided over as many CTAs as fit
// where clusters leave SMs idle: 20000 keys, 8 key heads of 128 21.9 -> 19, one 20.6 ->
// 10.2 in 38 parts; more of them cost their join (152: 12.1), so a part has 512 keys.
Parts plan_parts(const CrossParams& p, bool bf16, int device) {
  Parts best;
  const int64_t rows = static_cast<int64_t>(p.tq) * p.group;
  const int per = rows > 16 && p.d <= 128 ? 32 : 16;
  const int64_t row_tiles = (rows + per - 1) / per, units = static_cast<int64_t>(p.b) * p.hk * row_tiles;
  const double key = p.d <= 64 ? (per == 32 ? 4.8 : 3.7) : p.d <= 128 ? (per == 32 ? 11 : 6.8) : 13.3;
  const double start = p.d <= 64 ? (per == 32 ? 8200 : 4300) : p.d <= 128 ? (per == 32 ? 9500 : 5000) : 6400;
  const double least = start + traffic_ns(p);
  double joining = 1500;  // 500 for each doubling
  int slots = 0;
  for (int split = 8; split >= 1; split /= 2) {
    slots = cross_token_slots(p, bf16, split, device);
    if (slots <= 0 || units * split > INT_MAX) continue;
    const double rounds = std::ceil(static_cast<double>(units) * split / slots);
    const double cost = std::max(rounds * (static_cast<double>(p.kv) / split * key + start), least) + joining;
    joining -= 500;
    if (cost <= best.cost) best.cost = cost, best.split = split, best.parts = 1;
  }
  const int parts = static_cast<int>(std::min<int64_t>(slots / units, (p.kv + 511) / 512));
  if (parts > 8) {
    const double cost = std::max(static_cast<double>(p.kv) / parts * key + start, least) + 3000;
    if (cost < best.cost) best.cost = cost, best.split = 1, best.parts = parts;
  }
  return best;
}

cudaError_t run_tiles(const CrossParams& p, const Tiles& t, bool bf16, int device, cudaStream_t stream) {
  CrossTileLaunch L = {};
  L.p = p;
  L.per = 128 / p.group, L.tiles = t.tiles, L.blocks = t.blocks, L.items = t.items;
  L.whole = t.whole, L.cluster = t.cluster, L.grid = t.grid, L.device = device;
  const int keys = p.d <= 128 ? 128 : 64;
  // a shared dimension has one element, which the kernel reads for all
  const int64_t any = round8(p.d);
  const auto cache_map = [&](CUtensorMap* map, const void* base, const int64_t* s) {
    return heads_map(map, bf16, base, p.d, p.kv, s[1], s[2] ? p.hk : 1, s[2] ? s[2] : any, s[0] ? p.b : 1, s[0] ? s[0] : any,
                     keys, 1);
  };
  if (!heads_map(&L.map_q, bf16, p.q, p.d, p.hq, p.q_s[2], p.tq, p.q_s[1], p.q_s[0] ? p.b : 1, p.q_s[0] ? p.q_s[0] : any,
                 p.group, L.per) ||
      !heads_map(&L.map_o, bf16, p.o, p.d, p.hq, p.o_s[2], p.tq, p.o_s[1], p.b, p.o_s[0], p.group, L.per) ||
      !cache_map(&L.map_k, p.k, p.k_s) || !cache_map(&L.map_v, p.v, p.v_s))
    return cudaErrorInvalidValue;
  return launch_cross_tile(L, bf16, stream);
}

// Memory of one call, ordered on its stream.
struct Scratch {
  void* at = nullptr;
  cudaStream_t stream = nullptr;
  cudaError_t take(int device, int64_t bytes, cudaStream_t s) {
    cudaMemPool_t pool;
    cudaError_t e = token_pool(device, &pool);
    if (e == cudaSuccess) e = cudaMallocFromPoolAsync(&at, bytes, pool, s);
    if (e != cudaSuccess) at = nullptr;
    stream = s;
    return e;
  }
  cudaError_t give() {
    void* p = at;
    at = nullptr;
    return p ? cudaFreeAsync(p, stream) : cudaSuccess;
  }
};

cudaError_t run_aligned(CrossParams& p, bool bf16, int device, int sms, cudaStream_t stream) {
  const Parts parts = plan_parts(p, bf16, device);
  const Tiles tiles = plan_tiles(p, bf16, device, sms);
  if (tiles.cost < parts.cost) return run_tiles(p, tiles, bf16, device, stream);
  if (parts.cost == INFINITY) return cudaErrorInvalidValue;
  CrossTokenLaunch L = {};
  L.p = p, L.split = parts.split, L.parts = parts.parts, L.device = device;
  if (parts.parts == 1) return launch_cross_token(L, bf16, stream);
  Scratch work;
  cudaError_t e = work.take(device, static_cast<int64_t>(p.b) * p.hq * p.tq * parts.parts * cross_part_floats(p.d) * 4, stream);
  if (e != cudaSuccess) return e;
  L.work = static_cast<float*>(work.at);
  e = launch_cross_token(L, bf16, stream);
  const cudaError_t freed = work.give();
  return e != cudaSuccess ? e : freed;
}

cudaError_t run_cross(CrossParams& p, int precision, cudaStream_t stream) {
  int device, sms;
  cudaError_t e = token_device(&device, &sms, &p.status);
  if (e != cudaSuccess) return e;
  const bool bf16 = precision == OIDNX_PRECISION_BF16;
  const int64_t ld = round8(p.d);
  // the stride of a dimension of one element says nothing
  if (p.b == 1) p.q_s[0] = p.k_s[0] = p.v_s[0] = p.o_s[0] = ld;
  if (p.tq == 1) p.q_s[1] = p.o_s[1] = ld;
  if (p.kv == 1) p.k_s[1] = p.v_s[1] = ld;
  if (p.hq == 1) p.q_s[2] = p.o_s[2] = ld;
  if (p.hk == 1) p.k_s[2] = p.v_s[2] = ld;
  const bool negative = p.scale < 0.f;
  // The smallest number of fp32 for 0: a product with -infinity stays one, and the largest score
  // comes to 5e-7, less than a weight can show.
  if (p.scale == 0.f) p.scale = std::numeric_limits<float>::denorm_min();
  constexpr unsigned kSequences = 1, kHeads = 4;
  const bool move_q = negative || !fits(p.q, p.q_s, p.d, kSequences);
  const bool move_k = p.kv > 0 && !fits(p.k, p.k_s, p.d, kSequences | kHeads);
  const bool move_v = p.kv > 0 && !fits(p.v, p.v_s, p.d, kSequences | kHeads), move_o = !fits(p.o, p.o_s, p.d, 0);
  if (!move_q && !move_k && !move_v && !move_o) return run_aligned(p, bf16, device, sms, stream);

  const Dims nq = {{p.b, p.tq, p.hq}}, nk = {{p.b, p.kv, p.hk}};
  const int64_t q_bytes = move_q ? bytes_of_copy(p.q_s, nq, ld, kSequences) : 0;
  const int64_t k_bytes = move_k ? bytes_of_copy(p.k_s, nk, ld, kSequences | kHeads) : 0;
  const int64_t v_bytes = move_v ? bytes_of_copy(p.v_s, nk, ld, kSequences | kHeads) : 0;
  const int64_t o_bytes = move_o ? 2 * ld * p.b * p.tq * p.hq : 0;
  Scratch memory;
  e = memory.take(device, q_bytes + k_bytes + v_bytes + o_bytes, stream);
  if (e != cudaSuccess) return e;
  uint8_t* at = static_cast<uint8_t*>(memory.at);
  HeadsCopy copies[3] = {};
  int count = 0;
  const int d = p.d;
  const auto move = [&](const void** base, int64_t* s, const Dims& n, int64_t bytes, unsigned shared, bool negate) {
    HeadsCopy& c = copies[count++];
    c.from = *base, c.to = at, c.d = d, c.d_to = static_cast<int>(ld), c.negate = negate;
    int64_t step = ld;
    for (int i = 2; i >= 0; --i) {
      const bool once = s[i] == 0 && shared >> i & 1u;
      c.from_s[i] = s[i], c.n[i] = once ? 1 : n.n[i];
      c.to_s[i] = once ? 0 : step;
      step *= c.n[i];
    }
    for (int i = 0; i < 3; ++i) s[i] = c.to_s[i];
    *base = at;
    at += bytes;
  };
  if (move_q) move(&p.q, p.q_s, nq, q_bytes, kSequences, negative);
  if (move_k) move(&p.k, p.k_s, nk, k_bytes, kSequences | kHeads, false);
  if (move_v) move(&p.v, p.v_s, nk, v_bytes, kSequences | kHeads, false);
  if (negative) p.scale = -p.scale;
  void* out = p.o;
  int64_t out_s[3] = {p.o_s[0], p.o_s[1], p.o_s[2]};
  if (move_o) {
    p.o = at;
    p.o_s[2] = ld, p.o_s[1] = ld * p.hq, p.o_s[0] = p.o_s[1] * p.tq;
  }
  if (count) e = launch_heads_copy(copies, count, device, sms, stream);
  p.d = static_cast<int>(ld);
  if (e == cudaSuccess) e = run_aligned(p, bf16, device, sms, stream);
  if (e == cudaSuccess && move_o) {
    HeadsCopy c = {};
    c.from = p.o, c.to = out, c.d = c.d_to = d;
    for (int i = 0; i < 3; ++i) c.from_s[i] = p.o_s[i], c.to_s[i] = out_s[i], c.n[i] = nq.n[i];
    e = launch_heads_copy(&c, 1, device, sms, stream);
  }
  const cudaError_t freed = memory.give();
  return e != cudaSuccess ? e : freed;
}

}  // namespace

extern "C" {

oidnx_status oidnx_block_norm(const void* x, long long ldx, const void* residual, long long ldr, void* sum,
                              long long ld_sum, void* y, long long ldy, int post, const void* post_weight,
                              const void* post_bias, int pre, const void* pre_weight, const void* pre_bias, float eps,
                              const void* gate, long long ldg, int gate_act, const void* scale, long long lds,
                              const void* shift, long long ldh, const int* groups, int per, int count,
                              float residual_scale, float branch_scale, int t, int n, int precision, int sum_precision,
                              void* stream) {
  if (precision < OIDNX_PRECISION_FP32 || precision > OIDNX_PRECISION_BF16)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: unknown precision %d", precision);
  if (sum_precision == OIDNX_PRECISION_AUTO) sum_precision = precision;
  if (sum_precision != precision && sum_precision != OIDNX_PRECISION_FP32)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: the sum is of the values' precision or fp32, not %d", sum_precision);
  if (t < 0 || n < 0 || count < 0) return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: negative size (%d, %d, %d)", t, n, count);
  if (post < OIDNX_NORM_NONE || post > OIDNX_NORM_LAYER || pre < OIDNX_NORM_NONE || pre > OIDNX_NORM_LAYER)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: unknown norm (%d, %d)", post, pre);
  if (gate_act < OIDNX_GATE_PLAIN || gate_act > OIDNX_GATE_SIGMOID)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: unknown gate activation %d", gate_act);
  if (!groups && per <= 0) return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: %d rows a group", per);
  if (!(eps >= 0.f) || std::isinf(eps) || !std::isfinite(residual_scale) || !std::isfinite(branch_scale))
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: bad eps or factors");
  if (t > kMost || n > kMost) return fail(OIDNX_ERR_UNSUPPORTED, "block_norm: a size beyond 2^30");
  if (t == 0 || n == 0 || count == 0) return finish(cudaSuccess, "block_norm");
  if (!x || (!sum && !y)) return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: NULL x, or no output");
  if (ldx < n || (residual && ldr < n) || (sum && ld_sum < n) || (y && ldy < n) || (gate && ldg && ldg < n) ||
      (scale && lds && lds < n) || (shift && ldh && ldh < n))
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: a row stride is shorter than its row");
  const int size = precision == OIDNX_PRECISION_FP32 ? 4 : 2, held = sum_precision == OIDNX_PRECISION_FP32 ? 4 : 2;
  const struct {
    const void* p;
    int64_t ld;
    int size;
  } all[] = {{x, ldx, size}, {residual, ldr, held}, {sum, ld_sum, held}, {y, ldy, size}, {post_weight, 0, size},
             {post_bias, 0, size}, {pre_weight, 0, size}, {pre_bias, 0, size}, {gate, ldg, size}, {scale, lds, size},
             {shift, ldh, size}};
  bool vector = n % 8 == 0;
  for (const auto& a : all) {
    if (!aligned(a.p, a.size)) return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: pointers must be aligned to their elements");
    if (a.p) vector = vector && aligned(a.p, 16) && a.ld * a.size % 16 == 0;
  }
  if (!aligned(groups, 4)) return fail(OIDNX_ERR_INVALID_ARGUMENT, "block_norm: groups must be 4-byte aligned");
  BlockParams p = {};
  p.x = x, p.residual = residual, p.sum = sum, p.y = y;
  p.ldx = ldx, p.ldr = ldr, p.ld_sum = ld_sum, p.ldy = ldy;
  // without a norm there is nothing that its weight and bias go to
  if (post != OIDNX_NORM_NONE) p.weight[0] = post_weight, p.bias[0] = post_bias;
  if (pre != OIDNX_NORM_NONE) p.weight[1] = pre_weight, p.bias[1] = pre_bias;
  p.gate = gate, p.scale = scale, p.shift = shift;
  p.ldg = ldg, p.lds = lds, p.ldh = ldh;
  p.groups = groups, p.per = per, p.count = count;
  p.norm[0] = post, p.norm[1] = pre, p.gate_act = gate_act;
  p.eps = eps, p.alpha = residual_scale, p.beta = branch_scale;
  p.t = t, p.n = n;
  int device, sms, *status;
  cudaError_t e = token_device(&device, &sms, &status);
  if (e == cudaSuccess) e = launch_block_norm(p, vector, precision, sum_precision, device, sms, static_cast<cudaStream_t>(stream));
  return finish(e, "block_norm");
}

oidnx_status oidnx_cross_attention(const void* q, long long q_sb, long long q_st, long long q_sh, const void* k,
                                   long long k_sb, long long k_st, long long k_sh, const void* v, long long v_sb,
                                   long long v_st, long long v_sh, void* o, long long o_sb, long long o_st, long long o_sh,
                                   float* lse, const int* q_lens, const int* kv_lens, const unsigned char* mask,
                                   long long mask_sb, int b, int tq, int kv, int hq, int hk, int d, float scale,
                                   int precision, void* stream) {
  if (precision == OIDNX_PRECISION_FP32) return fail(OIDNX_ERR_UNSUPPORTED, "cross_attention: fp16 or bf16 only");
  if (precision != OIDNX_PRECISION_FP16 && precision != OIDNX_PRECISION_BF16)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "cross_attention: unknown precision %d", precision);
  if (b < 0 || tq < 0 || kv < 0 || hq < 0 || hk <= 0 || hq % hk || d <= 0)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "cross_attention: bad sizes (b %d, tq %d, kv %d, heads %d and %d, d %d)", b, tq,
                kv, hq, hk, d);
  if (tq > kMost || kv > kMost) return fail(OIDNX_ERR_UNSUPPORTED, "cross_attention: a length beyond 2^30");
  if (d > 256) return fail(OIDNX_ERR_UNSUPPORTED, "cross_attention: heads of more than 256 values (%d)", d);
  if (!std::isfinite(scale)) return fail(OIDNX_ERR_INVALID_ARGUMENT, "cross_attention: scale is not finite");
  if (mask && mask_sb != 0 && mask_sb < kv)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "cross_attention: the mask's stride is shorter than its row");
  if (b == 0 || tq == 0 || hq == 0) return finish(cudaSuccess, "cross_attention");
  if (static_cast<double>(b) * tq * hq > 4e9)
    return fail(OIDNX_ERR_UNSUPPORTED, "cross_attention: more than 4e9 query heads");
  if (static_cast<int64_t>(tq) * (hq / hk) > kMost)
    return fail(OIDNX_ERR_UNSUPPORTED, "cross_attention: more than 2^30 queries of a key head");
  if (!q || !o || (kv > 0 && (!k || !v))) return fail(OIDNX_ERR_INVALID_ARGUMENT, "cross_attention: NULL q, k, v or o");
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(o, 2) || !aligned(lse, 4) || !aligned(q_lens, 4) ||
      !aligned(kv_lens, 4))
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "cross_attention: pointers must be aligned to their elements");
  CrossParams p = {};
  p.q = q, p.k = k, p.v = v, p.o = o, p.lse = lse, p.q_lens = q_lens, p.kv_lens = kv_lens;
  p.mask = mask, p.mask_s = mask_sb;
  p.q_s[0] = q_sb, p.q_s[1] = q_st, p.q_s[2] = q_sh;
  p.k_s[0] = k_sb, p.k_s[1] = k_st, p.k_s[2] = k_sh;
  p.v_s[0] = v_sb, p.v_s[1] = v_st, p.v_s[2] = v_sh;
  p.o_s[0] = o_sb, p.o_s[1] = o_st, p.o_s[2] = o_sh;
  p.b = b, p.tq = tq, p.kv = kv, p.hq = hq, p.hk = hk, p.d = d, p.group = hq / hk, p.scale = scale;
  return finish(run_cross(p, precision, static_cast<cudaStream_t>(stream)), "cross_attention");
}

}  // extern "C"
