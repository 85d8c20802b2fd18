// Entry points of the token operators: argument checks and the choice of
// kernel.  Each is a direct call on device pointers; nothing is kept from one
// call for the next but the device error word.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "token_host.h"

using namespace oidnx;

namespace {

// ---------------------------------------------------------------- tensor maps
// A matrix of rows x cols 16-bit values with row stride ld, in boxes of
// box_cols (64: 128-byte rows, 32: 64-byte rows) x box_rows, swizzled.
bool matrix_map(CUtensorMap* map, bool bf16, const void* base, int64_t ld, int rows, int cols, int box_rows, int box_cols) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
  static const EncodeFn fn = driver_call<EncodeFn>("cuTensorMapEncodeTiled");
  return fn && fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                  const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows that TMA can address: all start on 16 bytes, strides below 2^40 bytes.
bool tma_rows(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0 && ld < (int64_t(1) << 38); }

// ---------------------------------------------------------------- linear: choice of form
constexpr int kMostSplit = 65535 * 32;  // rows of a grid of the split form's gathering tiles

// Few rows: K split over clusters, tokens as the narrow operand.
cudaError_t run_split(LinearTcLaunch& L, bool bf16, cudaStream_t stream) {
  const LinearParams& p = L.p;
  L.gather = p.k == 0 || !tma_rows(p.x, p.ldx) || !tma_rows(p.w, p.ldw);
  L.bn = p.m <= 16 ? 16 : p.m <= 32 || L.gather ? 32 : p.m <= 64 ? 64 : 128;
  const int64_t tiles = int64_t((p.n + 127) / 128) * ((p.m + L.bn - 1) / L.bn), blocks = (p.k + 63) / 64;
  L.split = 1;
  while (L.split < 8 && tiles * L.split <= L.sms && blocks / (L.split * 2) >= 4) L.split *= 2;
  if (!L.gather && !(matrix_map(&L.map_x, bf16, p.x, p.ldx, p.m, p.k, L.bn, 64) &&
                     matrix_map(&L.map_w, bf16, p.w, p.ldw, p.n, p.k, 128, 64)))
    return cudaErrorInvalidValue;
  return launch_linear_split(L, bf16, stream);
}

// Many rows, x and w with rows that TMA can address.
cudaError_t run_tiles(LinearTcLaunch& L, bool bf16, cudaStream_t stream) {
  const LinearParams& p = L.p;
  // Cycles of a tile shape: rounds of resident tiles times their K blocks, each
  // bound by its operands' way into the SM (64 bytes a cycle: 384 for 128 x 64
  // and for half a pair's 256 x 128, 512 for 128 x 128 and half of 256 x 256),
  // plus the last tile's epilogue, 28 a column, and a pair's start.  Measured for
  // the shapes in this order, us: 512 x 2048 x 2048: 10.6, 12.1, 11.6, 15.8;
  // 2000 x 1000 x 4000: 33, 20, 24, 24; 8192 x 512 x 4096: 55, 33, 37, 26;
  // 8192 x 256 x 256: 5.7, 6.4, 5.7, 7.9.
  struct Form {
    int rows, cols, pair, block;
  };
  static const Form forms[] = {{128, 64, 0, 384}, {256, 128, 1, 384}, {128, 128, 0, 512}, {256, 256, 1, 512}};
  const int64_t blocks = (p.k + 63) / 64;
  int64_t best = INT64_MAX;
  for (const Form& f : forms) {
    const int64_t tiles = int64_t((p.m + f.rows - 1) / f.rows) * ((p.n + f.cols - 1) / f.cols);
    const int64_t slots = f.pair ? L.sms / 2 : L.sms;
    const int64_t cost = (tiles + slots - 1) / slots * (blocks * f.block + 1500) + 28 * f.cols + 1200 * f.pair;
    if (cost < best) best = cost, L.pair = f.pair, L.bn = f.cols;
  }
  // TMA stores whole 16-byte pieces: one that the matrix ends in would be written
  // beyond it, whatever the map says of the row's length.
  L.tma_out = p.n % 8 == 0 && tma_rows(p.y, p.ldy) && (!p.residual || tma_rows(p.residual, p.ldr));
  const int cols = L.bn == 64 ? 32 : 64;
  const bool ok = matrix_map(&L.map_x, bf16, p.x, p.ldx, p.m, p.k, 128, 64) &&
                  matrix_map(&L.map_w, bf16, p.w, p.ldw, p.n, p.k, L.pair ? L.bn / 2 : L.bn, 64) &&
                  (!L.tma_out || matrix_map(&L.map_y, bf16, p.y, p.ldy, p.m, p.n, 32, cols)) &&
                  (!L.tma_out || !p.residual || matrix_map(&L.map_r, bf16, p.residual, p.ldr, p.m, p.n, 32, cols));
  return ok ? launch_linear_tc(L, bf16, stream) : cudaErrorInvalidValue;
}

cudaError_t run_linear(const LinearParams& params, bool bf16, cudaStream_t stream) {
  LinearTcLaunch L = {};
  L.p = params;
  LinearParams& p = L.p;
  cudaError_t e = token_device(&L.device, &L.sms, &p.status);
  if (e != cudaSuccess) return e;
  const bool x_fits = tma_rows(p.x, p.ldx), w_fits = tma_rows(p.w, p.ldw);
  // Few rows read the weight once, so they gather it as it lies (16 x 4000 x
  // 3501: 15 us, laid out anew first: 22); from 33 rows on, with one gathering
  // CTA an SM, its copying bounds it (64 rows: 34 and 26).  k = 0 has nothing to
  // fetch, which the gathering form's cleared blocks serve.
  if (p.k == 0 && p.m > kMostSplit) {
    for (int i = 0; i < params.m; i += kMostSplit) {  // rows of one grid at a time
      LinearParams part = params;
      part.m = std::min(kMostSplit, params.m - i);
      part.residual = params.residual ? static_cast<const uint8_t*>(params.residual) + 2 * i * params.ldr : nullptr;
      part.y = static_cast<uint8_t*>(params.y) + 2 * i * params.ldy;
      e = run_linear(part, bf16, stream);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  if (p.m <= 32 || p.k == 0 || (p.m <= 128 && x_fits && w_fits)) return run_split(L, bf16, stream);
  if (x_fits && w_fits) return run_tiles(L, bf16, stream);
  const int64_t ld = (static_cast<int64_t>(p.k) + 7) / 8 * 8;
  const int64_t x_bytes = x_fits ? 0 : ld * p.m * 2, w_bytes = w_fits ? 0 : ld * p.n * 2;
  cudaMemPool_t pool;
  void* scratch = nullptr;
  e = token_pool(L.device, &pool);
  if (e == cudaSuccess) e = cudaMallocFromPoolAsync(&scratch, x_bytes + w_bytes, pool, stream);
  if (e != cudaSuccess) return e;
  AlignParams a = {};
  a.k = p.k;
  int count = 0;
  if (!x_fits) {
    a.matrix[count++] = {p.x, scratch, p.ldx, ld, p.m};
    p.x = scratch, p.ldx = ld;
  }
  if (!w_fits) {
    void* to = static_cast<uint8_t*>(scratch) + x_bytes;
    a.matrix[count++] = {p.w, to, p.ldw, ld, p.n};
    p.w = to, p.ldw = ld;
  }
  e = launch_align_rows(a, count, L.device, L.sms, stream);
  if (e == cudaSuccess) e = p.m <= 128 ? run_split(L, bf16, stream) : run_tiles(L, bf16, stream);
  const cudaError_t freed = cudaFreeAsync(scratch, stream);
  return e != cudaSuccess ? e : freed;
}

// ---------------------------------------------------------------- attention: choice of form
cudaError_t run_attention(AttnParams& p, int precision, cudaStream_t stream) {
  int device, sms;
  const cudaError_t e = token_device(&device, &sms, &p.status);
  if (e != cudaSuccess) return e;
  const int group = p.hq / p.hk;
  // the stride of a dimension of one element says nothing
  const int64_t any = (static_cast<int64_t>(p.d) + 7) / 8 * 8;
  if (p.b == 1) p.q_s[0] = p.k_s[0] = p.v_s[0] = p.o_s[0] = any;
  if (p.tq == 1) p.q_s[1] = p.o_s[1] = any;
  if (p.cap == 1) p.k_s[1] = p.v_s[1] = any;
  if (p.hq == 1) p.q_s[2] = p.o_s[2] = any;
  if (p.hk == 1) p.k_s[2] = p.v_s[2] = any;
  bool pieces = p.d % 8 == 0 && p.d <= 128 && aligned(p.q, 16) && aligned(p.k, 16) && aligned(p.v, 16) && aligned(p.o, 16);
  for (int i = 0; i < 3; ++i)
    pieces = pieces && p.q_s[i] % 8 == 0 && p.k_s[i] % 8 == 0 && p.v_s[i] % 8 == 0 && p.o_s[i] % 8 == 0;
  const bool bf16 = precision == OIDNX_PRECISION_BF16;
  const int64_t rows = static_cast<int64_t>(p.tq) * group, row_tiles = (rows + 31) / 32, heads = static_cast<int64_t>(p.b) * p.hk;
  const int64_t units = heads * row_tiles;
  // Keys that a tile of some queries sees, at most and on average.
  const auto keys = [&](int64_t queries, bool mean) {
    const double all = mean ? p.cap - std::min(p.tq, p.cap) / 2.0 : p.cap;
    return p.window > 0 ? std::min(all, static_cast<double>(p.window) + p.held_sinks + queries) : all;
  };

  // Few queries: rounds of resident CTAs times a CTA's keys, plus its start and
  // the joining, 4 us more where rounds follow one another and share the memory.
  // Measured, us, one head of 128 values in eight parts: 16 rows over 600, 2300
  // and 8192 keys 8.7, 10.6, 17.3; 32 rows 12.5, 15, 24.4; of 64 values 6.1, 7.4,
  // 11.4 and 8.9, 10.5, 16.4.  64 ragged single tokens of 8 heads, up to 4100
  // keys: unsplit 134, in four 197.
  double token_cost = INFINITY;
  int split = 1;
  if (pieces && row_tiles <= 65535 && units < (1 << 27)) {
    const bool few = rows <= 16, small = p.d <= 64;
    const double key = few ? (small ? 5.6 : 9.1) : small ? 7.9 : 12.6;
    const double start = few ? (small ? 4000 : 6000) : small ? 6500 : 10000;
    const double seen = keys((31 + group) / group, units > sms);
    for (int s = 1; s <= 8; s *= 2) {
      const int slots = attn_token_slots(p, bf16, s, device);
      if (slots <= 0) continue;
      const double rounds = std::ceil(static_cast<double>(units) * s / slots);
      const double cost = rounds * (seen / s * key + start + (rounds > 1 ? 4000 : 0));
      if (cost < token_cost) token_cost = cost, split = s;
    }
  }
  bool tiles = pieces && group <= 128 && p.scale > 0.f && p.cap > 0;
  const int64_t far = int64_t(1) << 38;
  for (int i = 0; i < 3; ++i) {
    tiles = tiles && p.q_s[i] > 0 && p.q_s[i] < far && p.o_s[i] > 0 && p.o_s[i] < far;
    // keys and values may be shared by sequences and heads (stride 0)
    for (const int64_t s : {p.k_s[i], p.v_s[i]}) tiles = tiles && s < far && (i == 1 ? s > 0 : s >= 0);
  }
  const int per = group <= 128 ? 128 / group : 1;  // queries of a row tile
  const int64_t pairs = (static_cast<int64_t>(p.tq) + 2 * per - 1) / (2 * per), grid = pairs * heads;
  // Many queries: key tiles of 128, with one row tile and two on every SM, us:
  // heads of 128 values 1.41 and 1.66 (8192 keys 101 and 118), of 64 0.88 and 1.19
  // (64 and 85); 4 for a CTA's ends.  The longest CTA or the mean over the SMs, whichever is
  // more.
  const bool one = p.tq <= per;
  const double tile = p.d <= 64 ? (one ? 880 : 1190) : one ? 1410 : 1660;
  const int extra = p.window > 0 ? 1 : 0;
  const double longest = (std::ceil(keys(2 * per, false) / 128) + extra) * tile;
  const double mean = (std::ceil(keys(2 * per, true) / 128) + extra) * tile;
  const double prompt_cost = 4000 + std::max(longest, std::ceil(static_cast<double>(grid) / sms) * mean);
  // (a row tile of 128 with 16 rows or fewer has to win clearly: lengths are
  // upper bounds, and short sequences free a CTA of few queries sooner)
  if (token_cost < INFINITY && (!tiles || grid > INT_MAX || token_cost * (rows <= 16 ? 0.8 : 1.0) <= prompt_cost))
    return launch_attn_token(p, bf16, split, device, stream);
  if (tiles && grid <= INT_MAX) {
    // a shared dimension has one element, which the kernel reads for all
    const auto cache_map = [&](CUtensorMap* map, const void* base, const int64_t* s) {
      return heads_map(map, bf16, base, p.d, p.cap, s[1], s[2] ? p.hk : 1, s[2] ? s[2] : any, s[0] ? p.b : 1,
                       s[0] ? s[0] : any, 128, 1);
    };
    AttnLaunch L = {};
    L.p = p, L.p.group = group, L.p.per = per, L.p.pairs = static_cast<int>(pairs);
    L.device = device, L.grid = static_cast<unsigned>(grid);
    if (heads_map(&L.map_q, bf16, p.q, p.d, p.hq, p.q_s[2], p.tq, p.q_s[1], p.b, p.q_s[0], group, per) &&
        heads_map(&L.map_o, bf16, p.o, p.d, p.hq, p.o_s[2], p.tq, p.o_s[1], p.b, p.o_s[0], group, per) &&
        cache_map(&L.map_k, p.k, p.k_s) && cache_map(&L.map_v, p.v, p.v_s))
      return p.d <= 64 ? launch_attn_prompt64(L, bf16, stream) : launch_attn_prompt(L, bf16, stream);
  }
  return launch_attn_any(p, precision, device, stream);
}

// ---------------------------------------------------------------- norm and rotation: checks and parameters
// Index 0 = queries, 1 = keys, 2 = values.
struct HeadViews {
  const void* in[3];
  void* out[3];
  long long in_t[3], in_h[3], out_t[3], out_h[3];
};

oidnx_status norm_params(const char* name, const HeadViews& w, const void* q_weight, const void* k_weight, float eps,
                         const float* cos_table, const float* sin_table, long long table_rows, const int* positions,
                         const int* slots, long long cache_rows, int t, int hq, int hk, int d, int rot, int interleaved,
                         int precision, NormParams* out_params, bool* fast) {
  const void *q = w.in[0], *k = w.in[1], *v = w.in[2], *q_out = w.out[0], *k_out = w.out[1], *v_out = w.out[2];
  if (precision < OIDNX_PRECISION_FP32 || precision > OIDNX_PRECISION_BF16)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: unknown precision %d", name, precision);
  if (t < 0 || hq < 0 || hk < 0 || d <= 0 || rot < 0 || rot > d || rot % 2)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: bad sizes (t %d, heads %d and %d, d %d, rot %d)", name, t, hq, hk,
                d, rot);
  if (t > kMost) return fail(OIDNX_ERR_UNSUPPORTED, "%s: more than 2^30 tokens", name);
  if (hq > 65536 || hk > 65536) return fail(OIDNX_ERR_UNSUPPORTED, "%s: more than 65536 heads", name);
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: bad eps", name);
  if (t == 0 || (hq == 0 && hk == 0)) return finish(cudaSuccess, name);
  if ((hq && (!q || !q_out)) || (hk && (!k || !k_out)) || !v != !v_out)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: NULL heads", name);
  if (rot && (!cos_table || !sin_table || !positions || table_rows < 0))
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: NULL tables or positions", name);
  const size_t size = precision == OIDNX_PRECISION_FP32 ? 4 : 2;
  const void* all[] = {q, q_out, k, k_out, v, v_out, q_weight, k_weight};
  for (const void* a : all)
    if (!aligned(a, size))
      return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: pointers must be aligned to their elements", name);
  if (!aligned(cos_table, 4) || !aligned(sin_table, 4) || !aligned(positions, 4) || !aligned(slots, 4))
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: tables, positions and slots must be 4-byte aligned", name);
  NormParams& p = *out_params;
  p.heads[0] = hq, p.heads[1] = hk, p.heads[2] = v ? hk : 0;
  // Vector forms: heads in whole groups of four rotation pairs (eight: wide),
  // the rotated part and the rest alike, everything aligned to four values
  // (eight).  Values of 32 bits: four pairs and 16 bytes.
  const auto fits = [&](int pairs) {
    const size_t align = pairs * size;
    bool ok = d % (2 * pairs) == 0 && d / (2 * pairs) <= 32 && rot % (2 * pairs) == 0 && aligned(q_weight, align) &&
              aligned(k_weight, align) && aligned(cos_table, 16) && aligned(sin_table, 16);
    for (int i = 0; i < 3; ++i)
      if (p.heads[i])
        ok = ok && aligned(w.in[i], align) && aligned(w.out[i], align) && w.in_t[i] % pairs == 0 &&
             w.in_h[i] % pairs == 0 && w.out_t[i] % pairs == 0 && w.out_h[i] % pairs == 0;
    return ok;
  };
  for (int i = 0; i < 3; ++i) {
    p.in[i] = w.in[i], p.out[i] = w.out[i];
    p.in_t[i] = w.in_t[i], p.in_h[i] = w.in_h[i], p.out_t[i] = w.out_t[i], p.out_h[i] = w.out_h[i];
  }
  p.wide = size == 2 && fits(8);
  *fast = p.wide || fits(4);
  p.weight[0] = q_weight, p.weight[1] = k_weight;
  p.eps = eps, p.cos_t = cos_table, p.sin_t = sin_table, p.table_rows = table_rows;
  p.positions = positions, p.slots = slots, p.cache_rows = cache_rows;
  p.t = t, p.d = d, p.rot = rot, p.interleaved = interleaved != 0;
  return OIDNX_OK;
}

}  // namespace

extern "C" {

oidnx_status oidnx_linear(const void* x, long long ldx, const void* w, long long ldw, const void* bias,
                          const void* residual, long long ldr, void* y, long long ldy, int m, int n, int k, int act,
                          int precision, void* stream) {
  if (m < 0 || n < 0 || k < 0) return fail(OIDNX_ERR_INVALID_ARGUMENT, "linear: negative size (%d, %d, %d)", m, n, k);
  if (act < OIDNX_ACT_NONE || act > OIDNX_ACT_SILU)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "linear: unknown activation %d", act);
  if (precision == OIDNX_PRECISION_FP32) return fail(OIDNX_ERR_UNSUPPORTED, "linear: fp16 or bf16 only");
  if (precision != OIDNX_PRECISION_FP16 && precision != OIDNX_PRECISION_BF16)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "linear: unknown precision %d", precision);
  if (m > kMost || n > kMost || k > kMost) return fail(OIDNX_ERR_UNSUPPORTED, "linear: a size beyond 2^30");
  if (m == 0 || n == 0) return finish(cudaSuccess, "linear");
  if (!y || (k > 0 && (!x || !w))) return fail(OIDNX_ERR_INVALID_ARGUMENT, "linear: NULL x, w or y");
  if (ldx < k || ldw < k || ldy < n || (residual && ldr < n))
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "linear: a row stride is shorter than its row");
  if (!aligned(x, 2) || !aligned(w, 2) || !aligned(bias, 2) || !aligned(residual, 2) || !aligned(y, 2))
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "linear: pointers must be aligned to their elements");
  LinearParams p = {};
  p.x = x, p.w = w, p.bias = bias, p.residual = residual, p.y = y;
  p.ldx = ldx, p.ldw = ldw, p.ldr = ldr, p.ldy = ldy;
  p.m = m, p.n = n, p.k = k, p.act = act;
  return finish(run_linear(p, precision == OIDNX_PRECISION_BF16, static_cast<cudaStream_t>(stream)), "linear");
}

oidnx_status oidnx_qk_norm_rope(const void* q, long long q_st, long long q_sh, void* q_out, long long qo_st,
                                long long qo_sh, const void* k, long long k_st, long long k_sh, void* k_out,
                                long long ko_st, long long ko_sh, const void* v, long long v_st, long long v_sh,
                                void* v_out, long long vo_st, long long vo_sh, const void* q_weight,
                                const void* k_weight, float eps, const float* cos_table, const float* sin_table,
                                long long table_rows, const int* positions, const int* slots, long long cache_rows,
                                int t, int hq, int hk, int d, int rot, int interleaved, int precision, void* stream) {
  const HeadViews heads = {{q, k, v}, {q_out, k_out, v_out}, {q_st, k_st, v_st}, {q_sh, k_sh, v_sh}, {qo_st, ko_st, vo_st},
                           {qo_sh, ko_sh, vo_sh}};
  NormParams p = {};
  bool fast;
  const oidnx_status refused = norm_params("qk_norm_rope", heads, q_weight, k_weight, eps, cos_table, sin_table, table_rows,
                                           positions, slots, cache_rows, t, hq, hk, d, rot, interleaved, precision, &p, &fast);
  if (refused != OIDNX_OK || t == 0 || (hq == 0 && hk == 0)) return refused;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int device, sms, *status;
  cudaError_t e = token_device(&device, &sms, &status);
  if (e == cudaSuccess) e = fast ? launch_norm_vec(p, precision, device, sms, s) : launch_norm_any(p, precision, device, s);
  return finish(e, "qk_norm_rope");
}

oidnx_status oidnx_qk_norm_rope_axes(const void* q, long long q_st, long long q_sh, void* q_out, long long qo_st,
                                     long long qo_sh, const void* k, long long k_st, long long k_sh, void* k_out,
                                     long long ko_st, long long ko_sh, const void* v, long long v_st, long long v_sh,
                                     void* v_out, long long vo_st, long long vo_sh, int norm, const void* q_weight,
                                     const void* k_weight, float eps, const float* cos_table, const float* sin_table,
                                     long long table_rows, const int* positions, long long positions_stride, int axes,
                                     const unsigned char* pair_axes, const int* slots, long long cache_rows, int t, int hq,
                                     int hk, int d, int rot, int interleaved, int precision, void* stream) {
  const char* name = "qk_norm_rope_axes";
  if (axes < 1 || axes > kMostAxes) return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: %d axes (1 to %d)", name, axes, kMostAxes);
  const HeadViews heads = {{q, k, v}, {q_out, k_out, v_out}, {q_st, k_st, v_st}, {q_sh, k_sh, v_sh}, {qo_st, ko_st, vo_st},
                           {qo_sh, ko_sh, vo_sh}};
  AxesParams p = {};
  bool fast;
  const oidnx_status refused = norm_params(name, heads, q_weight, k_weight, eps, cos_table, sin_table, table_rows, positions,
                                           slots, cache_rows, t, hq, hk, d, rot, interleaved, precision, &p, &fast);
  if (refused != OIDNX_OK) return refused;
  if (rot > 2 * kMostPairs) return fail(OIDNX_ERR_UNSUPPORTED, "%s: more than %d rotated values (%d)", name, 2 * kMostPairs, rot);
  if (rot && t && positions_stride < t) return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: positions_stride below t", name);
  if (rot && !pair_axes) return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: NULL pair_axes", name);
  for (int r = 0; r < rot / 2; ++r) {
    if (pair_axes[r] >= axes) return fail(OIDNX_ERR_INVALID_ARGUMENT, "%s: pair %d turns by axis %d of %d", name, r, pair_axes[r], axes);
    p.pair_axis[r] = pair_axes[r];
  }
  if (t == 0 || (hq == 0 && hk == 0)) return finish(cudaSuccess, name);
  p.positions_stride = positions_stride, p.axes = axes, p.norm = norm != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int device, sms, *status;
  cudaError_t e = token_device(&device, &sms, &status);
  if (e == cudaSuccess) e = fast ? launch_axes_vec(p, precision, device, sms, s) : launch_axes_any(p, precision, device, s);
  return finish(e, name);
}

oidnx_status oidnx_window_attention(const void* q, long long q_sb, long long q_st, long long q_sh, const void* k,
                                    long long k_sb, long long k_st, long long k_sh, const void* v, long long v_sb,
                                    long long v_st, long long v_sh, void* o, long long o_sb, long long o_st,
                                    long long o_sh, float* lse, const int* q_lens, const int* kv_lens, int b, int tq,
                                    int cap, int hq, int hk, int d, int window, int sinks, float scale, int precision,
                                    void* stream) {
  if (precision == OIDNX_PRECISION_FP32) return fail(OIDNX_ERR_UNSUPPORTED, "window_attention: fp16 or bf16 only");
  if (precision != OIDNX_PRECISION_FP16 && precision != OIDNX_PRECISION_BF16)
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "window_attention: unknown precision %d", precision);
  if (b < 0 || tq < 0 || cap < 0 || hq < 0 || hk <= 0 || hq % hk || d <= 0 || window < 0 || sinks < 0)
    return fail(OIDNX_ERR_INVALID_ARGUMENT,
                "window_attention: bad sizes (b %d, tq %d, cap %d, heads %d and %d, d %d, window %d, sinks %d)", b, tq,
                cap, hq, hk, d, window, sinks);
  if (tq > kMost || cap > kMost) return fail(OIDNX_ERR_UNSUPPORTED, "window_attention: a length beyond 2^30");
  if (d > 256) return fail(OIDNX_ERR_UNSUPPORTED, "window_attention: heads of more than 256 values (%d)", d);
  if (!std::isfinite(scale)) return fail(OIDNX_ERR_INVALID_ARGUMENT, "window_attention: scale is not finite");
  if (b == 0 || tq == 0 || hq == 0) return finish(cudaSuccess, "window_attention");
  if (static_cast<double>(b) * tq * hq > 4e9)
    return fail(OIDNX_ERR_UNSUPPORTED, "window_attention: more than 4e9 query heads");
  if (!q || !o || (cap > 0 && (!k || !v))) return fail(OIDNX_ERR_INVALID_ARGUMENT, "window_attention: NULL q, k, v or o");
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(o, 2) || !aligned(lse, 4) || !aligned(q_lens, 4) ||
      !aligned(kv_lens, 4))
    return fail(OIDNX_ERR_INVALID_ARGUMENT, "window_attention: pointers must be aligned to their elements");
  AttnParams p = {};
  p.q = q, p.k = k, p.v = v, p.o = o, p.lse = lse, p.q_lens = q_lens, p.kv_lens = kv_lens;
  p.q_s[0] = q_sb, p.q_s[1] = q_st, p.q_s[2] = q_sh;
  p.k_s[0] = k_sb, p.k_s[1] = k_st, p.k_s[2] = k_sh;
  p.v_s[0] = v_sb, p.v_s[1] = v_st, p.v_s[2] = v_sh;
  p.o_s[0] = o_sb, p.o_s[1] = o_st, p.o_s[2] = o_sh;
  p.b = b, p.tq = tq, p.cap = cap, p.hq = hq, p.hk = hk, p.d = d;
  p.window = window, p.sinks = sinks, p.held_sinks = sinks < cap ? sinks : cap, p.scale = scale;
  return finish(run_attention(p, precision, static_cast<cudaStream_t>(stream)), "window_attention");
}

oidnx_status oidnx_token_sync_status(void* stream) {
  int word = 0;
  const cudaError_t e = token_status_take(&word, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess && word)
    return fail(OIDNX_ERR_TIMEOUT, "a device-side wait gave up (status bits 0x%x)", word);
  return finish(e, "token_sync_status");
}

}  // extern "C"

// ---------------------------------------------------------------- launches
cudaError_t oidnx::Kernel::find(const void* kernel, int smem, int device, CUfunction* f) {
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  cudaError_t e = cudaSuccess;
  smem = std::max(smem, most);
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  cudaFunction_t found = nullptr;
  if (e == cudaSuccess) e = cudaGetFuncBySymbol(&found, kernel);
  if (e != cudaSuccess) return e;
  fn[device].store(found, std::memory_order_release);
  *f = found;
  return cudaSuccess;
}

int oidnx::Kernel::count_clusters(const void* kernel, int device, int threads, int smem, int cluster) {
  const int at = cluster == 1 ? 0 : cluster == 2 ? 1 : cluster == 4 ? 2 : 3;
  int n = held[at][device].load(std::memory_order_relaxed);
  if (n > 0) return n;
  CUfunction f = fn[device].load(std::memory_order_acquire);
  if (!f && find(kernel, smem, device, &f) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = cluster;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  held[at][device].store(n, std::memory_order_relaxed);
  return n;
}

// Each kernel may start its prologue under the one before it in the stream
// (it waits for that one's results itself).
cudaError_t oidnx::Kernel::launch_found(CUfunction f, dim3 grid, int threads, int smem, int cluster,
                                        cudaStream_t stream, void** params) {
  static const auto call = driver_call<CUresult (*)(const CUlaunchConfig*, CUfunction, void**, void**)>("cuLaunchKernelEx");
  if (!call) return cudaErrorNotSupported;
  CUlaunchAttribute at[2] = {};
  at[0].id = CU_LAUNCH_ATTRIBUTE_PROGRAMMATIC_STREAM_SERIALIZATION;
  at[0].value.programmaticStreamSerializationAllowed = 1;
  at[1].id = CU_LAUNCH_ATTRIBUTE_CLUSTER_DIMENSION;
  at[1].value.clusterDim.x = cluster;
  at[1].value.clusterDim.y = at[1].value.clusterDim.z = 1;
  CUlaunchConfig cfg = {};
  cfg.gridDimX = grid.x, cfg.gridDimY = grid.y, cfg.gridDimZ = grid.z;
  cfg.blockDimX = threads, cfg.blockDimY = cfg.blockDimZ = 1;
  cfg.sharedMemBytes = smem;
  cfg.hStream = stream;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return static_cast<cudaError_t>(call(&cfg, f, params, nullptr));  // the two share their codes
}

// ---------------------------------------------------------------- error word
namespace {
__device__ int g_token_status;
constexpr int kMaxDevices = 64;
struct DeviceInfo {
  int* status = nullptr;
  int sms = 0;
  cudaMemPool_t pool = nullptr;
  cudaError_t pool_error = cudaSuccess;
};
std::mutex g_device_mutex;
DeviceInfo g_devices[kMaxDevices];

// A pool of the library's own, which keeps this much for later calls where the
// default pool hands everything back at every synchronisation; what is beyond it
// goes back there.  Getting memory anew costs 2 us a MiB (copies of 512 MiB, waited
// for after each call: 456 us kept, 1215 not), so that this holds the operands of
// 64k x 8k; it is 1 / 280 of the device's memory.
constexpr uint64_t kPoolKeeps = uint64_t(1) << 30;

cudaError_t make_pool(int device, cudaMemPool_t* out) {
  cudaMemPoolProps props = {};
  props.allocType = cudaMemAllocationTypePinned;
  props.location.type = cudaMemLocationTypeDevice;
  props.location.id = device;
  cudaError_t e = cudaMemPoolCreate(out, &props);
  if (e != cudaSuccess) return e;
  uint64_t keep = kPoolKeeps;
  e = cudaMemPoolSetAttribute(*out, cudaMemPoolAttrReleaseThreshold, &keep);
  if (e != cudaSuccess) cudaMemPoolDestroy(*out);
  return e;
}
}  // namespace

// The current device, its SM count and its error word (looked up once, and the pool
// made with them: it cannot be made while a stream is captured).
cudaError_t oidnx::token_device(int* device, int* sms, int** status) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  // The driver's calls need the device's context on the calling thread, which
  // the runtime binds at a thread's first call that needs it.
  static thread_local int bound = -1;
  if (bound != dev) {
    e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    bound = dev;
  }
  std::lock_guard<std::mutex> lock(g_device_mutex);
  DeviceInfo& d = g_devices[dev];
  if (!d.status) {
    void* p = nullptr;
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaGetSymbolAddress(&p, g_token_status);
    if (e != cudaSuccess) return e;
    d.pool_error = make_pool(dev, &d.pool);
    if (d.pool_error != cudaSuccess) cudaGetLastError();  // only calls that need the pool fail
    d.status = static_cast<int*>(p);
  }
  *device = dev;
  *sms = d.sms;
  *status = d.status;
  return cudaSuccess;
}

// Memory of one call, ordered on its stream, comes from here.  The device's look-up
// is behind the caller.
cudaError_t oidnx::token_pool(int device, cudaMemPool_t* pool) {
  std::lock_guard<std::mutex> lock(g_device_mutex);
  *pool = g_devices[device].pool;
  return g_devices[device].pool_error;
}

// Wait for `stream`, then read and clear the error word.
cudaError_t oidnx::token_status_take(int* word, cudaStream_t stream) {
  int device, sms, *at = nullptr;
  cudaError_t e = token_device(&device, &sms, &at);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyAsync(word, at, sizeof(int), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess && *word) {
    e = cudaMemsetAsync(at, 0, sizeof(int), stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  }
  return e;
}
