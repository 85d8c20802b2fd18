// Operand tiles of the linear layer that TMA cannot fetch (rows that do not
// all start on 16 bytes), in the same 128-byte-swizzled layout that TMA would
// have given.
#pragma once

#include "token_ptx.cuh"
#include "token.h"

namespace oidnx {

constexpr int kKB = 64;  // values of one K block: one 128-byte row of a tile

// Eight 16-bit values that start `s` values into the 32 bytes (lo, hi).
__device__ __forceinline__ uint4 shift_values(uint4 lo, uint4 hi, int s) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = s & 4 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = s & 2 ? w[i + 1] : w[i];
  const uint32_t pick = s & 1 ? 0x5432u : 0x3210u;
  return make_uint4(__byte_perm(w[0], w[1], pick), __byte_perm(w[1], w[2], pick), __byte_perm(w[2], w[3], pick),
                    __byte_perm(w[3], w[4], pick));
}

// Operand blocks of RA rows of one matrix and RB of another, 64 values each.
// Rows start anywhere, so four copying warps first bring the nine aligned
// 16-byte pieces that hold a row's 128 bytes to shared memory as they lie
// (asynchronously, a few blocks ahead), and eight placing warps shift them into
// the swizzled operand layout.  A row's shift is the same in every block, as
// blocks are 128 bytes apart.  Nothing outside [first value, last value] of a
// matrix is read.
constexpr int kCopyThreads = 128;
constexpr int kPlaceThreads = 256;

template <int RA, int RB> struct Gather {
  static constexpr int kRows = RA + RB;
  static constexpr int kRaw = 144;  // bytes of a row's pieces
  static constexpr int kStage = kRows * kRaw;

  struct Side {
    const uint8_t* begin;
    const uint8_t* end;
    int64_t ld;  // bytes
    int rows, r0;
  };
  Side a, b;
  int k;

  __device__ __forceinline__ void matrices(const void* base_a, int64_t ld_a, int rows_a, const void* base_b, int64_t ld_b,
                                           int rows_b, int values) {
    k = values;
    a = side(base_a, ld_a, rows_a), b = side(base_b, ld_b, rows_b);
  }
  __device__ __forceinline__ Side side(const void* base, int64_t ld, int rows) const {
    Side s;
    s.begin = static_cast<const uint8_t*>(base);
    s.end = k > 0 ? s.begin + 2 * ((rows - 1) * ld + k) : s.begin;
    s.ld = 2 * ld, s.rows = k > 0 ? rows : 0, s.r0 = 0;
    return s;
  }
  // A piece at the matrix's first or last bytes: what lies within it.
  static __device__ __noinline__ void copy_edge(uint8_t* dst, const uint8_t* from, const uint8_t* begin, const uint8_t* end) {
    for (int x = 0; x < 8; ++x) {
      const uint8_t* q = from + 2 * x;
      reinterpret_cast<uint16_t*>(dst)[x] = q >= begin && q < end ? *reinterpret_cast<const uint16_t*>(q) : uint16_t(0);
    }
  }
  // Rows past the matrix repeat its last one (their results are not stored);
  // what lies past a row's end is cleared when the block is placed.
  template <int ROWS, bool EDGE>
  __device__ __forceinline__ void copy_rows(uint8_t* raw, const Side& s, int k0, int tid) const {
    const uint8_t* base = s.begin + 2 * static_cast<int64_t>(k0);
    const int last = s.rows - 1;
    const auto one = [&](int row, int c) {
      const uint8_t* at = base + min(s.r0 + row, last) * s.ld;
      const uint8_t* from = at - (reinterpret_cast<uintptr_t>(at) & 15) + c * 16;
      uint8_t* dst = raw + row * kRaw + c * 16;
      if (!EDGE || (from >= s.begin && from + 16 <= s.end))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(from) : "memory");
      else
        copy_edge(dst, from, s.begin, s.end);
    };
#pragma unroll
    for (int i = 0; i < ROWS / (kCopyThreads / 8); ++i) one(i * (kCopyThreads / 8) + (tid >> 3), tid & 7);
#pragma unroll
    for (int i = 0; i < (ROWS + kCopyThreads - 1) / kCopyThreads; ++i)
      if (i * kCopyThreads + tid < ROWS) one(i * kCopyThreads + tid, 8);
  }
  template <int ROWS> __device__ __forceinline__ void copy_side(uint8_t* raw, const Side& s, int k0, int tid) const {
    if (s.rows == 0) return;  // k = 0: the block is cleared when it is placed
    const uint8_t* first = s.begin + s.r0 * s.ld + 2 * static_cast<int64_t>(k0);
    const uint8_t* last = s.begin + min(s.r0 + ROWS, s.rows) * s.ld - s.ld + 2 * static_cast<int64_t>(k0);
    if (first - 15 >= s.begin && last + 144 <= s.end) copy_rows<ROWS, false>(raw, s, k0, tid);
    else copy_rows<ROWS, true>(raw, s, k0, tid);
  }
  // The block's pieces on their way; `bar` gets two arrivals of each thread: one
  // when its copies have landed, one for what it wrote itself.
  __device__ __forceinline__ void copy_block(uint8_t* raw, uint64_t* bar, int k0, int tid) const {
    copy_side<RA>(raw, a, k0, tid);
    copy_side<RB>(raw + RA * kRaw, b, k0, tid);
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    mbar_arrive(bar);
  }
  template <int ROWS>
  __device__ __forceinline__ void place_side(const uint8_t* raw, uint8_t* dst, const Side& s, int values, int tid) const {
    constexpr int N = ROWS * 8 / kPlaceThreads;  // pieces of a thread (0: half of them have one)
    const int c = tid & 7, row0 = tid >> 3;
    const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s.begin)) + (s.r0 + row0) * static_cast<uint32_t>(s.ld);
    uint4 lo[N > 0 ? N : 1], hi[N > 0 ? N : 1];
    if (N == 0 && row0 >= ROWS) return;
#pragma unroll
    for (int i = 0; i < (N > 0 ? N : 1); ++i) {
      const uint4* q = reinterpret_cast<const uint4*>(raw + (row0 + 32 * i) * kRaw + c * 16);
      lo[i] = q[0], hi[i] = q[1];
    }
#pragma unroll
    for (int i = 0; i < (N > 0 ? N : 1); ++i) {
      const int r = row0 + 32 * i;
      const uint4 v = shift_values(lo[i], hi[i], static_cast<int>((low + 32 * i * static_cast<uint32_t>(s.ld)) >> 1 & 7));
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
      if (values < kKB) {
        const int valid = values - c * 8;
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] &= 2 * x + 1 < valid ? 0xFFFFFFFFu : 2 * x < valid ? 0xFFFFu : 0u;
      }
      *reinterpret_cast<uint4*>(dst + r * 128 + ((c ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // A block's pieces, all landed, into the operands' layout; values: of a row
  // from the block on.
  __device__ __forceinline__ void place(const uint8_t* raw, uint8_t* dst_a, uint8_t* dst_b, int values, int tid) const {
    place_side<RA>(raw, dst_a, a, values, tid);
    place_side<RB>(raw + RA * kRaw, dst_b, b, values, tid);
  }
};

}  // namespace oidnx
