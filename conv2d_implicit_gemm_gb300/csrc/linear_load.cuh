// Operand tiles of the linear layer that TMA cannot fetch (rows that do not
// all start on 16 bytes), in the same 128-byte-swizzled layout that TMA would
// have given.
#pragma once

#include "ptx.cuh"
#include "token.h"

namespace oidnx {

constexpr int kKB = 64;  // values of one K block: one 128-byte row of a tile

// Eight 16-bit values that start `s` values into the 32 bytes (lo, hi).
__device__ __forceinline__ uint4 shift_values(uint4 lo, uint4 hi, int s) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (s & 4) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (s & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (s & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Operand blocks of RA rows of one matrix and RB of another, 64 values each,
// for THREADS threads.  Rows start anywhere, so the nine aligned 16-byte pieces
// that hold a row's 128 bytes are first copied as they lie (asynchronously, a
// few blocks ahead), and then shifted into the swizzled operand layout.  A
// row's shift is the same in every block, as blocks are 128 bytes apart.
// Nothing outside [first value, last value] of a matrix is read.
template <int RA, int RB, int THREADS> struct Gather {
  static constexpr int kRows = RA + RB;
  static constexpr int kRaw = 144;                 // bytes of a row's pieces
  static constexpr int kStage = kRows * kRaw;
  static constexpr int kPer = (kRows * 8 + THREADS - 1) / THREADS;  // pieces of a thread

  struct Side {
    const uint8_t* begin;
    const uint8_t* end;
    int64_t ld;  // bytes
    int rows, r0;
  };
  Side a, b;
  int k, tid;

  static __device__ __forceinline__ Side side(const void* base, int64_t ld, int rows, int k) {
    Side s;
    s.begin = static_cast<const uint8_t*>(base);
    s.end = k > 0 ? s.begin + 2 * ((rows - 1) * ld + k) : s.begin;
    s.ld = 2 * ld, s.rows = rows, s.r0 = 0;
    return s;
  }
  __device__ __forceinline__ const Side& of(int row) const { return row < RA ? a : b; }
  __device__ __forceinline__ int index(int row) const { return of(row).r0 + (row < RA ? row : row - RA); }
  __device__ __forceinline__ const uint8_t* start(int row) const { return of(row).begin + index(row) * of(row).ld; }
  __device__ __forceinline__ bool inside(int row) const { return index(row) < of(row).rows; }

  __device__ __forceinline__ void copy(uint8_t* raw, int row, int piece, int k0) const {
    const Side& s = of(row);
    uint8_t* dst = raw + row * kRaw + piece * 16;
    const uint8_t* at = start(row) + 2 * k0;
    const uint8_t* from = at - (reinterpret_cast<uintptr_t>(at) & 15) + piece * 16;
    if (!inside(row) || from >= start(row) + 2 * k) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
    } else if (from < s.begin) {  // the matrix starts within this piece
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint8_t* q = from + 2 * i;
        v[i] = q >= s.begin && q < s.end ? *reinterpret_cast<const uint16_t*>(q) : 0u;
      }
      *reinterpret_cast<uint4*>(dst) =
          make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    } else {  // up to the matrix's last value
      const uint32_t bytes = s.end - from < 16 ? static_cast<uint32_t>(s.end - from) : 16u;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(from), "r"(bytes) : "memory");
    }
  }
  __device__ __forceinline__ void issue(uint8_t* raw, int k0) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * THREADS + tid;
      if (kRows * 8 % THREADS == 0 || e < kRows * 8) copy(raw, e / 8, e % 8, k0);
    }
    for (int row = tid; row < kRows; row += THREADS) copy(raw, row, 8, k0);
  }
  // The block's pieces, all landed, into the operands' layout.
  __device__ __forceinline__ void place(const uint8_t* raw, uint8_t* dst_a, uint8_t* dst_b, int k0) const {
#pragma unroll 2
    for (int i = 0; i < kPer; ++i) {
      const int e = i * THREADS + tid, row = e / 8, c = e % 8;
      if (kRows * 8 % THREADS != 0 && e >= kRows * 8) break;
      const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(start(row)) & 15) / 2;
      const uint4* q = reinterpret_cast<const uint4*>(raw + row * kRaw + c * 16);
      const uint4 v = shift_values(q[0], q[1], shift);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
      const int valid = inside(row) ? k - k0 - c * 8 : 0;  // values left in the row
      if (valid < 8) {
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] &= 2 * x + 1 < valid ? 0xFFFFFFFFu : 2 * x < valid ? 0xFFFFu : 0u;
      }
      const int r = row < RA ? row : row - RA;
      *reinterpret_cast<uint4*>((row < RA ? dst_a : dst_b) + r * 128 + ((c ^ (r & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

}  // namespace oidnx
