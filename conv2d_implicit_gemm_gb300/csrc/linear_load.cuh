// Operand tiles of the linear layer that TMA cannot fetch (rows that do not
// all start on 16 bytes): read with plain loads and written to shared memory
// in the same 128-byte-swizzled layout that TMA would have given.
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

// Rows [r0, r0 + ROWS) and values [k0, k0 + 64) of a matrix of `rows` x k with
// row stride ld into the tile at `dst` (ROWS x 128 bytes, swizzled; zeros
// outside the matrix), by THREADS threads.  A piece that starts off a 16-byte
// boundary is cut out of the two aligned pieces around it; next to the
// matrix's first and last byte, where those would reach outside it, it is read
// value by value.
template <int ROWS, int THREADS>
__device__ __forceinline__ void gather_tile(uint8_t* dst, const void* base, int64_t ld, int rows, int k, int r0, int k0,
                                            int tid) {
  static_assert(ROWS * 8 % THREADS == 0, "whole passes");
  constexpr int N = ROWS * 8 / THREADS;
  const uint8_t* begin = static_cast<const uint8_t*>(base);
  const uint8_t* end = begin + 2 * ((rows - 1) * ld + k);
  constexpr int B = N < 4 ? N : 4;  // pieces in flight
#pragma unroll 1
  for (int n = 0; n < N; n += B) {
    uint4 lo[B], hi[B];
    int valid[B], off[B];
    bool edge[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int e = (n + i) * THREADS + tid, r = r0 + e / 8, c = k0 + (e % 8) * 8;
      valid[i] = r < rows ? min(max(k - c, 0), 8) : 0;
      const uint8_t* at = begin + 2 * (r * ld + c);
      off[i] = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15) / 2;
      const uint8_t* down = at - 2 * off[i];
      const bool second = off[i] + valid[i] > 8;
      edge[i] = valid[i] > 0 && (down < begin || down + (second ? 32 : 16) > end);
      const bool go = valid[i] > 0 && !edge[i];
      lo[i] = go ? __ldg(reinterpret_cast<const uint4*>(down)) : make_uint4(0u, 0u, 0u, 0u);
      hi[i] = go && second ? __ldg(reinterpret_cast<const uint4*>(down + 16)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int e = (n + i) * THREADS + tid, row = e / 8, c = e % 8;
      uint4 v = shift_values(lo[i], hi[i], off[i]);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
      if (edge[i]) {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(begin) + (r0 + row) * ld + k0 + c * 8;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t a = 2 * q < valid[i] ? src[2 * q] : 0u;
          const uint32_t b = 2 * q + 1 < valid[i] ? src[2 * q + 1] : 0u;
          w[q] = a | b << 16;
        }
      } else if (valid[i] < 8) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[q] &= 2 * q + 1 < valid[i] ? 0xFFFFFFFFu : 2 * q < valid[i] ? 0xFFFFu : 0u;
      }
      *reinterpret_cast<uint4*>(dst + row * 128 + ((c ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace oidnx
