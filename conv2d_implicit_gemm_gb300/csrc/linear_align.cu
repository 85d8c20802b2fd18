// Matrices whose rows do not all start on 16 bytes, laid out anew with rows
// that do, so that TMA can fetch their tiles.
//
// One warp a row; each aligned piece of eight values is cut out of the two
// aligned pieces around it: a copy bound by memory (12 us for 2 x 41 MB), which
// costs a product of many rows less than gathering unaligned tiles in its main
// loop did (3000 x 5000 x 700: 95 us gathered).  For few rows the weight is
// read once anyway and linear_split.cu gathers.
#include <algorithm>

#include "linear_load.cuh"
#include "token.h"

namespace oidnx {
namespace {

__global__ void __launch_bounds__(256) align_rows_kernel(const AlignParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const AlignParams::Matrix& m = p.matrix[blockIdx.y];
  const uint8_t* begin = static_cast<const uint8_t*>(m.from);
  const int pieces = (p.k + 7) / 8, lane = threadIdx.x & 31;
  const int64_t warps = gridDim.x * 8ll;
  for (int64_t row = blockIdx.x * 8ll + (threadIdx.x >> 5); row < m.rows; row += warps) {
    const uint8_t* start = begin + 2 * row * m.ld;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(start) & 15);
    const uint8_t* from = start - off;
    uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(m.to) + row * m.ld_to);
    if (row * m.ld >= 8 && (m.rows - 1 - row) * m.ld >= 16) {
      // away from the matrix's ends: four pieces' loads before the first store
      for (int c0 = lane; c0 < pieces; c0 += 128) {
        uint4 lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c0 + 32 * i >= pieces) break;
          const uint4* q = reinterpret_cast<const uint4*>(from) + c0 + 32 * i;
          lo[i] = __ldg(q), hi[i] = __ldg(q + 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 32 * i < pieces) to[c0 + 32 * i] = shift_values(lo[i], hi[i], off / 2);
      }
      continue;
    }
    for (int c = lane; c < pieces; c += 32) {
      const int valid = min(p.k - c * 8, 8);
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = i < valid ? reinterpret_cast<const uint16_t*>(start)[c * 8 + i] : 0u;
      to[c] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
    // (what a row's last piece holds past k is never read)
  }
}

}  // namespace

cudaError_t launch_align_rows(const AlignParams& p, int count, int device, int sms, cudaStream_t stream) {
  int64_t most = 0;
  for (int i = 0; i < count; ++i) most = std::max<int64_t>(most, (p.matrix[i].rows + 7) / 8);
  static Kernel handle;
  return handle.launch(align_rows_kernel, device, dim3(static_cast<unsigned>(std::min<int64_t>(most, 8 * sms)), count), 256,
                       0, 1, stream, p);
}

}  // namespace oidnx
