// What the entry points of the token operators share on the host: errors, the
// driver's calls, tensor maps of heads.
#pragma once

#include <cstdio>

#include "../../include/oidnx.h"
#include "token.h"

namespace oidnx {

oidnx_status report_error(oidnx_status status, const char* message);
oidnx_status report_ok();
cudaError_t token_device(int* device, int* sms, int** status);
cudaError_t token_pool(int device, cudaMemPool_t* pool);
cudaError_t token_status_take(int* word, cudaStream_t stream);

template <typename... A>
oidnx_status fail(oidnx_status s, const char* fmt, A... args) {
  char buf[512];
  snprintf(buf, sizeof(buf), fmt, args...);
  return report_error(s, buf);
}
inline oidnx_status fail(oidnx_status s, const char* text) { return report_error(s, text); }

inline oidnx_status finish(cudaError_t e, const char* call) {
  if (e != cudaSuccess) {
    cudaGetLastError();  // a refused launch must not show up in the caller's next check
    return fail(e == cudaErrorMemoryAllocation ? OIDNX_ERR_OUT_OF_MEMORY : OIDNX_ERR_CUDA, "%s: %s", call,
                cudaGetErrorString(e));
  }
  return report_ok();
}

template <typename F> F driver_call(const char* name) {
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  return cudaGetDriverEntryPointByVersion(name, &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                 q == cudaDriverEntryPointSuccess
             ? reinterpret_cast<F>(ptr)
             : F(nullptr);
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kMost = 1 << 30;  // of a size, so that sums of a few of them stay within 32 bits

// ---------------------------------------------------------------- tensor maps
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Heads of 16-bit values as [sequence][outer][inner][value] in boxes of 64
// values x box1 x box2, 128-byte rows, swizzled.  outer and inner are tokens
// and heads in either order.
inline bool heads_map(CUtensorMap* map, bool bf16, const void* base, int d, int n1, int64_t s1, int n2, int64_t s2, int n3,
               int64_t s3, int box1, int box2) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2),
                              static_cast<cuuint64_t>(n3)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2,
                                 static_cast<cuuint64_t>(s3) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2), 1}, step[4] = {1, 1, 1, 1};
  static const EncodeFn fn = driver_call<EncodeFn>("cuTensorMapEncodeTiled");
  return fn && fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace oidnx
