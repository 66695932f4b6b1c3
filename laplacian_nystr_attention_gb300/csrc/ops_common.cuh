// ops_common.cuh -- what the kernels of the operators in include/lapl_ops.h share: typed loads and
// stores, and host-side checks.
#pragma once

#include <cuda_fp8.h>
#include <stdio.h>

#include "common.cuh"
#include "lapl_ops.h"

namespace lapl {

// A bit of the device error word beside those of common.cuh: the exchange between CTAs of the gated
// linear recurrence.
constexpr unsigned kErrBitScan = 8u;

namespace ops {

constexpr int kErrorText = 256;

inline bool is_float_dtype(int t) { return t == LAPL_F32 || t == LAPL_BF16; }
inline int dtype_bytes(int t) { return t == LAPL_F32 ? 4 : t == LAPL_BF16 ? 2 : 1; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline void set_error(char* text, cudaError_t e, const char* where) {
  snprintf(text, kErrorText, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

// LAPL_OK if `device` is current.
inline lapl_status check_device(int device, char* text, const char* where) {
  int now = -1;
  const cudaError_t e = cudaGetDevice(&now);
  if (e != cudaSuccess) {
    set_error(text, e, where);
    return LAPL_ERR_CUDA;
  }
  return now == device ? LAPL_OK : LAPL_ERR_INVALID_ARG;
}

// Two floats as two bf16 in a word (round to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_bits(uint16_t b) {
  return __uint_as_float((uint32_t)b << 16);
}

}  // namespace ops
}  // namespace lapl
