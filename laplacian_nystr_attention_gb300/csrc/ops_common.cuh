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

// One or two floats; two go through the packed fp32 instructions.
template <int V>
struct Vec {
  float f[V];
};
template <int V>
__device__ __forceinline__ Vec<V> fill(float v) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.f[i] = v;
  return r;
}
__device__ __forceinline__ Vec<1> fma(const Vec<1>& a, const Vec<1>& b, const Vec<1>& c) {
  return {{fmaf(a.f[0], b.f[0], c.f[0])}};
}
__device__ __forceinline__ Vec<1> mul(const Vec<1>& a, const Vec<1>& b) { return {{a.f[0] * b.f[0]}}; }
// Products below the normal range are zero.
__device__ __forceinline__ Vec<1> mul_flush(const Vec<1>& a, const Vec<1>& b) {
  Vec<1> d;
  asm("mul.rn.ftz.f32 %0, %1, %2;" : "=f"(d.f[0]) : "f"(a.f[0]), "f"(b.f[0]));
  return d;
}
__device__ __forceinline__ Vec<1> add(const Vec<1>& a, const Vec<1>& b) { return {{a.f[0] + b.f[0]}}; }
__device__ __forceinline__ Vec<1> sub(const Vec<1>& a, const Vec<1>& b) { return {{a.f[0] - b.f[0]}}; }
#define LAPL_PACKED(name, op)                                                              \
  __device__ __forceinline__ Vec<2> name(const Vec<2>& a, const Vec<2>& b) {                    \
    Vec<2> d;                                                                                   \
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t" op          \
        ".f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"                                          \
        : "=f"(d.f[0]), "=f"(d.f[1])                                                            \
        : "f"(a.f[0]), "f"(a.f[1]), "f"(b.f[0]), "f"(b.f[1]));                                  \
    return d;                                                                                   \
  }
LAPL_PACKED(mul, "mul.rn")
LAPL_PACKED(mul_flush, "mul.rn.ftz")
LAPL_PACKED(add, "add.rn")
LAPL_PACKED(sub, "sub.rn")
#undef LAPL_PACKED
__device__ __forceinline__ Vec<2> fma(const Vec<2>& a, const Vec<2>& b, const Vec<2>& c) {
  Vec<2> d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.f[0]), "=f"(d.f[1])
      : "f"(a.f[0]), "f"(a.f[1]), "f"(b.f[0]), "f"(b.f[1]), "f"(c.f[0]), "f"(c.f[1]));
  return d;
}

// A sum held as two floats, its value and what that lost (Knuth's two-sum): 48 bits without the
// double-precision units, of which this GPU has few (sums in double took 36 us of a pass of 57).
// Where the sum is not finite, hi says so and lo nothing.
struct Pair {
  float hi, lo;
  __device__ __forceinline__ void add(float v, float v_lo = 0.f) {
    const float s = hi + v, b = s - hi;
    lo += (hi - (s - b)) + (v - b) + v_lo;
    hi = s;
  }
  __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

__device__ __forceinline__ unsigned smem_u32(const void* p) {
  return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
// `bytes` of the 16 at src (both multiples of 16 bytes; none are read of 0), zeros for the rest.
__device__ __forceinline__ void copy16(unsigned dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void close_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the last kPending groups of this thread's copies are there.
template <int kPending>
__device__ __forceinline__ void copies_left() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

}  // namespace ops
}  // namespace lapl
