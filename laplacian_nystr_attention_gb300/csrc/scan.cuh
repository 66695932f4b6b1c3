// scan.cuh -- what the kernels of the gated linear recurrence share (lapl_scan_* of
// include/lapl_ops.h; scan.cu has the formulas): launch arguments, typed accesses, and the step.
#pragma once

#include "ops_common.cuh"

namespace lapl {
namespace scan {

constexpr int kT = LAPL_SCAN_CHUNK;   // tokens of a thread's run

struct Geo {
  int lanes, lanes_log2;   // threads across the channels
  int blocks;              // channel blocks of a sequence
  int threads;             // threads of a CTA
  int cluster;             // CTAs along the tokens
  int tiles;               // rounds of cluster tiles along the tokens
};

struct Args {
  const void* x;
  const void* g;
  const float* h0;
  const int* lengths;
  void* out;
  float* states;
  float* final_state;
  const void* dout;
  const float* dfinal;
  void* dx;
  void* dg;
  float* dh0;
  long long x_stride, g_stride;
  int sequences, n, c, chunks, reverse;
  // scan_pipe.cuh: x and g, and dout, copied in less than 16 bytes; the bound of a wait, and n > 0
  // where the n-th last round's maps are not sent (fault injection for tests).
  bool fine, fine_dout;
  int skip_last;
  unsigned long long wait_ns;
  Geo geo;
};

// The V channels of a thread, one or two.
using ops::Vec, ops::fill, ops::fma, ops::mul, ops::add, ops::sub;

// A thread's channels of a token, as they lie in memory: one word, or two for two fp32 values.
template <bool k16, int V>
struct Raw {
  uint32_t w[!k16 && V == 2 ? 2 : 1];
};
template <bool k16, int V>
__device__ __forceinline__ Raw<k16, V> load_raw(const void* p) {
  Raw<k16, V> r;
  if constexpr (k16 && V == 1) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (!k16 && V == 2) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    r.w[0] = t.x;
    r.w[1] = t.y;
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}
template <bool k16, int V>
__device__ __forceinline__ Raw<k16, V> zero_raw() {
  Raw<k16, V> r;
  r.w[0] = 0u;
  if constexpr (!k16 && V == 2) r.w[1] = 0u;
  return r;
}
template <bool k16, int V>
__device__ __forceinline__ Vec<V> widen(const Raw<k16, V>& r) {
  Vec<V> v;
  if constexpr (!k16) {
#pragma unroll
    for (int i = 0; i < V; ++i) v.f[i] = __uint_as_float(r.w[i]);
  } else {
    v.f[0] = bf16_lo(r.w[0]);
    if constexpr (V == 2) v.f[V - 1] = bf16_hi(r.w[0]);
  }
  return v;
}
template <bool k16, int V>
__device__ __forceinline__ void store_vec(void* p, const Vec<V>& v) {
  if constexpr (k16) {
    if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = ops::pack_bf16(v.f[0], v.f[V - 1]);
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)ops::pack_bf16(v.f[0], 0.f);
  } else {
    if constexpr (V == 2) *reinterpret_cast<float2*>(p) = make_float2(v.f[0], v.f[V - 1]);
    else *reinterpret_cast<float*>(p) = v.f[0];
  }
}

// A step's decay as it is kept: a (decay gate), or -z (sigmoid gate) with z = 1 - a = 1 / (1 + exp(g)).
//
// The hardware's base-2 exponential is good to 2 ulp, but its argument t = g log2 e is rounded, which
// is a relative error of |t| ulp in exp(g).  The part that the rounding lost, r = g log2 e - t, comes
// exactly out of one more fused step, and 2^(t + r) = 2^t (1 + r ln 2) puts it back.  g is held within
// [-87, 88], where neither overflows (z is 1 and 6e-39 there); NaN passes through.
template <bool kSig, bool k16, int V>
__device__ __forceinline__ Vec<V> gate_of(Raw<k16, V> w) {
  if constexpr (!kSig) {
    return widen(w);
  } else {
    Vec<V> g;
    if constexpr (k16) {   // both values at once (with one, the other half is 0)
      asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(w.w[0]) : "r"(0x42b042b0u));
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.w[0]) : "r"(0xc2aec2aeu));
      g = widen(w);
    } else {
      g = widen(w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        asm("min.NaN.f32 %0, %0, 0f42b00000;" : "+f"(g.f[i]));   // 88
        asm("max.NaN.f32 %0, %0, 0fc2ae0000;" : "+f"(g.f[i]));   // -87
      }
    }
    const Vec<V> t = mul(g, fill<V>(-1.44269504f));            // -g log2 e, rounded
    const Vec<V> r = fma(g, fill<V>(1.44269504f), t);
    Vec<V> e;
#pragma unroll
    for (int i = 0; i < V; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.f[i]) : "f"(-t.f[i]));
    Vec<V> z = fma(mul(e, fill<V>(-0.693147181f)), r, sub(fill<V>(-1.f), e));   // -1 - exp(g)
#pragma unroll
    for (int i = 0; i < V; ++i) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(z.f[i]));
    return z;
  }
}
// The decay of a step that leaves the state as it is.
template <bool kSig, int V>
__device__ __forceinline__ Vec<V> identity_gate() {
  return fill<V>(kSig ? 0.f : 1.f);
}
// h after a step: h - z (h - x), or a h + x.
template <bool kSig, int V>
__device__ __forceinline__ Vec<V> step(const Vec<V>& gate, const Vec<V>& x, const Vec<V>& h) {
  if constexpr (kSig) return fma(gate, sub(h, x), h);
  else return fma(gate, h, x);
}
// a times v.
template <bool kSig, int V>
__device__ __forceinline__ Vec<V> decayed(const Vec<V>& gate, const Vec<V>& v) {
  if constexpr (kSig) return fma(gate, v, v);
  else return mul(gate, v);
}
// The gradients of a step from D, with E = a D and slope = x_i - h_{i-1} (gate is -z) or h_{i-1}.
template <bool kSig, int V>
__device__ __forceinline__ void step_gradients(const Vec<V>& gate, const Vec<V>& slope,
                                               const Vec<V>& D, const Vec<V>& E, Vec<V>& dx,
                                               Vec<V>& dg) {
#pragma unroll
  for (int i = 0; i < V; ++i) dx.f[i] = kSig ? -gate.f[i] * D.f[i] : D.f[i];
  dg = kSig ? mul(mul(gate, slope), E) : mul(slope, D);
}

}  // namespace scan
}  // namespace lapl
