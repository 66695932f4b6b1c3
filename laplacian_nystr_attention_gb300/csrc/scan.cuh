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

// A step's decay, and with the sigmoid gate z = 1 - a = 1 / (1 + exp(g)) beside it, each good to some
// 2^-24 of itself: h = a h + z x keeps what either loses of the other where it is small.  (With z alone
// and a = 1 - z, gradients through a gate of -10 were off by 5e-4 of themselves, of -17 gone.)
template <int V>
struct Gate {
  Vec<V> a, z;   // z: sigmoid only
};
// The hardware's base-2 exponential is good to 2 ulp, but its argument t, g log2 e rounded, is a
// relative error of |t| ulp in exp(g).  What t lacks, r, comes out of one more step or two, and
// 2^(t + r) = 2^t (1 + r ln 2) puts it back.  (bf16: log2 e in two parts, of which 16 bits times g are
// exact; r ln 2 is at most 5e-4, whose square costs 2^-24 and a half at the ends.)  g is held within
// [-88, 88], where nothing overflows, and everything is scaled by 1/16, so that 16 / (1 + exp(g)) stays in
// the normal range: a and z below 2^-126 (|g| above 87.3) are zero, and the other one is then 1.  NaN
// passes through.
template <bool kSig, bool k16, int V>
__device__ __forceinline__ Gate<V> gate_of(Raw<k16, V> w) {
  if constexpr (!kSig) {
    return {widen(w), fill<V>(0.f)};
  } else {
    constexpr float kScale = 0.0625f, kLn2 = 0.693147181f;
    const Vec<V> sixteenth = fill<V>(kScale);
    Vec<V> g, t, e, r;   // r: ln 2 / 16 of what t lacks
    if constexpr (k16) {   // both values at once (with one, the other half is 0)
      asm("min.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(w.w[0]) : "r"(0x42b042b0u));   // 88
      g = widen(w);
      t = mul(g, fill<V>(1.44268799f));                       // 0x1.7154p+0, 16 bits
      r = mul(g, fill<V>(kScale * 4.88849515e-6f));           // (log2 e - that) ln 2
    } else {
      g = widen(w);
#pragma unroll
      for (int i = 0; i < V; ++i)
        asm("min.NaN.xorsign.abs.f32 %0, %0, 0f42b00000;" : "+f"(g.f[i]));
      t = mul(g, fill<V>(1.44269504f));
      Vec<V> minus;
#pragma unroll
      for (int i = 0; i < V; ++i) minus.f[i] = -t.f[i];
      // log2 e is 1.44269504f and 1.92596303e-8.
      r = mul(fma(g, fill<V>(1.92596303e-8f), fma(g, fill<V>(1.44269504f), minus)),
              fill<V>(kScale * kLn2));
    }
#pragma unroll
    for (int i = 0; i < V; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.f[i]) : "f"(t.f[i]));
    e = fma(e, r, mul(e, sixteenth));                         // exp(g) / 16
    Vec<V> u = add(e, sixteenth);
#pragma unroll
    for (int i = 0; i < V; ++i) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(u.f[i]));   // 16 / (1 + exp(g))
    Gate<V> gate = {ops::mul_flush(e, u), ops::mul_flush(u, sixteenth)};
    // In fp32 also the last bit of an open gate's a, which the tokens that the state remembers
    // repeat; bf16 inputs leave it (a packed value's four instructions of some fifty).
    if constexpr (!k16)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (gate.z.f[i] < 0.5f) gate.a.f[i] = 1.f - gate.z.f[i];
    return gate;
  }
}
// The factor of a run's map: the product of its decays.  With the sigmoid gate also 1 less it,
// c = z + a c, a sum of positive numbers: where the gates are nearly open the state remembers 1 / (1 - A)
// runs, and a rounding of every factor of A would be that much larger in it.
template <bool kSig, int V>
struct Factor {
  Vec<V> p = fill<V>(1.f), c = fill<V>(0.f);
  __device__ __forceinline__ void take(const Gate<V>& gate) {
    p = mul(gate.a, p);
    if constexpr (kSig) c = fma(gate.a, c, gate.z);
  }
  __device__ __forceinline__ Vec<V> value() const {
    Vec<V> r = p;
    if constexpr (kSig)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c.f[i] < 0.5f) r.f[i] = 1.f - c.f[i];
    return r;
  }
};
// use(u, gate) for each of kT sigmoid gates in turn, those from `live` on as steps that change nothing.
// kAtOnce at a time, whose latencies overlap.
template <int kAtOnce, bool k16, int V, class Use>
__device__ __forceinline__ void gates(const Raw<k16, V> (&w)[kT], int i0, int live, Use use) {
#pragma unroll
  for (int u0 = 0; u0 < kT; u0 += kAtOnce) {
    Gate<V> g[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) g[u] = gate_of<true>(w[u0 + u]);
    if (i0 + u0 + kAtOnce > live) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (i0 + u0 + u >= live) g[u] = {fill<V>(1.f), fill<V>(0.f)};
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) use(u0 + u, g[u]);
  }
}
// The gradients of a step from D and E = a D.
template <bool kSig, int V>
__device__ __forceinline__ void step_gradients(const Vec<V>& z, const Vec<V>& slope, const Vec<V>& D,
                                               const Vec<V>& E, Vec<V>& dx, Vec<V>& dg) {
  dx = kSig ? mul(z, D) : D;
  dg = mul(slope, kSig ? E : D);
}

}  // namespace scan
}  // namespace lapl
