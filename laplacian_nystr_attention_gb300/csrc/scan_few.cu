// scan_few.cu -- the gated linear recurrence over few tokens, as a model that answers token by token
// calls it: scan.cu's formulas without its exchange.
//
// A thread has all tokens of four channels (one where rows or pointers are not multiples of four
// elements) and goes through the steps with the state in registers: of up to four tokens it reads all
// at once, of more some at a time with the next ones on their way.  128 x 1 x 4096 bf16 takes 2.4 us where
// the kernel for longer sequences, 32 threads a CTA and 16 tokens a thread, takes 15.8; 64 x 1 x 512 1.7
// and 2.9; 20000 x 2 x 512 34 (89% of the copy's rate) and 317; 64 x 8 x 4096 4.1 and 9.8.  What bounds
// it is the launch, then the bytes.
#include "scan_few.cuh"

namespace lapl {
namespace scan {
namespace few {
namespace {

// V channels of a token: pairs of them, or one.
template <int V>
struct Parts {
  static constexpr int kW = V == 4 ? 2 : 1, kN = V / kW;
};
template <int V>
struct State {
  Vec<Parts<V>::kW> p[Parts<V>::kN];
};
template <bool k16, int V>
struct Token {
  Raw<k16, Parts<V>::kW> p[Parts<V>::kN];
};
template <bool k16, int V>
__device__ __forceinline__ Token<k16, V> load_token(const void* base, long long e) {
  Token<k16, V> t;
  const char* q = reinterpret_cast<const char*>(base) + e * (k16 ? 2 : 4);
  if constexpr (V == 1) {
    t.p[0] = load_raw<k16, 1>(q);
  } else if constexpr (k16) {
    const uint2 w = *reinterpret_cast<const uint2*>(q);
    t.p[0].w[0] = w.x;
    t.p[1].w[0] = w.y;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(q);
    t.p[0].w[0] = w.x; t.p[0].w[1] = w.y;
    t.p[1].w[0] = w.z; t.p[1].w[1] = w.w;
  }
  return t;
}
template <bool k16, int V>
__device__ __forceinline__ void store_state(void* base, long long e, const State<V>& h) {
  char* q = reinterpret_cast<char*>(base) + e * (k16 ? 2 : 4);
  if constexpr (V == 1) {
    store_vec<k16>(q, h.p[0]);
  } else if constexpr (k16) {
    *reinterpret_cast<uint2*>(q) = make_uint2(ops::pack_bf16(h.p[0].f[0], h.p[0].f[1]),
                                              ops::pack_bf16(h.p[1].f[0], h.p[1].f[1]));
  } else {
    *reinterpret_cast<float4*>(q) =
        make_float4(h.p[0].f[0], h.p[0].f[1], h.p[1].f[0], h.p[1].f[1]);
  }
}

// T: tokens at a time; kMore: and the next T on their way while those are worked on.
template <bool kIn16, bool kOut16, int V, bool kSig, int T, bool kMore>
__global__ void __launch_bounds__(kThreads) scan_few_kernel(const Args a) {
  constexpr int kW = Parts<V>::kW, kN = Parts<V>::kN;
  const int unit = blockIdx.x / a.geo.blocks, block = blockIdx.x - unit * a.geo.blocks;
  const long long s =
      (long long)unit * (kThreads >> a.geo.lanes_log2) + (threadIdx.x >> a.geo.lanes_log2);
  const int c = (block * a.geo.lanes + ((int)threadIdx.x & (a.geo.lanes - 1))) * V;
  if (s >= a.sequences || c >= a.c) return;
  const int len = a.lengths ? max(0, min(a.n, a.lengths[s])) : a.n;
  State<V> h;
#pragma unroll
  for (int k = 0; k < kN; ++k) h.p[k] = fill<kW>(0.f);
  auto row = [&](int i) { return s * a.n + (a.reverse ? len - 1 - i : i); };
  Token<kIn16, V> x[T], g[T];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < T; ++u)
      if (i0 + u < len) {
        g[u] = load_token<kIn16, V>(a.g, row(i0 + u) * a.g_stride + c);
        x[u] = load_token<kIn16, V>(a.x, row(i0 + u) * a.x_stride + c);
      }
  };
  fetch(0);
  if (a.h0) {
    const Token<false, V> t = load_token<false, V>(a.h0, s * a.c + c);
#pragma unroll
    for (int k = 0; k < kN; ++k) h.p[k] = widen(t.p[k]);
  }
  for (int i0 = 0; i0 < (kMore ? a.n : 1); i0 += T) {
    Token<kIn16, V> nx[T], ng[T];
#pragma unroll
    for (int u = 0; u < T; ++u) {
      nx[u] = x[u];
      ng[u] = g[u];
    }
    if (kMore) fetch(i0 + T);
    if (a.states && i0 % kT == 0)
      store_state<false>(a.states, (s * a.chunks + i0 / kT) * a.c + c, h);
#pragma unroll
    for (int u = 0; u < T; ++u) {
      const int i = i0 + u;
      if (i < len) {
#pragma unroll
        for (int k = 0; k < kN; ++k)
          h.p[k] = step<kSig>(gate_of<kSig>(ng[u].p[k]), widen(nx[u].p[k]), h.p[k]);
        store_state<kOut16>(a.out, row(i) * a.c + c, h);
      } else if (i < a.n) {
        State<V> zero;
#pragma unroll
        for (int k = 0; k < kN; ++k) zero.p[k] = fill<kW>(0.f);
        store_state<kOut16>(a.out, (s * a.n + i) * a.c + c, zero);
      }
    }
  }
  if (a.final_state) store_state<false>(a.final_state, s * a.c + c, h);
}

template <bool kIn16, bool kOut16, bool kSig>
Kernel pick(int v, int tokens) {
  constexpr int kAtOnce = kIn16 ? 8 : 4;
  if (tokens == 1)
    return v == 4 ? scan_few_kernel<kIn16, kOut16, 4, kSig, 1, false>
                  : scan_few_kernel<kIn16, kOut16, 1, kSig, 1, false>;
  if (tokens <= kTokens)
    return v == 4 ? scan_few_kernel<kIn16, kOut16, 4, kSig, kTokens, false>
                  : scan_few_kernel<kIn16, kOut16, 1, kSig, kTokens, false>;
  return v == 4 ? scan_few_kernel<kIn16, kOut16, 4, kSig, kAtOnce, true>
                : scan_few_kernel<kIn16, kOut16, 1, kSig, 8, true>;
}
template <bool kIn16, bool kOut16>
Kernel pick(bool sig, int v, int tokens) {
  return sig ? pick<kIn16, kOut16, true>(v, tokens) : pick<kIn16, kOut16, false>(v, tokens);
}

}  // namespace

Kernel forward(bool in16, bool out16, bool sig, int v, int tokens) {
  return in16 ? (out16 ? pick<true, true>(sig, v, tokens) : pick<true, false>(sig, v, tokens))
              : (out16 ? pick<false, true>(sig, v, tokens) : pick<false, false>(sig, v, tokens));
}

}  // namespace few
}  // namespace scan
}  // namespace lapl
