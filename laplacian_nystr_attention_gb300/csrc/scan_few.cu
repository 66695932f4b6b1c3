// scan_few.cu -- the gated linear recurrence over few tokens, as a model that answers token by token
// calls it: scan.cu's formulas without its exchange.
//
// A thread has all tokens of four channels (one where rows or pointers are not multiples of four
// elements) and goes through the steps with the state in registers: of up to four tokens it reads all
// at once, of more some at a time with the next ones on their way.  With the sigmoid gate 128 x 1 x 4096
// bf16 takes 2.5 us where the kernel for longer sequences, 32 threads a CTA and 16 tokens a thread, takes
// 13; 64 x 1 x 512 1.7 and 3.3; 20000 x 2 x 512 31 (78% of the copy's rate) and 231; 64 x 8 x 4096 4.3 and
// 8.5.  The backward of up to eight tokens holds them all: 64 x 1 x 4096 2.1 and 9.6 us, 64 x 8 x 4096 8.4
// and 11.  What bounds them is the launch, then the bytes, and with many tokens a thread its own steps.
#include "scan_few.cuh"

namespace lapl {
namespace scan {
namespace few {
namespace {

// V channels of a token, 4, 2 or 1: pairs of them, or one.
template <int V>
struct Parts {
  static constexpr int kW = V >= 2 ? 2 : 1, kN = V / kW;
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
  if constexpr (V <= 2) {
    t.p[0] = load_raw<k16, V>(q);
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
  if constexpr (V <= 2) {
    store_vec<k16>(q, h.p[0]);
  } else if constexpr (k16) {
    *reinterpret_cast<uint2*>(q) = make_uint2(ops::pack_bf16(h.p[0].f[0], h.p[0].f[1]),
                                              ops::pack_bf16(h.p[1].f[0], h.p[1].f[1]));
  } else {
    *reinterpret_cast<float4*>(q) =
        make_float4(h.p[0].f[0], h.p[0].f[1], h.p[1].f[0], h.p[1].f[1]);
  }
}

// What a thread is: sequence, first channel, tokens of the sequence.
template <int V>
struct Spot {
  long long s;
  int c, len;
  bool on;
  __device__ __forceinline__ explicit Spot(const Args& a) {
    const int unit = blockIdx.x / a.geo.blocks, block = blockIdx.x - unit * a.geo.blocks;
    s = (long long)unit * (kThreads >> a.geo.lanes_log2) + (threadIdx.x >> a.geo.lanes_log2);
    c = (block * a.geo.lanes + ((int)threadIdx.x & (a.geo.lanes - 1))) * V;
    on = s < a.sequences && c < a.c;
    len = on && a.lengths ? max(0, min(a.n, a.lengths[s])) : a.n;
  }
  // Row of the i-th token in processing order.
  __device__ __forceinline__ long long row(const Args& a, int i) const {
    return s * a.n + (a.reverse ? len - 1 - i : i);
  }
};
// The sigmoid gate's smaller side, -z or a by its sign: h + z (x - h) or x - a (x - h), and D - z D or
// a D, without the rounding of the other one.  A state that is handed on from call to call goes through
// thousands of steps, and an error of a that they share grows to 2^-24 / z.  (The decay gate: a.)
template <bool kSig, int V>
struct Side {
  Vec<V> n;
  Side() = default;
  __device__ __forceinline__ explicit Side(const Gate<V>& gate) : n(gate.a) {
    if constexpr (kSig)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (gate.z.f[i] < 0.5f) n.f[i] = -gate.z.f[i];
  }
  __device__ __forceinline__ bool open(int i) const { return __float_as_int(n.f[i]) < 0; }
  // h after a step.
  __device__ __forceinline__ Vec<V> step(const Vec<V>& x, const Vec<V>& h) const {
    if constexpr (!kSig) return fma(n, h, x);
    Vec<V> from;
#pragma unroll
    for (int i = 0; i < V; ++i) from.f[i] = open(i) ? h.f[i] : x.f[i];
    return fma(n, sub(h, x), from);
  }
  // The slope of a step in its decay: of a z with the sigmoid gate.
  __device__ __forceinline__ Vec<V> slope(const Vec<V>& x, const Vec<V>& before) const {
    return kSig ? sub(before, x) : before;
  }
  // From D: a D, and the step's gradients.
  __device__ __forceinline__ Vec<V> gradients(const Vec<V>& D, const Vec<V>& slope, Vec<V>& dx,
                                              Vec<V>& dg) const {
    if constexpr (!kSig) {
      dx = D;
      dg = mul(slope, D);
      return mul(n, D);
    }
    Vec<V> less, E;
#pragma unroll
    for (int i = 0; i < V; ++i) less.f[i] = fabsf(n.f[i]);
    const Vec<V> small = mul(less, D), large = sub(D, small);
    dg = mul(slope, mul(less, large));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dx.f[i] = open(i) ? small.f[i] : large.f[i];
      E.f[i] = open(i) ? large.f[i] : small.f[i];
    }
    return E;
  }
};
template <int V>
__device__ __forceinline__ State<V> zeros() {
  State<V> h;
#pragma unroll
  for (int k = 0; k < Parts<V>::kN; ++k) h.p[k] = fill<Parts<V>::kW>(0.f);
  return h;
}
template <int V>
__device__ __forceinline__ State<V> load_state(const float* base, long long e) {
  const Token<false, V> t = load_token<false, V>(base, e);
  State<V> h;
#pragma unroll
  for (int k = 0; k < Parts<V>::kN; ++k) h.p[k] = widen(t.p[k]);
  return h;
}

// T: tokens at a time; kMore: and the next T on their way while those are worked on.
template <bool kIn16, bool kOut16, int V, bool kSig, int T, bool kMore>
__global__ void __launch_bounds__(kThreads) scan_few_kernel(const Args a) {
  constexpr int kN = Parts<V>::kN;
  const Spot<V> spot(a);
  if (!spot.on) return;
  const long long s = spot.s;
  const int c = spot.c, len = spot.len;
  State<V> h = zeros<V>();
  Token<kIn16, V> x[T], g[T];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < T; ++u)
      if (i0 + u < len) {
        g[u] = load_token<kIn16, V>(a.g, spot.row(a, i0 + u) * a.g_stride + c);
        x[u] = load_token<kIn16, V>(a.x, spot.row(a, i0 + u) * a.x_stride + c);
      }
  };
  fetch(0);
  if (a.h0) h = load_state<V>(a.h0, s * a.c + c);
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
          h.p[k] = Side<kSig, Parts<V>::kW>(gate_of<kSig>(ng[u].p[k])).step(widen(nx[u].p[k]), h.p[k]);
        store_state<kOut16>(a.out, spot.row(a, i) * a.c + c, h);
      } else if (i < a.n) {
        store_state<kOut16>(a.out, (s * a.n + i) * a.c + c, zeros<V>());
      }
    }
  }
  if (a.final_state) store_state<false>(a.final_state, s * a.c + c, h);
}

// Backward of up to T tokens, all in registers.
template <bool kIn16, bool kGrad16, int V, bool kSig, int T>
__global__ void __launch_bounds__(kThreads) scan_few_backward_kernel(const Args a) {
  constexpr int kN = Parts<V>::kN;
  const Spot<V> spot(a);
  if (!spot.on) return;
  const long long s = spot.s;
  const int c = spot.c, len = spot.len;
  Token<kIn16, V> x[T], g[T];
  Token<kGrad16, V> dh[T];
#pragma unroll
  for (int i = 0; i < T; ++i)
    if (i < len) {
      const long long row = spot.row(a, i);
      g[i] = load_token<kIn16, V>(a.g, row * a.g_stride + c);
      x[i] = load_token<kIn16, V>(a.x, row * a.x_stride + c);
      dh[i] = load_token<kGrad16, V>(a.dout, row * a.c + c);
    }
  State<V> h = load_state<V>(a.states, s * a.c + c), E = zeros<V>();   // one kept state a sequence
  if (a.dfinal) E = load_state<V>(a.dfinal, s * a.c + c);
  Side<kSig, Parts<V>::kW> gate[T][kN];
  State<V> slope[T];
#pragma unroll
  for (int i = 0; i < T; ++i)
    if (i < len)
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const auto in = widen(x[i].p[k]);
        gate[i][k] = Side<kSig, Parts<V>::kW>(gate_of<kSig>(g[i].p[k]));
        slope[i].p[k] = gate[i][k].slope(in, h.p[k]);
        h.p[k] = gate[i][k].step(in, h.p[k]);
      }
#pragma unroll
  for (int i = T - 1; i >= 0; --i) {
    if (i >= a.n) continue;
    State<V> dx = zeros<V>(), dg = zeros<V>();
    if (i < len)
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const auto D = add(widen(dh[i].p[k]), E.p[k]);
        E.p[k] = gate[i][k].gradients(D, slope[i].p[k], dx.p[k], dg.p[k]);
      }
    const long long row = i < len ? spot.row(a, i) : s * a.n + i;
    store_state<kGrad16>(a.dx, row * a.x_stride + c, dx);
    store_state<kGrad16>(a.dg, row * a.g_stride + c, dg);
  }
  if (a.dh0) store_state<false>(a.dh0, s * a.c + c, E);
}

template <bool kIn16, bool kGrad16, bool kSig>
Kernel pick_backward(int v, int tokens) {
  if (tokens == 1)
    return v == 4 ? scan_few_backward_kernel<kIn16, kGrad16, 4, kSig, 1>
                  : scan_few_backward_kernel<kIn16, kGrad16, 1, kSig, 1>;
  if (tokens <= kTokens)
    return v == 4 ? scan_few_backward_kernel<kIn16, kGrad16, 4, kSig, kTokens>
                  : scan_few_backward_kernel<kIn16, kGrad16, 1, kSig, kTokens>;
  return v == 2 ? scan_few_backward_kernel<kIn16, kGrad16, 2, kSig, kBackwardTokens>
                : scan_few_backward_kernel<kIn16, kGrad16, 1, kSig, kBackwardTokens>;
}
template <bool kIn16, bool kGrad16>
Kernel pick_backward(bool sig, int v, int tokens) {
  return sig ? pick_backward<kIn16, kGrad16, true>(v, tokens)
             : pick_backward<kIn16, kGrad16, false>(v, tokens);
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
Kernel backward(bool in16, bool grad16, bool sig, int v, int tokens) {
  return in16 ? (grad16 ? pick_backward<true, true>(sig, v, tokens)
                        : pick_backward<true, false>(sig, v, tokens))
              : (grad16 ? pick_backward<false, true>(sig, v, tokens)
                        : pick_backward<false, false>(sig, v, tokens));
}

}  // namespace few
}  // namespace scan
}  // namespace lapl
