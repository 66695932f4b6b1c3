// rope.cu -- a projection's rows as heads, with the norm of each query and key head and the rotary
// positions: lapl_rope_* of include/lapl_ops.h.
//
//   y = R(x rstd w),  rstd = 1 / sqrt(mean(x^2) + eps);  backward, with g = R^T dy, t = g w, u = x rstd:
//   dx = rstd (t - u mean(t u)),  dw = sum over rows of g u.
//
// HBM-bound: every value is read and written once.  A CTA takes a few tokens, all their heads: the
// tokens' cosines and sines are formed once, in shared memory, for all heads of q and k.  A group of
// lanes takes a row (a token's head); a lane has two vectors of it that hold whole pairs (of a head's two
// halves, or next to each other), so that turning needs no exchange and the norm one sum over the group.
// Rows are taken token after token within a head, so that what a CTA writes to a head is one run.
//
// Angles.  A position times a frequency in fp32 is off by 2^-24 of itself: half a radian at 2^23.  A
// frequency is held as a 64-bit fraction of a turn instead, whose product with a 32-bit position, modulo
// a turn, is one integer multiplication and off by 2^-33 of a turn; what is left, half a turn either way, is
// rounded to fp32, which is off by 2^-26 of a turn at most, as much as half a unit of cosine and sine makes out.
//
// Measured, of 6.8 TB/s: 4 x 16384 tokens of 24 heads of 64, bf16, forward 98 us (4.1 TB/s of 403 MB) with
// instructions issued in 63% of the cycles, some 25 a value; backward 134 us (4.0 TB/s of 537 MB), 55%,
// with the 16 warps of an SM that registers allow.  8 x 3136 tokens of 6 heads of 32 in fp32 16 us,
// a token 3.3 us.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "ops_common.cuh"

namespace lapl {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxPairs = LAPL_ROPE_MAX_DIM / 2;
constexpr int kTokens = 16, kMaxTokens = 32;   // tokens of a CTA at a time, powers of two
// Rows of a group in flight, forward.
constexpr int rows_of(int vec) { return vec == 8 ? 3 : 4; }
constexpr int back_rows_of(int vec) { return vec == 8 ? 1 : 2; }   // and backward, of two tensors
constexpr int kBackCtas = 2;   // CTAs of an SM, by registers (3 with 80 registers: spills, and no faster)

struct Part {            // q, k or v
  const void* in;        // rows [B,N,heads*d]  (backward: what it was, or null without a norm)
  void* out;             // [B,heads,N,d]       (backward: null)
  const void* grad;      // backward: gradient [B,heads,N,d]
  void* din;             // backward: gradient of the rows
  const float* weight;
  int heads;             // of the launch
  int all_heads;
  int stride;
};
struct Args {
  Part part[3];
  const int* positions;
  float* partial;        // backward: [CTAs][2][d] sums as pairs of floats
  unsigned long long turn[kMaxPairs];   // frequencies, in 2^-64 of a turn
  long long rows;        // B * N tokens
  int tokens, d, pairs, axes, first1, first2;   // first1, first2: first pairs of axes 1 and 2
  int at_once;           // tokens of a CTA at a time, a power of two
  int lanes_log2;        // lanes of a row
  int norm;
  float eps;
};

// V values as they are in memory, in words of 32 bits (one bf16 value: in the low half).
template <int V, bool kHalf>
struct Raw {
  static constexpr int kWords = kHalf ? (V + 1) / 2 : V;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* p, long long at) {
    constexpr int kBytes = V * (kHalf ? 2 : 4);
    const char* q = static_cast<const char*>(p) + at * (kHalf ? 2 : 4);
    if constexpr (kBytes == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(q);
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(q);
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(q);
      w[0] = v.x, w[1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(q);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (!kHalf) return __uint_as_float(w[i]);
    return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
};
template <int V, bool kHalf>
__device__ __forceinline__ void store(void* p, long long at, const float (&x)[V]) {
  char* q = static_cast<char*>(p) + at * (kHalf ? 2 : 4);
  if constexpr (kHalf && V == 1) {
    *reinterpret_cast<uint16_t*>(q) = (uint16_t)ops::pack_bf16(x[0], 0.f);
  } else {
    uint32_t w[Raw<V, kHalf>::kWords];
#pragma unroll
    for (int i = 0; i < Raw<V, kHalf>::kWords; ++i)
      w[i] = kHalf ? ops::pack_bf16(x[2 * i % V], x[(2 * i + 1) % V]) : __float_as_uint(x[i % V]);
    if constexpr (sizeof(w) == 4) *reinterpret_cast<uint32_t*>(q) = w[0];
    else if constexpr (sizeof(w) == 8) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The two vectors of a lane's slot: where they start in a head, whether they are there, and the first
// pair that each turns, or -1.  Pairs of a head's halves: the first pairs / V slots are turned, a vector of
// one half and one of the other; the rest hold the values after them.  Interleaved: a head's vectors in
// their order, which hold whole pairs each.
template <int V, bool kInterleaved>
struct Slot {
  int at[2];
  bool on[2];
  int pair[2];
  __device__ __forceinline__ Slot(int s, int d, int pairs) {
    if (kInterleaved && V > 1) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        at[e] = V * (2 * s + e);
        on[e] = at[e] < d;
        pair[e] = at[e] < 2 * pairs ? at[e] / 2 : -1;
      }
    } else if (s < pairs / V) {
      at[0] = kInterleaved ? 2 * s : V * s;
      at[1] = kInterleaved ? 2 * s + 1 : at[0] + pairs;
      on[0] = on[1] = true;
      pair[0] = pair[1] = V * s;
    } else {
      at[0] = 2 * pairs + 2 * V * (s - pairs / V);
      at[1] = at[0] + V;
      on[0] = at[0] < d;
      on[1] = at[1] < d;
      pair[0] = pair[1] = -1;
    }
  }
};

// Where the cosine and sine of the CTA's i-th (token, pair) are: 16-byte units of two pairs, spread so that
// eight lanes' units a vector or two apart lie in different banks.
__device__ __forceinline__ int turn_at(int i) {
  const int u = i >> 1;
  return (u ^ ((u >> 2) & 7)) * 2 + (i & 1);
}
__host__ __device__ __forceinline__ int turns_of(int n) { return (n + 15) & ~15; }   // room

// V floats of shared memory that start on a vector.
template <int V>
__device__ __forceinline__ void read(float (&x)[V], const float* p) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
    }
  } else if constexpr (V == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    x[0] = f.x, x[1] = f.y;
  } else {
    x[0] = *p;
  }
}

// Turns x, y by the angle.
template <bool kBack>
__device__ __forceinline__ void turn_one(float& x, float& y, float c, float s) {
  if (kBack) s = -s;
  const float p = x, q = y;
  x = fmaf(p, c, -(q * s));
  y = fmaf(q, c, p * s);
}
// Turns a slot's pairs (back with kBack); first: the token's first place among the turns.
template <int V, bool kInterleaved, bool kBack>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const Slot<V, kInterleaved>& s,
                                     const float2* cs, int first) {
  if constexpr (V == 1) {
    if (s.pair[0] < 0) return;
    const float2 t = cs[turn_at(first + s.pair[0])];
    turn_one<kBack>(a[0], b[0], t.x, t.y);
  } else if constexpr (kInterleaved) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (s.pair[e] < 0) continue;
      float (&x)[V] = e ? b : a;
      if constexpr (V == 2) {
        const float2 t = cs[turn_at(first + s.pair[e])];
        turn_one<kBack>(x[0], x[1], t.x, t.y);
      } else {
#pragma unroll
        for (int i = 0; i < V / 2; i += 2) {
          const float2 t = cs[turn_at(first + s.pair[e] + i)], u = cs[turn_at(first + s.pair[e] + i + 1)];
          turn_one<kBack>(x[2 * i], x[2 * i + 1], t.x, t.y);
          turn_one<kBack>(x[2 * i + 2], x[2 * i + 3], u.x, u.y);
        }
      }
    }
  } else {
    if (s.pair[0] < 0) return;
#pragma unroll
    for (int i = 0; i < V; i += 2) {   // (a token's pairs are a multiple of V: even places)
      const float4 t = *reinterpret_cast<const float4*>(cs + turn_at(first + s.pair[0] + i));
      turn_one<kBack>(a[i], b[i], t.x, t.y);
      turn_one<kBack>(a[i + 1], b[i + 1], t.z, t.w);
    }
  }
}

// cos and sin of `count` tokens' pairs from token `first` on, zeros for the others of the CTA's.
__device__ __forceinline__ void fill_turns(float2* cs, const Args& a, long long first, int count) {
  for (int i = threadIdx.x; i < a.at_once * a.pairs; i += kThreads) {
    const int t = i / a.pairs, p = i - t * a.pairs;
    if (t >= count) {
      cs[turn_at(i)] = make_float2(0.f, 0.f);
      continue;
    }
    const int axis = (p >= a.first1) + (p >= a.first2);
    const long long pos = a.positions[(first + t) * a.axes + axis];
    const long long part = (long long)(a.turn[p] * (unsigned long long)pos);   // signed: -1/2 .. 1/2
    float s, c;
    sincospif(__ll2float_rn(part) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
    cs[turn_at(i)] = make_float2(c, s);
  }
}

// Both weights in shared memory, ones where there are none, [2][padded].
__host__ __device__ __forceinline__ int padded(int d) { return (d + 7) & ~7; }
__device__ __forceinline__ void fill_weights(float* w, const Args& a) {
  for (int i = threadIdx.x; i < 2 * padded(a.d); i += kThreads) {
    const int which = i >= padded(a.d), e = i - which * padded(a.d);
    const float* from = which ? a.part[1].weight : a.part[0].weight;
    w[i] = from && e < a.d ? from[e] : 1.f;
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A group's token of the CTA's tokens from `first` on, and its places in all parts: of head 0, and from
// there to the next heads.
struct Place {
  bool live;
  int token;            // of the CTA's
  long long in[3], out[3];
  __device__ __forceinline__ Place(const Args& a, long long first, int token_of_group) {
    token = token_of_group;
    const unsigned at = (unsigned)first + (unsigned)token;
    live = at < (unsigned long long)a.rows;
    const unsigned b = at / (unsigned)a.tokens, n = at - b * (unsigned)a.tokens;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      in[i] = (long long)at * a.part[i].stride;
      out[i] = ((long long)b * a.part[i].all_heads * a.tokens + n) * a.d;
    }
  }
};

template <int V, int NS, bool kInterleaved, bool kHalfIn, bool kHalfOut>
__global__ void __launch_bounds__(kThreads, 3)
rope_forward_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) float smem[];
  constexpr int kRows = rows_of(V);
  const int pad = padded(a.d);
  const float* weights = smem;
  float2* cs = reinterpret_cast<float2*>(smem + 2 * pad);
  if (a.norm) {
    fill_weights(smem, a);
    __syncthreads();
  }
  const int lanes = 1 << a.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int group = threadIdx.x >> a.lanes_log2, groups = kThreads >> a.lanes_log2;
  const float inv_d = 1.f / (float)a.d;
  // A group has one of the tokens, and every step-th head of it.
  const int token = group & (a.at_once - 1), head0 = group / a.at_once, step = groups / a.at_once;
  const int heads_q = a.part[0].heads, heads_qk = heads_q + a.part[1].heads;
  const int heads = heads_qk + a.part[2].heads;
  const long long plane = (long long)a.tokens * a.d;
  const Slot<V, kInterleaved> slot0(lane, a.d, a.pairs);
  for (long long first = (long long)blockIdx.x * a.at_once; first < a.rows;
       first += (long long)gridDim.x * a.at_once) {
    const int count = (int)min((long long)a.at_once, a.rows - first);
    const Place place(a, first, token);
    Raw<V, kHalfIn> raw[kRows][NS][2];
    auto load = [&](int h0) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (h0 - head0 + u * step >= heads) break;   // (no group has a row there)
        const int h = h0 + u * step, which = (h >= heads_q) + (h >= heads_qk);
        const int head = h - (which == 0 ? 0 : which == 1 ? heads_q : heads_qk);
        const long long at = (which == 0 ? place.in[0] : which == 1 ? place.in[1] : place.in[2]) +
                             (long long)head * a.d;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const Slot<V, kInterleaved> s = NS == 1 ? slot0 : Slot<V, kInterleaved>(lane + j * lanes, a.d, a.pairs);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (place.live && h < heads && s.on[e]) raw[u][j][e].load(a.part[which].in, at + s.at[e]);
            else raw[u][j][e].zero();
          }
        }
      }
    };
    load(head0);   // on their way while the turns are formed
    if (a.pairs) {
      __syncthreads();   // the last tokens' turns are used up
      fill_turns(cs, a, first, count);
      __syncthreads();
    }
#pragma unroll 1
    for (int h0 = head0; h0 - head0 < heads; h0 += kRows * step) {
      if (h0 != head0) load(h0);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (h0 - head0 + u * step >= heads) break;
        const int h = h0 + u * step, which = (h >= heads_q) + (h >= heads_qk);
        const int head = h - (which == 0 ? 0 : which == 1 ? heads_q : heads_qk);
        float x[NS][2][V];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              x[j][e][i] = raw[u][j][e].value(i);
              sum = fmaf(x[j][e][i], x[j][e][i], sum);
            }
        const bool norm = a.norm && which < 2;
        float rstd = 1.f;
        if (a.norm) rstd = rsqrtf(fmaf(group_sum(sum, lanes), inv_d, a.eps));   // off by 2 units
        if (!place.live || h >= heads) continue;
        const float* weight = weights + (which ? pad : 0);
        const long long at = (which == 0 ? place.out[0] : which == 1 ? place.out[1] : place.out[2]) + head * plane;
        void* out = a.part[which].out;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const Slot<V, kInterleaved> s = NS == 1 ? slot0 : Slot<V, kInterleaved>(lane + j * lanes, a.d, a.pairs);
          if (norm) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float w[V];
              read<V>(w, weight + (s.on[e] ? s.at[e] : 0));
#pragma unroll
              for (int i = 0; i < V; ++i) x[j][e][i] *= rstd * w[i];
            }
          }
          if (which < 2)
            turn<V, kInterleaved, false>(x[j][0], x[j][1], s, cs, place.token * a.pairs);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (s.on[e]) store<V, kHalfOut>(out, at + s.at[e], x[j][e]);
        }
      }
    }
  }
}

// Adds what the CTA's threads have of a weight's gradient to its sums in shared memory, in pairs of
// floats and a fixed order: a warp's groups by shuffles, then warp after warp.
template <int V, int NS, bool kInterleaved>
__device__ __forceinline__ void add_to_sums(const Args& a, const float (&dw)[NS][2][V], float2* sums,
                                            int lane, int lanes) {
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const Slot<V, kInterleaved> s(lane + j * lanes, a.d, a.pairs);
    ops::Pair v[2][V];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[e][i] = {dw[j][e][i], 0.f};
        for (int o = lanes; o < 32; o *= 2) {
          const float hi = __shfl_xor_sync(0xffffffffu, v[e][i].hi, o);
          v[e][i].add(hi, __shfl_xor_sync(0xffffffffu, v[e][i].lo, o));
        }
      }
    for (int w = 0; w < kThreads / 32; ++w) {
      __syncthreads();
      if (w != warp || (threadIdx.x & 31) >= lanes) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (s.on[e]) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 old = sums[s.at[e] + i];
            ops::Pair sum = {old.x, old.y};
            sum.add(v[e][i].hi, v[e][i].lo);
            sums[s.at[e] + i] = make_float2(sum.hi, sum.lo);
          }
        }
    }
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p, long long bytes) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const unsigned char*>(p) + bytes));
}

// dw: a thread's rows are summed in fp32, fewer than 2 kSummed of them, what follows in pairs of floats.
// (Whole tiles are summed: a launch has no more heads than give a thread kSummed rows of a tile.  Turns of so
// many heads within the kernel took 139 us for what takes 135 of 4 x 16384 tokens of 24 heads of 64.)
constexpr int kSummed = 64;
template <int V, int NS, bool kInterleaved, bool kHalfIn, bool kHalfGrad>
__global__ void __launch_bounds__(kThreads, kBackCtas)
rope_backward_kernel(const __grid_constant__ Args a) {
  constexpr int kBackRows = back_rows_of(V);
  extern __shared__ __align__(16) float smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int pad = padded(a.d);
  float2* cs = reinterpret_cast<float2*>(smem + 2 * pad);
  float2* sums = cs + turns_of(a.pairs * a.at_once);   // [2][d]
  if (a.norm) {
    fill_weights(smem, a);
    __syncthreads();
  }
  const int lanes = 1 << a.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int group = threadIdx.x >> a.lanes_log2, groups = kThreads >> a.lanes_log2;
  const float inv_d = 1.f / (float)a.d;
  const int token = group & (a.at_once - 1), head0 = group / a.at_once, step = groups / a.at_once;
  const long long plane = (long long)a.tokens * a.d;
  const Slot<V, kInterleaved> slot0(lane, a.d, a.pairs);
  auto slot = [&](int j) { return NS == 1 ? slot0 : Slot<V, kInterleaved>(lane + j * lanes, a.d, a.pairs); };
  if (a.partial)
    for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) sums[i] = make_float2(0.f, 0.f);
  float dw[2][NS][2][V];
  auto clear = [&] {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < V; ++i) dw[w][j][e][i] = 0.f;
  };
  clear();
  const int rows_of_tile = (max(a.part[0].heads, a.part[1].heads) + step - 1) / step;
  int summed = 0;
  for (long long first = (long long)blockIdx.x * a.at_once; first < a.rows;
       first += (long long)gridDim.x * a.at_once) {
    const int count = (int)min((long long)a.at_once, a.rows - first);
    const Place place(a, first, token);
    Raw<V, kHalfGrad> rg[kBackRows][NS][2];
    Raw<V, kHalfIn> rx[kBackRows][NS][2];
    auto load = [&](int which, int h0) {
      const Part& p = a.part[which];
#pragma unroll
      for (int u = 0; u < kBackRows; ++u) {
        if (h0 - head0 + u * step >= p.heads) break;   // (no group has a row there)
        const int h = h0 + u * step;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const Slot<V, kInterleaved> s = slot(j);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool on = place.live && h < p.heads && s.on[e];
            rg[u][j][e].zero();
            rx[u][j][e].zero();
            if (on) rg[u][j][e].load(p.grad, place.out[which] + h * plane + s.at[e]);
            if (on && which < 2 && a.norm)
              rx[u][j][e].load(p.in, place.in[which] + (long long)h * a.d + s.at[e]);
          }
        }
      }
    };
    // Rows into L2, on their way while the ones before are worked on, which a thread's registers have no room
    // for (without it 155 us instead of 134 of 4 x 16384 tokens of 24 heads of 64).
    auto prefetch = [&](int which, int h) {
      const Part& p = a.part[which];
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const Slot<V, kInterleaved> s = slot(j);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!place.live || h >= p.heads || !s.on[e]) continue;
          prefetch_l2(p.grad, (place.out[which] + h * plane + s.at[e]) * (kHalfGrad ? 2 : 4));
          if (which < 2 && a.norm)
            prefetch_l2(p.in, (place.in[which] + (long long)h * a.d + s.at[e]) * (kHalfIn ? 2 : 4));
        }
      }
    };
    load(0, head0);   // on their way while the turns are formed
    if (a.pairs) {
      __syncthreads();   // the last tokens' turns are used up
      fill_turns(cs, a, first, count);
      __syncthreads();
    }
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      const Part& p = a.part[which];
      const bool norm = which < 2 && a.norm;
#pragma unroll 1
      for (int h0 = head0; h0 - head0 < p.heads; h0 += kBackRows * step) {
        if (which > 0 || h0 != head0) load(which, h0);
#pragma unroll
        for (int u = 0; u < kBackRows; ++u) {
          const int h = h0 + (kBackRows + u) * step;
          if (h0 + kBackRows * step - head0 < p.heads) prefetch(which, h);
          else if (which < 2) prefetch(which + 1, head0 + u * step);
        }
#pragma unroll
        for (int u = 0; u < kBackRows; ++u) {
          if (h0 - head0 + u * step >= p.heads) break;
          const int h = h0 + u * step;
          const bool live = place.live && h < p.heads;
          float x[NS][2][V], g[NS][2][V];
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            const Slot<V, kInterleaved> s = slot(j);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < V; ++i) {
                g[j][e][i] = rg[u][j][e].value(i);
                x[j][e][i] = rx[u][j][e].value(i);
                sum = fmaf(x[j][e][i], x[j][e][i], sum);
              }
            if (which < 2)
              turn<V, kInterleaved, true>(g[j][0], g[j][1], s, cs, place.token * a.pairs);
          }
          if (norm) {
            // (Rows that are not there: all zeros, whose rstd may be infinite.  Rounded in full, rstd left fp32
            // gradients 9.2e-8 off instead of 1.0e-7, and the kernel 3% slower.)
            const float mean = fmaf(group_sum(sum, lanes), inv_d, a.eps);
            const float rstd = live ? rsqrtf(mean) : 0.f;   // off by 2 units
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              const Slot<V, kInterleaved> s = slot(j);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float w[V];
                read<V>(w, smem + (which ? pad : 0) + (s.on[e] ? s.at[e] : 0));
#pragma unroll
                for (int i = 0; i < V; ++i) {
                  const float v = x[j][e][i] * rstd;
                  x[j][e][i] = v;
                  dw[which & 1][j][e][i] = fmaf(g[j][e][i], v, dw[which & 1][j][e][i]);
                  g[j][e][i] *= w[i];
                  dot = fmaf(g[j][e][i], v, dot);
                }
              }
            }
            dot = group_sum(dot, lanes) * inv_d;
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < V; ++i)
                  g[j][e][i] = rstd * fmaf(-x[j][e][i], dot, g[j][e][i]);
          }
          if (live) {
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              const Slot<V, kInterleaved> s = slot(j);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (s.on[e])
                  store<V, kHalfGrad>(p.din, place.in[which] + (long long)h * a.d + s.at[e], g[j][e]);
            }
          }
        }
      }
    }
    summed += rows_of_tile;
    if (a.partial && (summed >= kSummed || first + (long long)gridDim.x * a.at_once >= a.rows)) {
#pragma unroll
      for (int which = 0; which < 2; ++which)
        add_to_sums<V, NS, kInterleaved>(a, dw[which], sums + which * a.d, lane, lanes);
      clear();
      summed = 0;
    }
  }
  if (a.partial) {
    __syncthreads();
    float2* out = reinterpret_cast<float2*>(a.partial) + (long long)blockIdx.x * 2 * a.d;
    for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) out[i] = sums[i];
  }
}

// The weights' gradients from all partials: a warp for each of 2 d values, in a fixed order.  (304 CTAs'
// partials of 64 values: 8 us from a cold cache, one load deep.)
__global__ void __launch_bounds__(kThreads)
rope_weights_kernel(const float2* partial, int parts, int d, float* dq, float* dk) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are written
  const int lane = threadIdx.x & 31, i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  float* out = i < d ? dq : dk;
  if (i >= 2 * d || !out) return;
  ops::Pair s = {0.f, 0.f};
  for (int k = lane; k < parts; k += 32) {
    const float2 v = partial[(long long)k * 2 * d + i];
    s.add(v.x, v.y);
  }
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_down_sync(0xffffffffu, s.hi, o);
    s.add(hi, __shfl_down_sync(0xffffffffu, s.lo, o));
  }
  if (lane == 0) out[i < d ? i : i - d] = s.value();
}

// kernel<...>(V, slots of a lane, interleaved, types) as a function pointer.
using Kernel = void (*)(const Args);
template <bool kBackward, int V, int NS, bool kInterleaved>
Kernel by_type(bool half_in, bool half_out) {
  if constexpr (kBackward) {
    if (half_in) return half_out ? rope_backward_kernel<V, NS, kInterleaved, true, true>
                                 : rope_backward_kernel<V, NS, kInterleaved, true, false>;
    return half_out ? rope_backward_kernel<V, NS, kInterleaved, false, true>
                    : rope_backward_kernel<V, NS, kInterleaved, false, false>;
  } else {
    if (half_in) return half_out ? rope_forward_kernel<V, NS, kInterleaved, true, true>
                                 : rope_forward_kernel<V, NS, kInterleaved, true, false>;
    return half_out ? rope_forward_kernel<V, NS, kInterleaved, false, true>
                    : rope_forward_kernel<V, NS, kInterleaved, false, false>;
  }
}
template <bool kBackward, bool kInterleaved>
Kernel by_shape(int vec, int ns, bool half_in, bool half_out) {
  // 16 bytes of both types.
  if (vec == 8)
    return kBackward ? rope_backward_kernel<8, 1, kInterleaved, true, true>
                     : rope_forward_kernel<8, 1, kInterleaved, true, true>;
  if (vec == 4) return by_type<kBackward, 4, 1, kInterleaved>(half_in, half_out);
  if (vec == 2 && ns == 1) return by_type<kBackward, 2, 1, kInterleaved>(half_in, half_out);
  if (vec == 2) return by_type<kBackward, 2, 2, kInterleaved>(half_in, half_out);
  if (ns == 1) return by_type<kBackward, 1, 1, kInterleaved>(half_in, half_out);
  if (ns == 2) return by_type<kBackward, 1, 2, kInterleaved>(half_in, half_out);
  return by_type<kBackward, 1, 4, kInterleaved>(half_in, half_out);
}

}  // namespace rope
}  // namespace lapl

struct lapl_rope_plan {
  lapl_rope_config cfg;
  lapl::rope::Args args;    // sizes, strides and turns
  int sms, device;
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

// Largest frequency, a power of 2: what turns() cuts off 1 / (2 pi), times this, is 2^-128 of a turn.
constexpr double kMostRadians = 3.402823669209384634634e38;   // 2^128

lapl_status validate(const lapl_rope_config* c) {
  if (!c || c->batch < 0 || c->tokens < 1 || c->q_heads < 1 || c->k_heads < 0 || c->v_heads < 0 ||
      c->head_dim < 1 || c->axes < 1 || c->axes > 3 || !c->pairs)
    return LAPL_ERR_INVALID_ARG;
  if (c->interleaved < 0 || c->interleaved > 1 || c->norm < 0 || c->norm > 1 || !(c->eps >= 0.f) ||
      !std::isfinite(c->eps))
    return LAPL_ERR_INVALID_ARG;
  if (!ops::is_float_dtype(c->in_dtype) || !ops::is_float_dtype(c->out_dtype) ||
      !ops::is_float_dtype(c->grad_dtype))
    return LAPL_ERR_INVALID_ARG;
  if (c->head_dim > LAPL_ROPE_MAX_DIM || c->q_heads > 4096 || c->k_heads > 4096 || c->v_heads > 4096 ||
      (long long)c->batch * c->tokens > (1LL << 31) - 1)
    return LAPL_ERR_UNSUPPORTED;
  int pairs = 0;
  for (int i = 0; i < c->axes; ++i) {
    if (c->pairs[i] < 0 || c->pairs[i] > LAPL_ROPE_MAX_DIM) return LAPL_ERR_INVALID_ARG;
    pairs += c->pairs[i];
  }
  if (2 * pairs > c->head_dim || (pairs > 0 && !c->frequencies)) return LAPL_ERR_INVALID_ARG;
  for (int i = 0; i < pairs; ++i)
    if (!std::isfinite(c->frequencies[i])) return LAPL_ERR_INVALID_ARG;
  for (int i = 0; i < pairs; ++i)
    if (std::fabs(c->frequencies[i]) >= kMostRadians) return LAPL_ERR_UNSUPPORTED;
  const int heads[3] = {c->q_heads, c->k_heads, c->v_heads};
  const int strides[3] = {c->q_stride, c->k_stride, c->v_stride};
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0) return LAPL_ERR_INVALID_ARG;
    if (heads[i] > 0 && strides[i] != 0 && strides[i] < heads[i] * c->head_dim)
      return LAPL_ERR_INVALID_ARG;
  }
  return LAPL_OK;
}

// radians as a fraction of a turn, in 2^-64, rounded down.  In integers: a long double has as many bits as the
// machine likes, too few of them for more than some radians.
unsigned long long turns(double radians) {
  if (radians == 0.0) return 0;
  // 1 / (2 pi) in 2^-256, the first bits first.
  static const unsigned long long kInverse[4] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull,
                                                 0x36d8a5664f10e410ull, 0x7f9458eaf7aef158ull};
  int e = 0;
  const unsigned long long m = (unsigned long long)std::ldexp(std::frexp(std::fabs(radians), &e), 53);
  e -= 53;   // m 2^e radians
  unsigned long long product[6] = {};   // m / (2 pi) in 2^-256, the last bits first
  unsigned __int128 carry = 0;
  for (int i = 0; i < 4; ++i) {
    carry += (unsigned __int128)m * kInverse[3 - i];
    product[i] = (unsigned long long)carry;
    carry >>= 64;
  }
  product[4] = (unsigned long long)carry;
  const int at = 192 - e, word = at / 64, bit = at % 64;   // the fraction's last bit; e <= 75
  unsigned long long part = 0;
  if (word < 5) part = product[word] >> bit | (bit ? product[word + 1] << (64 - bit) : 0ull);
  // (Never a whole number of 2^-64: pi is not rational.)
  return radians < 0.0 ? ~part : part;
}

bool rows_fit(const void* p, int stride, int dtype, int vec) {
  return p == nullptr || (ops::aligned(p, (size_t)ops::dtype_bytes(dtype) * vec) && stride % vec == 0);
}
bool heads_fit(const void* p, int dtype, int vec) {
  return p == nullptr || ops::aligned(p, (size_t)ops::dtype_bytes(dtype) * vec);
}

// Widest vectors that hold whole pairs and that every row and head starts on.
int vector_of(const lapl_rope_plan& p, const rope::Args& a, bool backward) {
  const lapl_rope_config& c = p.cfg;
  const bool half = c.in_dtype == LAPL_BF16 && (backward ? c.grad_dtype : c.out_dtype) == LAPL_BF16;
  for (int vec = half ? 8 : 4; vec > 1; vec /= 2) {
    bool fits = a.d % vec == 0 && (c.interleaved ? 2 * a.pairs : a.pairs) % vec == 0;
    for (int i = 0; i < 3 && fits; ++i) {
      const rope::Part& t = a.part[i];
      if (t.heads == 0) continue;
      fits = rows_fit(t.in, t.stride, c.in_dtype, vec);
      if (!backward) fits = fits && heads_fit(t.out, c.out_dtype, vec);
      else fits = fits && heads_fit(t.grad, c.grad_dtype, vec) && rows_fit(t.din, t.stride, c.grad_dtype, vec);
    }
    if (fits) return vec;
  }
  return 1;
}

cudaError_t launch(const lapl_rope_plan& p, rope::Args& a, bool backward, int* ctas, cudaStream_t st) {
  const lapl_rope_config& c = p.cfg;
  const int vec = vector_of(p, a, backward);
  const int rest = a.d - 2 * a.pairs;
  const int slots = c.interleaved && vec > 1 ? (a.d + 2 * vec - 1) / (2 * vec)
                                             : a.pairs / vec + (rest + 2 * vec - 1) / (2 * vec);
  int lanes_log2 = 0;
  while (lanes_log2 < 5 && (1 << lanes_log2) < slots) ++lanes_log2;
  const int ns = (slots + 31) / 32;
  a.lanes_log2 = lanes_log2;
  // More tokens to a CTA where its groups of lanes would be more than their heads; fewer where that many
  // would not give a CTA to every SM.
  const int groups = rope::kThreads >> lanes_log2;
  const int heads = a.part[0].heads + (backward ? 0 : a.part[1].heads + a.part[2].heads);
  int at_once = std::min(rope::kTokens, groups);   // a group has one token of the CTA's at most
  while (at_once < std::min(rope::kMaxTokens, groups) && groups / at_once > heads) at_once *= 2;
  while (at_once > 1 && a.rows < (long long)at_once * 2 * p.sms) at_once /= 2;
  // Heads of a launch: with weights' gradients, no more than give a thread kSummed rows of a tile; fewer tokens
  // to a CTA first.
  int all = 0, some = 0;
  for (const rope::Part& t : a.part) all = std::max(all, t.heads);
  some = all;
  if (backward && a.partial) {
    while (at_once > 1 && groups / at_once * rope::kSummed < all) at_once /= 2;
    some = groups / at_once * rope::kSummed;
  }
  a.at_once = at_once;
  const long long tiles = (a.rows + at_once - 1) / at_once;
  const long long most = backward ? (long long)rope::kBackCtas * p.sms : 1LL << 30;
  const int grid = (int)std::min(tiles, most);
  *ctas = 0;
  const int ns_rounded = ns <= 1 ? 1 : ns == 2 ? 2 : 4;
  const bool hi = c.in_dtype == LAPL_BF16;
  const bool ho = (backward ? c.grad_dtype : c.out_dtype) == LAPL_BF16;
  rope::Kernel k;
  if (backward)
    k = c.interleaved ? rope::by_shape<true, true>(vec, ns_rounded, hi, ho)
                      : rope::by_shape<true, false>(vec, ns_rounded, hi, ho);
  else
    k = c.interleaved ? rope::by_shape<false, true>(vec, ns_rounded, hi, ho)
                      : rope::by_shape<false, false>(vec, ns_rounded, hi, ho);
  // Both weights, the turns, and in the backward both weights' sums.
  const size_t smem =
      sizeof(float2) *
                      (rope::padded(a.d) + rope::turns_of(a.pairs * at_once) + (backward ? 2 * a.d : 0));
  cudaError_t e = cudaSuccess;
  for (int low = 0; low < all && e == cudaSuccess; low += some) {
    rope::Args s = a;
    for (rope::Part& t : s.part) {
      const long long row = (long long)low * a.d, plane = row * a.tokens;
      auto moved = [](const void* q, long long n, int dtype) -> const void* {
        return q ? static_cast<const char*>(q) + n * ops::dtype_bytes(dtype) : nullptr;
      };
      t.heads = std::max(0, std::min(t.heads - low, some));
      t.in = moved(t.in, row, c.in_dtype);
      t.out = const_cast<void*>(moved(t.out, plane, c.out_dtype));
      t.grad = moved(t.grad, plane, c.grad_dtype);
      t.din = const_cast<void*>(moved(t.din, row, c.grad_dtype));
    }
    if (s.partial) s.partial += (long long)*ctas * 4 * a.d;
    k<<<grid, rope::kThreads, smem, st>>>(s);
    e = cudaGetLastError();
    *ctas += grid;
  }
  return e;
}

lapl_status check_pointers(std::initializer_list<std::pair<const void*, int>> list) {
  for (const auto& x : list)
    if (!ops::aligned(x.first, x.second)) return LAPL_ERR_ALIGNMENT;
  return LAPL_OK;
}

}  // namespace

extern "C" {

lapl_status lapl_rope_create(const lapl_rope_config* cfg, lapl_rope_handle* out) {
  if (!out) return LAPL_ERR_INVALID_ARG;
  *out = nullptr;
  const lapl_status st = validate(cfg);
  if (st != LAPL_OK) return st;
  int sms = 0, device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return LAPL_ERR_CUDA;
  lapl_rope_plan* p = new (std::nothrow) lapl_rope_plan();
  if (!p) return LAPL_ERR_INVALID_ARG;
  p->cfg = *cfg;
  p->sms = sms;
  p->device = device;
  rope::Args& a = p->args;
  a = {};
  int pairs[3] = {0, 0, 0};
  for (int i = 0; i < cfg->axes; ++i) pairs[i] = cfg->pairs[i];
  a.pairs = pairs[0] + pairs[1] + pairs[2];
  a.first1 = pairs[0];
  a.first2 = pairs[0] + pairs[1];
  if (cfg->axes < 3) a.first2 = rope::kMaxPairs;
  if (cfg->axes < 2) a.first1 = rope::kMaxPairs;
  for (int i = 0; i < a.pairs; ++i) a.turn[i] = turns(cfg->frequencies[i]);
  p->cfg.pairs = nullptr;          // the caller's, for the call only
  p->cfg.frequencies = nullptr;
  a.rows = (long long)cfg->batch * cfg->tokens;
  a.tokens = cfg->tokens;
  a.d = cfg->head_dim;
  a.axes = cfg->axes;
  a.norm = cfg->norm;
  a.eps = cfg->eps;
  const int heads[3] = {cfg->q_heads, cfg->k_heads, cfg->v_heads};
  const int strides[3] = {cfg->q_stride, cfg->k_stride, cfg->v_stride};
  for (int i = 0; i < 3; ++i) {
    a.part[i].heads = a.part[i].all_heads = heads[i];
    a.part[i].stride = strides[i] ? strides[i] : heads[i] * cfg->head_dim;
  }
  *out = p;
  return LAPL_OK;
}

lapl_status lapl_rope_workspace_size(lapl_rope_handle p, size_t* bytes) {
  if (!p || !bytes) return LAPL_ERR_INVALID_ARG;
  // Launches: a CTA of one token has 8 groups of lanes at least.
  const int heads = std::max(p->cfg.q_heads, std::max(p->cfg.k_heads, p->cfg.v_heads));
  const int least = rope::kThreads / 32 * rope::kSummed, launches = (heads + least - 1) / least;
  *bytes = align_up((size_t)launches * rope::kBackCtas * p->sms * 2 * p->cfg.head_dim * sizeof(float2), kAlign);
  return LAPL_OK;
}

lapl_status lapl_rope_forward(lapl_rope_handle p, const void* q, const void* k, const void* v,
                              const int* positions, const float* q_weight, const float* k_weight,
                              void* q_out, void* k_out, void* v_out, void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  const lapl_rope_config& c = p->cfg;
  if (!c.norm && (q_weight || k_weight)) return LAPL_ERR_INVALID_ARG;
  if (c.batch > 0) {
    if (!q || !q_out || (c.k_heads && (!k || !k_out)) || (c.v_heads && (!v || !v_out)) ||
        (p->args.pairs && !positions))
      return LAPL_ERR_INVALID_ARG;
  }
  const int i = ops::dtype_bytes(c.in_dtype), o = ops::dtype_bytes(c.out_dtype);
  lapl_status st = check_pointers({{q, i}, {k, i}, {v, i}, {positions, 4}, {q_weight, 4}, {k_weight, 4},
                                   {q_out, o}, {k_out, o}, {v_out, o}});
  if (st != LAPL_OK) return st;
  st = ops::check_device(p->device, p->last_error, "rope_forward/device");
  if (st != LAPL_OK || c.batch == 0) return st;
  rope::Args a = p->args;
  const void* in[3] = {q, k, v};
  void* out[3] = {q_out, k_out, v_out};
  const float* weight[3] = {q_weight, k_weight, nullptr};
  for (int n = 0; n < 3; ++n) {
    a.part[n].in = a.part[n].heads ? in[n] : nullptr;
    a.part[n].out = a.part[n].heads ? out[n] : nullptr;
    a.part[n].weight = weight[n];
  }
  a.positions = positions;
  int ctas = 0;
  const cudaError_t e = launch(*p, a, false, &ctas, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "rope_forward");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

lapl_status lapl_rope_backward(lapl_rope_handle p, const void* q, const void* k,
                               const int* positions, const float* q_weight, const float* k_weight,
                               const void* dq_out, const void* dk_out, const void* dv_out, void* dq,
                               void* dk, void* dv, float* dq_weight, float* dk_weight,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  const lapl_rope_config& c = p->cfg;
  if (!c.norm && (q_weight || k_weight || dq_weight || dk_weight)) return LAPL_ERR_INVALID_ARG;
  if (c.batch > 0) {
    if (!dq_out || !dq || (c.k_heads && (!dk_out || !dk)) || (c.v_heads && (!dv_out || !dv)) ||
        (p->args.pairs && !positions) || (c.norm && (!q || (c.k_heads && !k))))
      return LAPL_ERR_INVALID_ARG;
  }
  const bool weights = dq_weight || dk_weight;
  const int i = ops::dtype_bytes(c.in_dtype), g = ops::dtype_bytes(c.grad_dtype);
  lapl_status st = check_pointers({{q, i}, {k, i}, {positions, 4}, {q_weight, 4}, {k_weight, 4},
                                   {dq_out, g}, {dk_out, g}, {dv_out, g}, {dq, g}, {dk, g}, {dv, g},
                                   {dq_weight, 4}, {dk_weight, 4}});
  if (st != LAPL_OK) return st;
  if (weights) {
    size_t need = 0;
    lapl_rope_workspace_size(p, &need);
    if (!workspace) return LAPL_ERR_INVALID_ARG;
    if (!ops::aligned(workspace, 16)) return LAPL_ERR_ALIGNMENT;
    if (workspace_bytes < need) return LAPL_ERR_WORKSPACE;
  }
  st = ops::check_device(p->device, p->last_error, "rope_backward/device");
  if (st != LAPL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  int ctas = 0;
  if (c.batch > 0) {
    rope::Args a = p->args;
    const void* in[3] = {q, k, nullptr};
    const void* grad[3] = {dq_out, dk_out, dv_out};
    void* din[3] = {dq, dk, dv};
    const float* weight[3] = {q_weight, k_weight, nullptr};
    for (int n = 0; n < 3; ++n) {
      rope::Part& t = a.part[n];
      t.in = t.heads && c.norm ? in[n] : nullptr;
      t.grad = t.heads ? grad[n] : nullptr;
      t.din = t.heads ? din[n] : nullptr;
      t.weight = weight[n];
    }
    a.positions = positions;
    a.partial = weights ? static_cast<float*>(workspace) : nullptr;
    e = launch(*p, a, true, &ctas, s);
  }
  if (e == cudaSuccess && weights) {
    float* dkw = c.k_heads ? dk_weight : nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((2 * c.head_dim + rope::kThreads / 32 - 1) / (rope::kThreads / 32)));
    cfg.blockDim = dim3(rope::kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = c.batch > 0 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, rope::rope_weights_kernel, static_cast<const float2*>(workspace), ctas,
                           c.head_dim, dq_weight, dkw);
    if (e == cudaSuccess && dk_weight && !dkw)   // no key heads: nothing that depends on it
      e = cudaMemsetAsync(dk_weight, 0, sizeof(float) * c.head_dim, s);
  }
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "rope_backward");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

const char* lapl_rope_last_error(lapl_rope_handle p) { return p ? p->last_error : ""; }

lapl_status lapl_rope_destroy(lapl_rope_handle p) {
  delete p;
  return LAPL_OK;
}

}  // extern "C"
