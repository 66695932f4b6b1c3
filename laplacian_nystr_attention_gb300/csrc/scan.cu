// scan.cu -- gated linear recurrence over the tokens: lapl_scan_* of include/lapl_ops.h.
//
// Per sequence and channel, in processing order i = 0 .. len-1,
//   h_i = a_i h_{i-1} + b_i,   b = x (decay gate) or (1 - a) x (sigmoid gate),
// and backward, with E_i the gradient that step i hands to step i-1 (E_len = dfinal),
//   D_i = dh_i + E_{i+1},  E_i = a_i D_i,  dx_i = D_i or (1 - a_i) D_i,
//   dg_i = h_{i-1} D_i, or a_i (1 - a_i) (h_{i-1} - x_i) D_i.
// Steps are affine maps of one number, so a run of them is one map (A, B): h -> A h + B, and runs
// compose: that is the scan.
//
// Work split.  A thread takes kT = 16 consecutive tokens of one or two channels (4 bytes of input
// a token), `lanes` threads lie across the channels and the rest of the CTA along the tokens: a
// tile.  Each thread reduces its run to (A, B) from registers, the runs of the CTA meet in shared
// memory, every thread walks the maps of the runs before its own (at most 256 / lanes), and then
// repeats its 16 steps from the true state: x and g are read from memory once and nothing but
// maps is exchanged.  The CTA goes along the sequence tile by tile with the state in registers.
// Where sequences and channels are too few to fill the GPU, a cluster of up to 16 CTAs takes
// consecutive tiles at once and exchanges the tiles' maps through distributed shared memory.
// The order of every composition is fixed, so results are the same bit for bit from call to call.
//
// The sigmoid gate's steps are written h + z (x - h) with z = 1 - a = 1 / (1 + exp(g)) computed as
// such: near a = 1 the rounding of a would be a relative error of z of 2^-24 / z, and that error
// compounds over the 1 / z tokens the state remembers.
#include <cooperative_groups.h>

#include <algorithm>
#include <new>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace lapl {
namespace scan {

constexpr int kT = LAPL_SCAN_CHUNK;   // tokens of a thread's run
constexpr int kThreads = 256;
constexpr int kMaxCluster = 16;
constexpr int kMaxChannels = 64;      // channels of a tile: 32 lanes x 2

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
  int n, c, chunks, reverse;
  Geo geo;
};

// One lane's V channels of a token, as they lie in memory.
template <bool k16, int V>
__device__ __forceinline__ uint32_t load_raw(const void* base, long long e) {
  if constexpr (!k16) return __ldg(reinterpret_cast<const uint32_t*>(base) + e);
  else if constexpr (V == 2) return __ldg(reinterpret_cast<const uint32_t*>(
      reinterpret_cast<const uint16_t*>(base) + e));
  else return (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(base) + e);
}
template <bool k16, int V>
__device__ __forceinline__ void widen(uint32_t w, float (&f)[V]) {
  if constexpr (!k16) f[0] = __uint_as_float(w);
  else if constexpr (V == 2) { f[0] = bf16_lo(w); f[1] = bf16_hi(w); }
  else f[0] = bf16_lo(w);
}
template <bool k16, int V>
__device__ __forceinline__ void store_vec(void* base, long long e, const float (&f)[V]) {
  if constexpr (k16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + e;
    if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = ops::pack_bf16(f[0], f[1]);
    else *p = (uint16_t)ops::pack_bf16(f[0], 0.f);
  } else {
    float* p = reinterpret_cast<float*>(base) + e;
    if constexpr (V == 2) *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    else *p = f[0];
  }
}

// z = 1 - a = 1 / (1 + exp(g)) of the sigmoid gate.  exp(g) = 2^n 2^f with n = round(g log2 e) and
// f = g log2 e - n by one fused step, so that the hardware's exponential sees |f| <= 1/2 and its
// relative error (2 ulp) is not multiplied by |g|; 2^n is an exponent field.  g is held within
// [-87, 88], where neither overflows (z is 1 and 6e-39 there); NaN passes through.
__device__ __forceinline__ float sigmoid_z(float g) {
  constexpr float kLog2e = 1.44269504f;
  constexpr float kRound = 12582912.f;   // 1.5 2^23: adding it leaves the rounded value in the low bits
  asm("min.NaN.f32 %0, %0, 0f42b00000;" : "+f"(g));   // 88
  asm("max.NaN.f32 %0, %0, 0fc2ae0000;" : "+f"(g));   // -87
  const float m = fmaf(g, kLog2e, kRound);
  const float f = fmaf(g, kLog2e, -(m - kRound));
  float e, z;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(f));
  const float scale = __uint_as_float((__float_as_uint(m) << 23) + 0x3f800000u);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(fmaf(e, scale, 1.f)));
  return z;
}

// A step's decay as one register: a (decay gate) or z = 1 - a (sigmoid gate).
template <bool kSig>
__device__ __forceinline__ float gate_of(float g) {
  if constexpr (kSig) return sigmoid_z(g);
  else return g;
}
template <bool kSig>
__device__ __forceinline__ float identity_gate() { return kSig ? 0.f : 1.f; }
// h after a step.
template <bool kSig>
__device__ __forceinline__ float step(float gate, float x, float h) {
  if constexpr (kSig) return fmaf(gate, x - h, h);
  else return fmaf(gate, h, x);
}
// a times v.
template <bool kSig>
__device__ __forceinline__ float decayed(float gate, float v) {
  if constexpr (kSig) return fmaf(-gate, v, v);
  else return gate * v;
}

struct Shared {
  float2 run[2][kThreads * 2];                          // maps of the runs, by round parity
  float2 tile[2][kMaxCluster][kMaxChannels];            // maps of the cluster's tiles
};

// From the run map (A, B) of every thread: the value that enters this thread's run, and `carry`
// moved past the whole round.  kDown: runs and CTAs in descending order.
template <int V, bool kCluster, bool kDown>
__device__ __forceinline__ void exchange(Shared& sm, int parity, int lane, int group, int groups,
                                         int lanes, int rank, int cluster, const float (&A)[V],
                                         const float (&B)[V], float (&carry)[V],
                                         float (&enter)[V]) {
  const int cpb = lanes * V;
#pragma unroll
  for (int v = 0; v < V; ++v)
    sm.run[parity][group * cpb + lane * V + v] = make_float2(A[v], B[v]);
  __syncthreads();
  const float2* runs = &sm.run[parity][(kDown ? (groups - 1) * cpb : 0) + lane * V];
  const int step = kDown ? -cpb : cpb;
  const int mine = kDown ? groups - 1 - group : group;   // runs before this one
  if constexpr (!kCluster) {
#pragma unroll 4
    for (int k = 0; k < groups; ++k, runs += step) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k == mine) enter[v] = carry[v];
        carry[v] = fmaf(runs[v].x, carry[v], runs[v].y);
      }
    }
  } else {
    // One thread a channel composes the CTA's runs and hands the map to every CTA of the cluster.
    if ((int)threadIdx.x < cpb) {
      const float2* p = &sm.run[parity][(kDown ? (groups - 1) * cpb : 0) + threadIdx.x];
      float ta = 1.f, tb = 0.f;
#pragma unroll 4
      for (int k = 0; k < groups; ++k, p += step) {
        tb = fmaf(p->x, tb, p->y);
        ta *= p->x;
      }
      float2* to = &sm.tile[parity][rank][threadIdx.x];
      for (int r = 0; r < cluster; ++r)
        *cg::this_cluster().map_shared_rank(to, r) = make_float2(ta, tb);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    // Meanwhile, the map of the CTA's runs before this thread's.
    float pa[V], pb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      pa[v] = 1.f;
      pb[v] = 0.f;
    }
#pragma unroll 4
    for (int k = 0; k < mine; ++k, runs += step) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        pb[v] = fmaf(runs[v].x, pb[v], runs[v].y);
        pa[v] *= runs[v].x;
      }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll 4
    for (int k = 0; k < cluster; ++k) {
      const int r = kDown ? cluster - 1 - k : k;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (r == rank) enter[v] = fmaf(pa[v], carry[v], pb[v]);
        const float2 m = sm.tile[parity][r][lane * V + v];
        carry[v] = fmaf(m.x, carry[v], m.y);
      }
    }
  }
}

// What a thread is: sequence, channels, place along the tokens.
struct Place {
  long long s;
  int c, lane, group, groups, rank, len;
  bool on;   // has channels
};
template <int V>
__device__ __forceinline__ Place place_of(const Args& a) {
  Place p;
  const int unit = blockIdx.x / a.geo.cluster;
  p.rank = blockIdx.x - unit * a.geo.cluster;
  p.s = unit / a.geo.blocks;
  p.lane = threadIdx.x & (a.geo.lanes - 1);
  p.group = threadIdx.x >> a.geo.lanes_log2;
  p.groups = blockDim.x >> a.geo.lanes_log2;
  p.c = ((unit - (int)p.s * a.geo.blocks) * a.geo.lanes + p.lane) * V;
  p.on = p.c < a.c;
  p.len = a.n;
  if (a.lengths) p.len = max(0, min(a.n, a.lengths[p.s]));
  return p;
}

// Where a thread's run of round t lies: its first place in processing order, and the address step
// from one place to the next.
struct Run {
  int i0;            // clipped to N
  long long row;     // of place i0
};
__device__ __forceinline__ Run run_of(const Args& a, const Place& p, int t, int tile) {
  const long long start = ((long long)t * a.geo.cluster + p.rank) * tile + p.group * kT;
  Run r;
  r.i0 = (int)min(start, (long long)a.n);
  r.row = p.s * a.n + (a.reverse ? p.len - 1 - r.i0 : r.i0);
  return r;
}

// kT tokens of one tensor, zeros where `live` ends.
template <bool k16, int V>
__device__ __forceinline__ void load_run(uint32_t (&w)[kT], const void* base, const Run& r,
                                         long long stride, int c, bool reverse, int live) {
  constexpr int kBytes = k16 ? 2 : 4;
  const char* q = reinterpret_cast<const char*>(base) + (r.row * stride + c) * kBytes;
  const long long step = (reverse ? -stride : stride) * kBytes;
  if (r.i0 + kT <= live) {
#pragma unroll
    for (int u = 0; u < kT; ++u) {
      w[u] = load_raw<k16, V>(q, 0);
      q += step;
    }
  } else {
#pragma unroll
    for (int u = 0; u < kT; ++u) {
      w[u] = 0u;
      if (r.i0 + u < live) w[u] = load_raw<k16, V>(q, 0);
      q += step;
    }
  }
}

template <bool kIn16, bool kOut16, int V, bool kSig, bool kCluster>
__global__ void __launch_bounds__(kThreads, 2)
scan_forward_kernel(const Args a) {
  __shared__ Shared sm;
  const Place p = place_of<V>(a);
  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    carry[v] = a.h0 && p.on ? a.h0[p.s * a.c + p.c + v] : 0.f;
  const int tile = p.groups * kT;
  const int live = p.on ? p.len : 0;
  // No CTA writes into another's shared memory before that one runs.
  if constexpr (kCluster) cg::this_cluster().sync();
  uint32_t rx[kT], rg[kT];
  Run run = run_of(a, p, 0, tile);
  load_run<kIn16, V>(rx, a.x, run, a.x_stride, p.c, a.reverse, live);
  load_run<kIn16, V>(rg, a.g, run, a.g_stride, p.c, a.reverse, live);
  for (int t = 0; t < a.geo.tiles; ++t) {
    float gate[kT][V], x[kT][V];
#pragma unroll
    for (int u = 0; u < kT; ++u) {
      widen<kIn16, V>(rx[u], x[u]);
      widen<kIn16, V>(rg[u], gate[u]);
#pragma unroll
      for (int v = 0; v < V; ++v) gate[u][v] = gate_of<kSig>(gate[u][v]);
    }
    const Run now = run;
    if (now.i0 + kT > live) {
#pragma unroll
      for (int u = 0; u < kT; ++u)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (now.i0 + u >= live) gate[u][v] = identity_gate<kSig>();
    }
    // The next round's tokens are on their way while this one is exchanged and written.
    if (t + 1 < a.geo.tiles) {
      run = run_of(a, p, t + 1, tile);
      load_run<kIn16, V>(rx, a.x, run, a.x_stride, p.c, a.reverse, live);
      load_run<kIn16, V>(rg, a.g, run, a.g_stride, p.c, a.reverse, live);
    }
    float A[V], B[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; B[v] = 0.f; }
#pragma unroll
    for (int u = 0; u < kT; ++u)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] = decayed<kSig>(gate[u][v], A[v]);
        B[v] = step<kSig>(gate[u][v], x[u][v], B[v]);
      }
    exchange<V, kCluster, false>(sm, t & 1, p.lane, p.group, p.groups, a.geo.lanes, p.rank,
                                 a.geo.cluster, A, B, carry, h);
    if (p.on && now.i0 < a.n) {
      if (a.states) {
        float* st = a.states + (p.s * a.chunks + now.i0 / kT) * a.c + p.c;
#pragma unroll
        for (int v = 0; v < V; ++v) st[v] = h[v];
      }
      constexpr int kBytes = kOut16 ? 2 : 4;
      char* q = reinterpret_cast<char*>(a.out) + (now.row * a.c + p.c) * kBytes;
      const long long by = (a.reverse ? -(long long)a.c : (long long)a.c) * kBytes;
      if (now.i0 + kT <= live) {
#pragma unroll
        for (int u = 0; u < kT; ++u) {
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = step<kSig>(gate[u][v], x[u][v], h[v]);
          store_vec<kOut16, V>(q, 0, h);
          q += by;
        }
      } else {
#pragma unroll
        for (int u = 0; u < kT; ++u) {
          const int i = now.i0 + u;
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = step<kSig>(gate[u][v], x[u][v], h[v]);
          if (i < live) {
            store_vec<kOut16, V>(q, 0, h);
          } else if (i < a.n) {
            const float none[V] = {};
            store_vec<kOut16, V>(a.out, (p.s * a.n + i) * a.c + p.c, none);
          }
          q += by;
        }
      }
    }
  }
  if (a.final_state && p.on && p.rank == 0 && p.group == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.final_state[p.s * a.c + p.c + v] = carry[v];
  }
}

template <bool kIn16, bool kGrad16, int V, bool kSig, bool kCluster>
__global__ void __launch_bounds__(kThreads, 2)
scan_backward_kernel(const Args a) {
  __shared__ Shared sm;
  const Place p = place_of<V>(a);
  float carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    carry[v] = a.dfinal && p.on ? a.dfinal[p.s * a.c + p.c + v] : 0.f;
  const int tile = p.groups * kT;
  const int live = p.on ? p.len : 0;
  if constexpr (kCluster) cg::this_cluster().sync();
  for (int t = a.geo.tiles - 1; t >= 0; --t) {
    const Run run = run_of(a, p, t, tile);
    float gate[kT][V], x[kT][V], dh[kT][V], h[V];
    {
      uint32_t rx[kT], rg[kT];
      load_run<kIn16, V>(rg, a.g, run, a.g_stride, p.c, a.reverse, live);
      load_run<kIn16, V>(rx, a.x, run, a.x_stride, p.c, a.reverse, live);
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = p.on && run.i0 < a.n ? a.states[(p.s * a.chunks + run.i0 / kT) * a.c + p.c + v] : 0.f;
      if constexpr (kGrad16 || V == 1) {
        uint32_t rd[kT];
        load_run<kGrad16, V>(rd, a.dout, run, a.c, p.c, a.reverse, live);
#pragma unroll
        for (int u = 0; u < kT; ++u) widen<kGrad16, V>(rd[u], dh[u]);
      } else {
        const float* q = reinterpret_cast<const float*>(a.dout) + run.row * a.c + p.c;
#pragma unroll
        for (int u = 0; u < kT; ++u) {
          float2 d = make_float2(0.f, 0.f);
          if (run.i0 + u < live) d = *reinterpret_cast<const float2*>(q);
          dh[u][0] = d.x;
          dh[u][V - 1] = d.y;
          q += a.reverse ? -a.c : a.c;
        }
      }
#pragma unroll
      for (int u = 0; u < kT; ++u) {
        widen<kIn16, V>(rx[u], x[u]);
        widen<kIn16, V>(rg[u], gate[u]);
#pragma unroll
        for (int v = 0; v < V; ++v) gate[u][v] = gate_of<kSig>(gate[u][v]);
      }
    }
    if (run.i0 + kT > live) {
#pragma unroll
      for (int u = 0; u < kT; ++u)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (run.i0 + u >= live) gate[u][v] = identity_gate<kSig>();
    }
    // The slope of a step in its decay, h_{i-1} - x_i or h_{i-1}, in x's place.
#pragma unroll
    for (int u = 0; u < kT; ++u)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float before = h[v];
        h[v] = step<kSig>(gate[u][v], x[u][v], h[v]);
        x[u][v] = kSig ? before - x[u][v] : before;
      }
    float A[V], B[V], E[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; B[v] = 0.f; }
#pragma unroll
    for (int u = kT - 1; u >= 0; --u)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] = decayed<kSig>(gate[u][v], A[v]);
        B[v] = decayed<kSig>(gate[u][v], dh[u][v] + B[v]);
      }
    exchange<V, kCluster, true>(sm, t & 1, p.lane, p.group, p.groups, a.geo.lanes, p.rank,
                                a.geo.cluster, A, B, carry, E);
    if (p.on && run.i0 < a.n) {
      constexpr int kBytes = kGrad16 ? 2 : 4;
      const int last = run.i0 + kT - 1;
      const long long row = run.row + (a.reverse ? 1 - kT : kT - 1);
      char* qx = reinterpret_cast<char*>(a.dx) + (row * a.x_stride + p.c) * kBytes;
      char* qg = reinterpret_cast<char*>(a.dg) + (row * a.g_stride + p.c) * kBytes;
      const long long bx = (a.reverse ? a.x_stride : -a.x_stride) * kBytes;
      const long long bg = (a.reverse ? a.g_stride : -a.g_stride) * kBytes;
#pragma unroll
      for (int u = kT - 1; u >= 0; --u) {
        float dx[V], dg[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float D = dh[u][v] + E[v];
          E[v] = decayed<kSig>(gate[u][v], D);
          dx[v] = kSig ? gate[u][v] * D : D;
          dg[v] = kSig ? gate[u][v] * x[u][v] * E[v] : x[u][v] * D;
        }
        if (last < live || run.i0 + u < live) {
          store_vec<kGrad16, V>(qx, 0, dx);
          store_vec<kGrad16, V>(qg, 0, dg);
        } else if (run.i0 + u < a.n) {
          const float none[V] = {};
          const long long at = p.s * a.n + run.i0 + u;
          store_vec<kGrad16, V>(a.dx, at * a.x_stride + p.c, none);
          store_vec<kGrad16, V>(a.dg, at * a.g_stride + p.c, none);
        }
        qx += bx;
        qg += bg;
      }
    }
  }
  if (a.dh0 && p.on && p.rank == 0 && p.group == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.dh0[p.s * a.c + p.c + v] = carry[v];
  }
}

// ---- host --------------------------------------------------------------------------------

using Kernel = void (*)(Args);

template <bool kIn16, bool kOther16, bool kSig, bool kBackward>
Kernel pick_v(int v, bool cluster) {
  if constexpr (kIn16)
    if (v == 2) {
      if constexpr (kBackward)
        return cluster ? scan_backward_kernel<true, kOther16, 2, kSig, true>
                       : scan_backward_kernel<true, kOther16, 2, kSig, false>;
      else
        return cluster ? scan_forward_kernel<true, kOther16, 2, kSig, true>
                       : scan_forward_kernel<true, kOther16, 2, kSig, false>;
    }
  if constexpr (kBackward)
    return cluster ? scan_backward_kernel<kIn16, kOther16, 1, kSig, true>
                   : scan_backward_kernel<kIn16, kOther16, 1, kSig, false>;
  else
    return cluster ? scan_forward_kernel<kIn16, kOther16, 1, kSig, true>
                   : scan_forward_kernel<kIn16, kOther16, 1, kSig, false>;
}
template <bool kBackward>
Kernel pick(bool in16, bool other16, bool sig, int v, bool cluster) {
  if (in16)
    return other16 ? (sig ? pick_v<true, true, true, kBackward>(v, cluster)
                          : pick_v<true, true, false, kBackward>(v, cluster))
                   : (sig ? pick_v<true, false, true, kBackward>(v, cluster)
                          : pick_v<true, false, false, kBackward>(v, cluster));
  return other16 ? (sig ? pick_v<false, true, true, kBackward>(v, cluster)
                        : pick_v<false, true, false, kBackward>(v, cluster))
                 : (sig ? pick_v<false, false, true, kBackward>(v, cluster)
                        : pick_v<false, false, false, kBackward>(v, cluster));
}

// Launch geometry with v channels a lane.
Geo geometry(const lapl_scan_config& c, int num_sms, int v) {
  Geo g;
  const int need = (c.channels + v - 1) / v;   // lanes' worth of channels
  const int runs = (c.tokens + kT - 1) / kT;
  // The most lanes of which at most a quarter are idle: full 128-byte rows where there are
  // channels for them.
  g.lanes = 32;
  while (g.lanes > 4 && 3LL * ((need + g.lanes - 1) / g.lanes) * g.lanes > 4LL * need)
    g.lanes >>= 1;
  // Two CTAs for every SM: by splitting the tokens over a cluster, and where that is not enough
  // the channels further, down to 32-byte pieces of a row.
  for (;; g.lanes >>= 1) {
    g.blocks = (need + g.lanes - 1) / g.lanes;
    int groups = kThreads / g.lanes;
    while (groups > 1 && groups / 2 >= runs && groups / 2 * g.lanes >= 32) groups >>= 1;
    g.threads = groups * g.lanes;
    const long long units = (long long)c.sequences * g.blocks;
    g.cluster = 1;
    while (g.cluster < kMaxCluster && units * g.cluster * 5 < 8LL * num_sms &&
           g.cluster * groups < runs)
      g.cluster *= 2;
    const int per_round = g.cluster * groups;
    g.tiles = (runs + per_round - 1) / per_round;
    if (g.lanes <= 8 || g.tiles == 1 || units * g.cluster * 5 >= 8LL * num_sms) break;
  }
  g.lanes_log2 = 0;
  while ((1 << g.lanes_log2) < g.lanes) ++g.lanes_log2;
  return g;
}

lapl_status validate(const lapl_scan_config* c) {
  if (!c) return LAPL_ERR_INVALID_ARG;
  if (c->sequences < 0 || c->tokens < 1 || c->channels < 1) return LAPL_ERR_INVALID_ARG;
  if (c->gate != LAPL_GATE_DECAY && c->gate != LAPL_GATE_SIGMOID) return LAPL_ERR_INVALID_ARG;
  if (c->reverse != 0 && c->reverse != 1) return LAPL_ERR_INVALID_ARG;
  if (!ops::is_float_dtype(c->in_dtype) || !ops::is_float_dtype(c->out_dtype) ||
      !ops::is_float_dtype(c->grad_dtype))
    return LAPL_ERR_INVALID_ARG;
  if ((c->x_stride != 0 && c->x_stride < c->channels) ||
      (c->g_stride != 0 && c->g_stride < c->channels))
    return LAPL_ERR_INVALID_ARG;
  if (c->tokens > (1 << 30) || c->channels > (1 << 24)) return LAPL_ERR_UNSUPPORTED;
  // The grid has up to 16 CTAs for each sequence and each 4 channels.
  if ((long long)c->sequences * ((c->channels + 3) / 4) > (1LL << 26)) return LAPL_ERR_UNSUPPORTED;
  return LAPL_OK;
}

}  // namespace scan
}  // namespace lapl

struct lapl_scan_plan {
  lapl_scan_config cfg;
  int device;
  lapl::scan::Geo geo[2];   // by channels a lane: 1, 2
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

// Channels a lane takes: two bf16 values where rows and pointers let it load them as one word.
int lane_channels(const lapl_scan_plan& p, std::initializer_list<const void*> in,
                  std::initializer_list<const void*> other, int other_dtype, long long xs,
                  long long gs) {
  if (p.cfg.in_dtype != LAPL_BF16 || p.cfg.channels % 2 || xs % 2 || gs % 2) return 1;
  for (const void* q : in)
    if (!ops::aligned(q, 4)) return 1;
  for (const void* q : other)
    if (!ops::aligned(q, 2 * ops::dtype_bytes(other_dtype))) return 1;
  return 2;
}

lapl_status launch(lapl_scan_plan* p, scan::Kernel k, scan::Args& a, int v, void* stream,
                   const char* where) {
  a.geo = p->geo[v - 1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p->cfg.sequences * a.geo.blocks * a.geo.cluster));
  cfg.blockDim = dim3((unsigned)a.geo.threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.geo.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.geo.cluster > 1 ? 1 : 0;
  cudaError_t e = cudaSuccess;
  if (a.geo.cluster > 8)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, k, a);
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, where);
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

scan::Args base_args(const lapl_scan_plan& p) {
  scan::Args a = {};
  const lapl_scan_config& c = p.cfg;
  a.n = c.tokens;
  a.c = c.channels;
  a.chunks = (c.tokens + scan::kT - 1) / scan::kT;
  a.reverse = c.reverse;
  a.x_stride = c.x_stride ? c.x_stride : c.channels;
  a.g_stride = c.g_stride ? c.g_stride : c.channels;
  return a;
}

}  // namespace

extern "C" {

lapl_status lapl_scan_create(const lapl_scan_config* cfg, lapl_scan_handle* out) {
  if (!out) return LAPL_ERR_INVALID_ARG;
  *out = nullptr;
  const lapl_status st = scan::validate(cfg);
  if (st != LAPL_OK) return st;
  lapl_scan_plan* p = new (std::nothrow) lapl_scan_plan();
  if (!p) return LAPL_ERR_INVALID_ARG;
  p->cfg = *cfg;
  int sms = 0;
  cudaError_t e = cudaGetDevice(&p->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, p->device);
  if (e != cudaSuccess) {
    delete p;
    return LAPL_ERR_CUDA;
  }
  for (int v = 1; v <= 2; ++v) p->geo[v - 1] = scan::geometry(*cfg, sms, v);
  *out = p;
  return LAPL_OK;
}

lapl_status lapl_scan_forward(lapl_scan_handle p, const void* x, const void* g, const float* h0,
                              const int* lengths, void* out, float* states, float* final_state,
                              void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  if (p->cfg.sequences == 0) return LAPL_OK;
  if (!x || !g || !out) return LAPL_ERR_INVALID_ARG;
  const lapl_scan_config& c = p->cfg;
  if (!ops::aligned(x, ops::dtype_bytes(c.in_dtype)) ||
      !ops::aligned(g, ops::dtype_bytes(c.in_dtype)) ||
      !ops::aligned(out, ops::dtype_bytes(c.out_dtype)) || !ops::aligned(h0, 4) ||
      !ops::aligned(lengths, 4) || !ops::aligned(states, 4) || !ops::aligned(final_state, 4))
    return LAPL_ERR_ALIGNMENT;
  const lapl_status st = ops::check_device(p->device, p->last_error, "scan_forward/device");
  if (st != LAPL_OK) return st;
  scan::Args a = base_args(*p);
  a.x = x;
  a.g = g;
  a.h0 = h0;
  a.lengths = lengths;
  a.out = out;
  a.states = states;
  a.final_state = final_state;
  const int v = lane_channels(*p, {x, g}, {out}, c.out_dtype, a.x_stride, a.g_stride);
  const scan::Kernel k = scan::pick<false>(c.in_dtype == LAPL_BF16, c.out_dtype == LAPL_BF16,
                                           c.gate == LAPL_GATE_SIGMOID, v,
                                           p->geo[v - 1].cluster > 1);
  return launch(p, k, a, v, stream, "scan_forward");
}

lapl_status lapl_scan_backward(lapl_scan_handle p, const void* x, const void* g,
                               const float* states, const int* lengths, const void* dout,
                               const float* dfinal, void* dx, void* dg, float* dh0,
                               void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  if (p->cfg.sequences == 0) return LAPL_OK;
  if (!x || !g || !states || !dout || !dx || !dg) return LAPL_ERR_INVALID_ARG;
  const lapl_scan_config& c = p->cfg;
  const int ib = ops::dtype_bytes(c.in_dtype), gb = ops::dtype_bytes(c.grad_dtype);
  if (!ops::aligned(x, ib) || !ops::aligned(g, ib) || !ops::aligned(dout, gb) ||
      !ops::aligned(dx, gb) || !ops::aligned(dg, gb) || !ops::aligned(states, 4) ||
      !ops::aligned(lengths, 4) || !ops::aligned(dfinal, 4) || !ops::aligned(dh0, 4))
    return LAPL_ERR_ALIGNMENT;
  const lapl_status st = ops::check_device(p->device, p->last_error, "scan_backward/device");
  if (st != LAPL_OK) return st;
  scan::Args a = base_args(*p);
  a.x = x;
  a.g = g;
  a.states = const_cast<float*>(states);
  a.lengths = lengths;
  a.dout = dout;
  a.dfinal = dfinal;
  a.dx = dx;
  a.dg = dg;
  a.dh0 = dh0;
  const int v =
      lane_channels(*p, {x, g}, {dout, dx, dg}, c.grad_dtype, a.x_stride, a.g_stride);
  const scan::Kernel k = scan::pick<true>(c.in_dtype == LAPL_BF16, c.grad_dtype == LAPL_BF16,
                                          c.gate == LAPL_GATE_SIGMOID, v,
                                          p->geo[v - 1].cluster > 1);
  return launch(p, k, a, v, stream, "scan_backward");
}

lapl_status lapl_scan_plan_info_get(lapl_scan_handle p, lapl_scan_plan_info* info) {
  if (!p || !info) return LAPL_ERR_INVALID_ARG;
  const int v = p->cfg.in_dtype == LAPL_BF16 && p->cfg.channels % 2 == 0 ? 2 : 1;
  info->cluster = p->geo[v - 1].cluster;
  info->lanes = p->geo[v - 1].lanes;
  info->threads = p->geo[v - 1].threads;
  return LAPL_OK;
}

const char* lapl_scan_last_error(lapl_scan_handle p) { return p ? p->last_error : ""; }

lapl_status lapl_scan_destroy(lapl_scan_handle p) {
  delete p;
  return LAPL_OK;
}

}  // extern "C"
