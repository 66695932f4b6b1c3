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
// What bounds it is the exchange: a round of tiles costs a load, a barrier and a walk one after the
// other, whatever the bytes.  These kernels take sequences longer than scan_few.cu's few tokens and
// shorter than scan_pipe.cuh's are made for (512 x 256 x 64 bf16, sigmoid and decay gate: 14.7 and 11.7 us
// forward, 23.3 and 18.8 backward, of which 7.4 and 12.7 are bytes), odd bf16 channel counts, and rows
// of odd lengths where they are many (16 x 4096 x 333 fp32: 69 and 62 us of 39).
//
// The sigmoid gate's a and z = 1 - a are computed each for itself: neither is accurate as 1 less the
// other where it is small.  Near a = 1 the rounding of a is a relative error of z of 2^-24 / z, and that
// error compounds over the 1 / z tokens the state remembers; what crosses from run to run goes by
// 1 - A, summed as such (scan.cuh).  Of the two a thread's registers have room for one: between its two
// walks z x, or in the backward z, waits in shared memory.
#include <cooperative_groups.h>

#include <algorithm>
#include <new>

#include "scan_few.cuh"
#include "scan_pipe.cuh"

namespace cg = cooperative_groups;

namespace lapl {
namespace scan {

constexpr int kThreads = 256;
constexpr int kMaxCluster = 16;
constexpr int kMaxChannels = 64;      // channels of a tile: 32 lanes x 2

// In dynamic shared memory: maps of the runs, by round parity ([2][kThreads V]); of the cluster's tiles
// ([2][kMaxCluster][kMaxChannels]); and with the sigmoid gate what a thread keeps of each token from
// its first walk to the second ([kT][threads] of V values).
template <int V, bool kCluster>
struct Shared {
  unsigned char* base;
  __device__ __forceinline__ float2* run(int parity) const {
    return reinterpret_cast<float2*>(base) + parity * kThreads * V;
  }
  __device__ __forceinline__ float2* tile(int parity, int rank) const {
    return run(2) + (parity * kMaxCluster + rank) * kMaxChannels;
  }
  __device__ __forceinline__ Vec<V>* kept() const {
    return reinterpret_cast<Vec<V>*>(run(2) + (kCluster ? 2 * kMaxCluster * kMaxChannels : 0)) +
           threadIdx.x;
  }
};
constexpr unsigned shared_bytes(int threads, int v, bool cluster, bool sig) {
  return 8u * (2 * kThreads * v + (cluster ? 2 * kMaxCluster * kMaxChannels : 0)) +
         (sig ? 4u * v * kT * threads : 0u);
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

// From the run map (A, B) of every thread: the value that enters this thread's run, and `carry`
// moved past the whole round.  kDown: runs and CTAs in descending order.
template <int V, bool kCluster, bool kDown>
__device__ __forceinline__ void exchange(const Shared<V, kCluster>& sm, int parity, const Place& p, int lanes,
                                         int cluster, const Vec<V>& A, const Vec<V>& B,
                                         Vec<V>& carry, Vec<V>& enter) {
  const int cpb = lanes * V, groups = p.groups;
#pragma unroll
  for (int v = 0; v < V; ++v)
    sm.run(parity)[p.group * cpb + p.lane * V + v] = make_float2(A.f[v], B.f[v]);
  __syncthreads();
  const float2* runs = sm.run(parity) + (kDown ? (groups - 1) * cpb : 0) + p.lane * V;
  const int by = kDown ? -cpb : cpb;
  const int mine = kDown ? groups - 1 - p.group : p.group;   // runs before this one
  if constexpr (!kCluster) {
#pragma unroll 4
    for (int k = 0; k < groups; ++k, runs += by) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k == mine) enter.f[v] = carry.f[v];
        carry.f[v] = fmaf(runs[v].x, carry.f[v], runs[v].y);
      }
    }
  } else {
    // One thread a channel composes the CTA's runs and hands the map to every CTA of the cluster.
    if ((int)threadIdx.x < cpb) {
      const float2* q = sm.run(parity) + (kDown ? (groups - 1) * cpb : 0) + threadIdx.x;
      float ta = 1.f, tb = 0.f;
#pragma unroll 4
      for (int k = 0; k < groups; ++k, q += by) {
        tb = fmaf(q->x, tb, q->y);
        ta *= q->x;
      }
      float2* to = sm.tile(parity, p.rank) + threadIdx.x;
      for (int r = 0; r < cluster; ++r)
        *cg::this_cluster().map_shared_rank(to, r) = make_float2(ta, tb);
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    // Meanwhile, the map of the CTA's runs before this thread's.
    Vec<V> pa = fill<V>(1.f), pb = fill<V>(0.f);
#pragma unroll 4
    for (int k = 0; k < mine; ++k, runs += by) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        pb.f[v] = fmaf(runs[v].x, pb.f[v], runs[v].y);
        pa.f[v] *= runs[v].x;
      }
    }
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
#pragma unroll 4
    for (int k = 0; k < cluster; ++k) {
      const int r = kDown ? cluster - 1 - k : k;
      if (r == p.rank) enter = fma(pa, carry, pb);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 m = sm.tile(parity, r)[p.lane * V + v];
        carry.f[v] = fmaf(m.x, carry.f[v], m.y);
      }
    }
  }
}

// Where a thread's run of round t lies: its first place in processing order, and that place's row.
struct Run {
  int i0;            // clipped to N
  long long row;
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
__device__ __forceinline__ void load_run(Raw<k16, V> (&w)[kT], const void* base, const Run& r,
                                         long long stride, int c, bool reverse, int live) {
  constexpr int kBytes = k16 ? 2 : 4;
  const char* q = reinterpret_cast<const char*>(base) + (r.row * stride + c) * kBytes;
  const long long by = (reverse ? -stride : stride) * kBytes;
  if (r.i0 + kT <= live) {
#pragma unroll
    for (int u = 0; u < kT; ++u, q += by) w[u] = load_raw<k16, V>(q);
  } else {
#pragma unroll
    for (int u = 0; u < kT; ++u, q += by)
      w[u] = r.i0 + u < live ? load_raw<k16, V>(q) : zero_raw<k16, V>();
  }
}

template <bool kIn16, bool kOut16, int V, bool kSig, bool kCluster>
__global__ void __launch_bounds__(kThreads, 3)
scan_forward_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  const Shared<V, kCluster> sm = {dynamic};
  Vec<V>* const kept = sm.kept();
  const Place p = place_of<V>(a);
  Vec<V> carry = fill<V>(0.f);
  if (a.h0 && p.on) carry = widen(load_raw<false, V>(a.h0 + p.s * a.c + p.c));
  const int tile = p.groups * kT;
  const int live = p.on ? p.len : 0;
  // No CTA writes into another's shared memory before that one runs.
  if constexpr (kCluster) cg::this_cluster().sync();
  for (int t = 0; t < a.geo.tiles; ++t) {
    const Run now = run_of(a, p, t, tile);
    Raw<kIn16, V> rx[kT];
    Vec<V> decay[kT], B = fill<V>(0.f), h;
    Factor<kSig, V> A;
    {
      Raw<kIn16, V> rg[kT];
      load_run(rg, a.g, now, a.g_stride, p.c, a.reverse, live);
      load_run(rx, a.x, now, a.x_stride, p.c, a.reverse, live);
      if constexpr (kSig) {
        gates<4, kIn16, V>(rg, now.i0, live, [&](int u, const Gate<V>& g) {
          const Vec<V> b = mul(g.z, widen(rx[u]));
          A.take(g);
          B = fma(g.a, B, b);
          kept[u * blockDim.x] = b;
          decay[u] = g.a;
        });
      } else {
#pragma unroll
        for (int u = 0; u < kT; ++u) decay[u] = widen(rg[u]);
        if (now.i0 + kT > live) {
#pragma unroll
          for (int u = 0; u < kT; ++u)
            if (now.i0 + u >= live) decay[u] = fill<V>(1.f);
        }
#pragma unroll
        for (int u = 0; u < kT; ++u) {
          A.take({decay[u], {}});
          B = fma(decay[u], B, widen(rx[u]));
        }
      }
    }
    auto next = [&](int u, const Vec<V>& h) {
      if constexpr (kSig) return fma(decay[u], h, kept[u * blockDim.x]);
      else return fma(decay[u], h, widen(rx[u]));
    };
    exchange<V, kCluster, false>(sm, t & 1, p, a.geo.lanes, a.geo.cluster, A.value(), B, carry, h);
    if (p.on && now.i0 < a.n) {
      if (a.states)
        store_vec<false>(a.states + (p.s * a.chunks + now.i0 / kT) * a.c + p.c, h);
      constexpr int kBytes = kOut16 ? 2 : 4;
      char* q = reinterpret_cast<char*>(a.out) + (now.row * a.c + p.c) * kBytes;
      const long long by = (a.reverse ? -(long long)a.c : (long long)a.c) * kBytes;
      if (now.i0 + kT <= live) {
#pragma unroll
        for (int u = 0; u < kT; ++u, q += by) {
          h = next(u, h);
          store_vec<kOut16>(q, h);
        }
      } else {
#pragma unroll
        for (int u = 0; u < kT; ++u, q += by) {
          const int i = now.i0 + u;
          h = next(u, h);
          if (i < live)
            store_vec<kOut16>(q, h);
          else if (i < a.n)
            store_vec<kOut16>(reinterpret_cast<char*>(a.out) + ((p.s * a.n + i) * a.c + p.c) * kBytes,
                              fill<V>(0.f));
        }
      }
    }
  }
  if (a.final_state && p.on && p.rank == 0 && p.group == 0)
    store_vec<false>(a.final_state + p.s * a.c + p.c, carry);
}

template <bool kIn16, bool kGrad16, int V, bool kSig, bool kCluster>
__global__ void __launch_bounds__(kThreads, 2)
scan_backward_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  const Shared<V, kCluster> sm = {dynamic};
  Vec<V>* const kept = sm.kept();
  const Place p = place_of<V>(a);
  Vec<V> carry = fill<V>(0.f);
  if (a.dfinal && p.on) carry = widen(load_raw<false, V>(a.dfinal + p.s * a.c + p.c));
  const int tile = p.groups * kT;
  const int live = p.on ? p.len : 0;
  if constexpr (kCluster) cg::this_cluster().sync();
  for (int t = a.geo.tiles - 1; t >= 0; --t) {
    const Run run = run_of(a, p, t, tile);
    Vec<V> decay[kT], slope[kT], dh[kT], h = fill<V>(0.f);
    Factor<kSig, V> A;
    {
      Raw<kIn16, V> rx[kT], rg[kT];
      Raw<kGrad16, V> rd[kT];
      load_run(rg, a.g, run, a.g_stride, p.c, a.reverse, live);
      load_run(rx, a.x, run, a.x_stride, p.c, a.reverse, live);
      load_run(rd, a.dout, run, a.c, p.c, a.reverse, live);
      if (p.on && run.i0 < a.n)
        h = widen(load_raw<false, V>(a.states + (p.s * a.chunks + run.i0 / kT) * a.c + p.c));
      if constexpr (kSig) {
        gates<4, kIn16, V>(rg, run.i0, live, [&](int u, const Gate<V>& g) {
          const Vec<V> x = widen(rx[u]);
          A.take(g);
          slope[u] = mul(g.z, sub(h, x));
          h = fma(g.a, h, mul(g.z, x));
          kept[u * blockDim.x] = g.z;
          decay[u] = g.a;
        });
      } else {
#pragma unroll
        for (int u = 0; u < kT; ++u) decay[u] = widen(rg[u]);
        if (run.i0 + kT > live) {
#pragma unroll
          for (int u = 0; u < kT; ++u)
            if (run.i0 + u >= live) decay[u] = fill<V>(1.f);
        }
#pragma unroll
        for (int u = 0; u < kT; ++u) {
          slope[u] = h;
          h = fma(decay[u], h, widen(rx[u]));
        }
      }
#pragma unroll
      for (int u = 0; u < kT; ++u) dh[u] = widen(rd[u]);
    }
    Vec<V> B = fill<V>(0.f), E;
#pragma unroll
    for (int u = kT - 1; u >= 0; --u) {
      if constexpr (!kSig) A.take({decay[u], {}});
      B = mul(decay[u], add(dh[u], B));
    }
    exchange<V, kCluster, true>(sm, t & 1, p, a.geo.lanes, a.geo.cluster, A.value(), B, carry, E);
    if (p.on && run.i0 < a.n) {
      constexpr int kBytes = kGrad16 ? 2 : 4;
      const bool whole = run.i0 + kT <= live;
      const long long row = run.row + (a.reverse ? 1 - kT : kT - 1);
      char* qx = reinterpret_cast<char*>(a.dx) + (row * a.x_stride + p.c) * kBytes;
      char* qg = reinterpret_cast<char*>(a.dg) + (row * a.g_stride + p.c) * kBytes;
      const long long bx = (a.reverse ? a.x_stride : -a.x_stride) * kBytes;
      const long long bg = (a.reverse ? a.g_stride : -a.g_stride) * kBytes;
#pragma unroll
      for (int u = kT - 1; u >= 0; --u, qx += bx, qg += bg) {
        const Vec<V> D = add(dh[u], E);
        E = mul(decay[u], D);
        Vec<V> z = {}, dx, dg;
        if constexpr (kSig) z = kept[u * blockDim.x];
        step_gradients<kSig>(z, slope[u], D, E, dx, dg);
        const int i = run.i0 + u;
        if (whole || i < live) {
          store_vec<kGrad16>(qx, dx);
          store_vec<kGrad16>(qg, dg);
        } else if (i < a.n) {
          const long long at = p.s * a.n + i;
          store_vec<kGrad16>(reinterpret_cast<char*>(a.dx) + (at * a.x_stride + p.c) * kBytes, fill<V>(0.f));
          store_vec<kGrad16>(reinterpret_cast<char*>(a.dg) + (at * a.g_stride + p.c) * kBytes, fill<V>(0.f));
        }
      }
    }
  }
  if (a.dh0 && p.on && p.rank == 0 && p.group == 0)
    store_vec<false>(a.dh0 + p.s * a.c + p.c, carry);
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

// A kernel of scan_pipe.cuh with its launch shape; kernel null where it is not taken.
struct Pipe {
  pipe::Pick pick;
  Geo geo;
};

// Clusters of 1 .. kMaxCluster pipelined CTAs that the device holds at once: by cluster size, the
// same for all these kernels (each takes an SM to itself).
struct Held {
  int clusters[pipe::kMaxCluster + 1];
};
cudaError_t clusters_held(const pipe::Pick& k, Held* out) {
  for (int n = 1; n <= pipe::kMaxCluster; ++n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n);
    cfg.blockDim = dim3((unsigned)(k.teams * k.warps + 2) * 32);
    cfg.dynamicSmemBytes = k.layout.total(n);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)n;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&out->clusters[n], k.kernel, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

pipe::Pick pick_pipe(const lapl_scan_config& c, bool backward, int lanes) {
  const bool in16 = c.in_dtype == LAPL_BF16, sig = c.gate == LAPL_GATE_SIGMOID;
  const bool other16 = (backward ? c.grad_dtype : c.out_dtype) == LAPL_BF16;
  if (backward)
    return in16 ? pipe::backward_bf16(other16, sig, lanes) : pipe::backward_f32(other16, sig, lanes);
  return in16 ? pipe::forward_bf16(other16, sig, lanes) : pipe::forward_f32(other16, sig, lanes);
}

// The shape with the least work on the longest path: waves of clusters, as many as the GPU holds at
// once, times rounds, and three rounds' time to start and end each wave.  Of nearly equal ones
// (within 5%) the one with the longest pieces of a row.
cudaError_t choose_pipe(const lapl_scan_config& c, bool backward, const Held& held,
                        unsigned smem_most, Pipe* out) {
  const int v = c.in_dtype == LAPL_BF16 ? 2 : 1;
  out->pick.kernel = nullptr;
  double best = 0;
  for (int lanes = 32; lanes >= 8; lanes /= 2) {
    const pipe::Pick k = pick_pipe(c, backward, lanes);
    Geo g = {};
    g.lanes = lanes;
    g.blocks = (c.channels + lanes * v - 1) / (lanes * v);
    g.threads = (k.teams * k.warps + 2) * 32;
    const long long units = (long long)c.sequences * g.blocks;
    const int tile = k.warps * (32 / lanes) * kT;
    for (g.cluster = 1; g.cluster <= pipe::kMaxCluster; ++g.cluster) {
      const int at_once = held.clusters[g.cluster];
      if (at_once < 1 || k.layout.total(g.cluster) > smem_most) continue;
      const long long round = (long long)g.cluster * tile;
      g.tiles = (int)((c.tokens + round - 1) / round);
      const double cost = (double)((units + at_once - 1) / at_once) * (g.tiles + 3);
      if (!out->pick.kernel || cost < 0.95 * best) {
        best = cost;
        out->pick = k;
        out->geo = g;
      }
    }
  }
  if (!out->pick.kernel) return cudaSuccess;
  // The most there is, whatever this plan's clusters take: it is the kernel's, and other plans' too.
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(out->pick.kernel),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_most);
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
  unsigned* dev_err;
  lapl::scan::Geo geo[2];   // by channels a lane: 1, 2
  lapl::scan::Pipe fwd, bwd;
  bool few;                 // forward by scan_few.cu
  unsigned long long wait_ns;
  int skip_last;
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

constexpr unsigned long long kWaitNs = 1000000000ull;   // one second

// Tokens from which the pipelined kernels are taken; shorter sequences leave their teams without work.
// In percent of the other kernel's time, 40 to 700 sequences of 32 to 128 channels, both gates, mean and
// range: forward at 800 tokens bf16 97 (90 to 108), fp32 108 (95 to 123), which breaks even later, at
// 1600 95 (84 to 101); at 512 117 and 129.  Backward at 800 bf16 82 (61 to 99), fp32 91 (71 to 106), at 512
// 98 (83 to 120) and 110 (88 to 128), at 256 bf16 118.
constexpr int kPipeTokens = 768, kPipeTokensBackward16 = 512;

bool whole(std::initializer_list<const void*> pointers, int bytes) {
  for (const void* q : pointers)
    if (!ops::aligned(q, bytes)) return false;
  return true;
}
// Whether a tensor's rows, `stride` elements apart, all start at multiples of 16 bytes.
bool coarse(const void* base, long long stride, int bytes) {
  return ops::aligned(base, 16) && stride * bytes % 16 == 0;
}

// Channels a lane takes: two bf16 values where rows and pointers let it load them as one word, and
// two of the other tensors' values (other_bytes each) and of the fp32 states at once.
int lane_channels(const lapl_scan_plan& p, std::initializer_list<const void*> in,
                  std::initializer_list<const void*> other, int other_bytes,
                  std::initializer_list<const void*> states, const scan::Args& a) {
  const bool pairs = p.cfg.in_dtype == LAPL_BF16 && p.cfg.channels % 2 == 0 &&
                     a.x_stride % 2 == 0 && a.g_stride % 2 == 0;
  return pairs && whole(in, 4) && whole(other, 2 * other_bytes) && whole(states, 8) ? 2 : 1;
}

lapl_status launch(lapl_scan_plan* p, scan::Kernel k, scan::Args& a, int v, void* stream,
                   const char* where) {
  a.geo = p->geo[v - 1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p->cfg.sequences * a.geo.blocks * a.geo.cluster));
  cfg.blockDim = dim3((unsigned)a.geo.threads);
  const bool sig = p->cfg.gate == LAPL_GATE_SIGMOID;
  cfg.dynamicSmemBytes = scan::shared_bytes(a.geo.threads, v, a.geo.cluster > 1, sig);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.geo.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.geo.cluster > 1 ? 1 : 0;
  cudaError_t e = cudaSuccess;
  if (cfg.dynamicSmemBytes > 48 * 1024)   // the most there is, whatever this plan's takes: it is the kernel's
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)scan::shared_bytes(scan::kThreads, 2, true, true));
  if (e == cudaSuccess && a.geo.cluster > 8)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, k, a);
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, where);
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

lapl_status launch_pipe(lapl_scan_plan* p, const scan::Pipe& k, scan::Args& a, void* stream,
                        const char* where) {
  a.geo = k.geo;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p->cfg.sequences * a.geo.blocks * a.geo.cluster));
  cfg.blockDim = dim3((unsigned)a.geo.threads);
  cfg.dynamicSmemBytes = k.pick.layout.total(a.geo.cluster);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.geo.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k.pick.kernel, a, p->dev_err);
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, where);
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

scan::Geo few_geometry(const lapl_scan_config& c, int v) {
  const int need = (c.channels + v - 1) / v;
  scan::Geo g = {};
  g.lanes = 1;
  while (g.lanes < need && g.lanes < scan::few::kThreads) {
    g.lanes *= 2;
    ++g.lanes_log2;
  }
  g.blocks = (need + g.lanes - 1) / g.lanes;
  g.threads = scan::few::kThreads;
  g.cluster = g.tiles = 1;
  return g;
}

// Few tokens: v channels a thread where every tensor's rows start at multiples of them, else one.
// in, other, states: the tensors in in_dtype, in other_dtype, and of states.
lapl_status launch_few(lapl_scan_plan* p, bool backward, scan::Args& a, int v,
                       std::initializer_list<const void*> in,
                       std::initializer_list<const void*> other, int other_dtype,
                       std::initializer_list<const void*> states, void* stream, const char* where) {
  const lapl_scan_config& c = p->cfg;
  if (c.channels % v || a.x_stride % v || a.g_stride % v ||
      !whole(in, v * ops::dtype_bytes(c.in_dtype)) ||
      !whole(other, v * ops::dtype_bytes(other_dtype)) || !whole(states, v * 4))
    v = 1;
  const scan::Geo& g = a.geo = few_geometry(c, v);
  const int per = scan::few::kThreads >> g.lanes_log2;
  const long long ctas = (long long)((c.sequences - 1) / per + 1) * g.blocks;
  const bool in16 = c.in_dtype == LAPL_BF16, other16 = other_dtype == LAPL_BF16;
  const bool sig = c.gate == LAPL_GATE_SIGMOID;
  const scan::few::Kernel k = backward ? scan::few::backward(in16, other16, sig, v, c.tokens)
                                       : scan::few::forward(in16, other16, sig, v, c.tokens);
  k<<<(unsigned)ctas, scan::few::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, where);
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

scan::Args base_args(const lapl_scan_plan& p) {
  scan::Args a = {};
  const lapl_scan_config& c = p.cfg;
  a.sequences = c.sequences;
  a.n = c.tokens;
  a.c = c.channels;
  a.chunks = (c.tokens + scan::kT - 1) / scan::kT;
  a.reverse = c.reverse;
  a.wait_ns = p.wait_ns;
  a.skip_last = p.skip_last;
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
  p->wait_ns = kWaitNs;
  int sms = 0;
  cudaError_t e = cudaGetDevice(&p->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, p->device);
  if (e != cudaSuccess) {
    cudaGetLastError();
    delete p;
    return LAPL_ERR_CUDA;
  }
  for (int v = 1; v <= 2; ++v) p->geo[v - 1] = scan::geometry(*cfg, sms, v);
  // Tokens one after the other in a thread: where there are few, and with threads for the GPU some more
  // (sigmoid gate, bf16 and fp32, 8 tokens of 64 x 4096 channels: 50 and 54% of the other kernel's time, of
  // 1 x 4096, 100 and 115; 32 tokens of 64 x 4096: 101 and 84, of 256 x 512: 107 and 98).
  p->few = cfg->tokens <= 8 ||
           (cfg->tokens <= 32 && (long long)cfg->sequences * cfg->channels >= 1600LL * sms);
  // Long sequences: the pipelined kernels, for bf16 inputs in pairs of channels.
  e = device_error_word(&p->dev_err);
  const bool pairs = cfg->in_dtype == LAPL_F32 ||
                     (cfg->channels % 2 == 0 && cfg->x_stride % 2 == 0 && cfg->g_stride % 2 == 0);
  const bool forward = cfg->tokens >= kPipeTokens;
  const bool backward =
      cfg->tokens >= (cfg->in_dtype == LAPL_BF16 ? kPipeTokensBackward16 : kPipeTokens);
  if (e == cudaSuccess && pairs && backward && cfg->sequences > 0) {
    scan::Held held = {};
    const scan::pipe::Pick one = scan::pick_pipe(*cfg, false, 32);
    int most = 0;
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, p->device);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(one.kernel),
                               cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = scan::clusters_held(one, &held);
    if (e == cudaSuccess && forward)
      e = scan::choose_pipe(*cfg, false, held, (unsigned)most, &p->fwd);
    if (e == cudaSuccess) e = scan::choose_pipe(*cfg, true, held, (unsigned)most, &p->bwd);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    delete p;
    return LAPL_ERR_CUDA;
  }
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
  const int ib = ops::dtype_bytes(c.in_dtype), ob = ops::dtype_bytes(c.out_dtype);
  if (p->few)
    return launch_few(p, false, a, 4, {x, g}, {out}, c.out_dtype, {h0, states, final_state}, stream,
                      "scan_forward");
  if (p->fwd.pick.kernel) {
    const int pair = c.in_dtype == LAPL_BF16 ? 2 : 1;
    a.fine = !coarse(x, a.x_stride, ib) || !coarse(g, a.g_stride, ib);
    // Without 16-byte pieces, and with sequences and channels for nearly the whole GPU, the other
    // kernel is the faster one (sigmoid gate, 16 x 4096 x 333 fp32, clusters of 2: 68 against 87 us;
    // 5 x 8484 x 23, of 16: 12 against 8; 2 x 9001 x 257: 25 against 19).
    const bool other = a.fine && p->geo[pair - 1].cluster <= 2;
    if (!other && whole({x, g}, 4) && whole({out}, pair * ob) &&
        whole({h0, states, final_state}, pair * 4))
      return launch_pipe(p, p->fwd, a, stream, "scan_forward");
  }
  const int v = lane_channels(*p, {x, g}, {out}, ob, {h0, states, final_state}, a);
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
  if (c.tokens <= scan::few::kBackwardTokens)
    return launch_few(p, true, a, c.tokens <= scan::few::kTokens ? 4 : 2, {x, g}, {dout, dx, dg},
                      c.grad_dtype, {states, dfinal, dh0}, stream, "scan_backward");
  if (p->bwd.pick.kernel) {
    const int pair = c.in_dtype == LAPL_BF16 ? 2 : 1;
    a.fine = !coarse(x, a.x_stride, ib) || !coarse(g, a.g_stride, ib);
    a.fine_dout = !coarse(dout, a.c, gb);
    // As forward, for the whole GPU (sigmoid gate, 24 x 4096 x 333 fp32: 151 against 166 us; 64 x 1024 x
    // 99: 35 against 47; 16 x 4096 x 333, clusters of 2: 142 against 127).
    const bool other = a.fine && p->geo[pair - 1].cluster == 1;
    if (!other && whole({x, g}, 4) && whole({dout, dx, dg}, pair * gb) &&
        whole({states, dfinal, dh0}, pair * 4) && !(a.fine_dout && pair * gb < 4))
      return launch_pipe(p, p->bwd, a, stream, "scan_backward");
  }
  const int v = lane_channels(*p, {x, g}, {dout, dx, dg}, gb, {states, dfinal, dh0}, a);
  const scan::Kernel k = scan::pick<true>(c.in_dtype == LAPL_BF16, c.grad_dtype == LAPL_BF16,
                                          c.gate == LAPL_GATE_SIGMOID, v,
                                          p->geo[v - 1].cluster > 1);
  return launch(p, k, a, v, stream, "scan_backward");
}

lapl_status lapl_scan_plan_info_get(lapl_scan_handle p, lapl_scan_plan_info* info) {
  if (!p || !info) return LAPL_ERR_INVALID_ARG;
  const int v = p->cfg.in_dtype == LAPL_BF16 && p->cfg.channels % 2 == 0 ? 2 : 1;
  const bool pipe = p->fwd.pick.kernel != nullptr;
  const scan::Geo g = p->few ? few_geometry(p->cfg, p->cfg.channels % 4 == 0 ? 4 : 1)
                      : pipe ? p->fwd.geo : p->geo[v - 1];
  info->cluster = g.cluster;
  info->lanes = g.lanes;
  info->threads = g.threads;
  info->teams = pipe ? p->fwd.pick.teams : 0;
  return LAPL_OK;
}

lapl_status lapl_scan_device_errors(lapl_scan_handle p, void* stream, unsigned* flags) {
  if (!p || !flags) return LAPL_ERR_INVALID_ARG;
  const lapl_status ok = ops::check_device(p->device, p->last_error, "device_errors/device");
  if (ok != LAPL_OK) return ok;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, p->dev_err, sizeof(word), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(p->dev_err, 0, sizeof(word), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "device_errors");
    return LAPL_ERR_CUDA;
  }
  *flags = word;
  if (!word) return LAPL_OK;
  snprintf(p->last_error, sizeof(p->last_error),
           "device error flags 0x%x: a bounded wait gave up in:%s%s", word,
           (word & kErrBitScan) ? " the recurrence's exchange between CTAs;" : "",
           (word & ~kErrBitScan) ? " a kernel of the attention;" : "");
  return LAPL_ERR_DEVICE_TIMEOUT;
}

lapl_status lapl_scan_set_fault_injection(lapl_scan_handle p, unsigned long long wait_ns,
                                          int skip_last) {
  if (!p || skip_last < 0) return LAPL_ERR_INVALID_ARG;
  p->wait_ns = wait_ns ? wait_ns : kWaitNs;
  p->skip_last = skip_last;
  return LAPL_OK;
}

const char* lapl_scan_last_error(lapl_scan_handle p) { return p ? p->last_error : ""; }

lapl_status lapl_scan_destroy(lapl_scan_handle p) {
  delete p;
  return LAPL_OK;
}

}  // extern "C"
