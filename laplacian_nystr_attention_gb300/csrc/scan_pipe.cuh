// scan_pipe.cuh -- the gated linear recurrence over long sequences: the kernels of scan.cu's
// formulas with the tokens copied ahead, and the exchange of maps taken out of the threads' way.
//
// As in scan.cu a thread reduces a run of 16 tokens to an affine map and repeats it from the true
// state once it knows that; what comes between is a chain over the whole sequence, and waiting for
// it is what bounds scan.cu's kernels on long sequences with few channels.  Here:
//   * A CTA has teams of four worker warps that take the rounds of tiles in turn: while one waits
//     for its states, the others reduce their runs.
//   * Two more warps do nothing but the chain.  The sending warp composes a tile's runs and sends
//     the tile's map to every CTA of the cluster (st.async into distributed shared memory, counted
//     by an mbarrier there), and leaves each run the map of those before it; the receiving warp
//     composes the tiles of the cluster in order and hands the team the state that enters its tile.
//     A thread's part in the exchange is one store and two loads, and a round's maps are under way
//     while the round before is still being received.
//   * Each warp copies its own tokens ahead into its own ring of stages (cp.async, 16 bytes at a
//     time): no barrier between warps, and the bytes in flight are those of the ring.  A stage is kept
//     until its tokens are read a second time, so that registers hold the decays alone (and in the
//     backward the slopes): holding the tokens as well took 73 us instead of 58 once.  With the
//     sigmoid gate a thread leaves there, in the place of the warp's g and x, what it needs the second
//     time: z x, or in the backward z.
// Two values go through the packed fp32 instructions (bf16 inputs).
//
// Measured (of 6.78 TB/s): 32 x 16384 x 64 bf16, sigmoid gate: 40.3 us forward (74%) and 60.7 us backward
// (84%), decay gate 33.7 (88%) and 55.2 (92%); 4 x 8192 x 512 fp32, sigmoid: 34.7 and 53.6 us (86 and
// 93%).  bf16 with the sigmoid gate is bound by issue and by the chain, the others by memory.  Teams of
// four warps put one on each scheduler, so that all four end together: with three teams of six the
// slowest scheduler held up the chain (50.8 us where four of four took 44.0).  Sequences and channels too
// few for the GPU's clusters cost the rest: 8 x 65536 x 64 bf16 runs in 32-byte pieces of a row on 128
// SMs, 47.5 us (65%) with the sigmoid gate and the states kept.  That gate's numbers are worked out for 8
// tokens at a time, 16 in the backward: of 2, 4, 8 and 16 the best (forward 49.5, 48.6, 48.1 and 49.4 us
// there; backward 64.4, 63.5, 63.5 and 61.9 at 32 x 16384 x 64).
//
// Copies are of 16 bytes where rows and pointers allow it, else of each thread's own 4 or 8 (which
// takes more instructions).  scan.cu's kernels take short sequences and what is odd beyond that; where
// they meet is in lapl_scan_create, lapl_scan_forward and lapl_scan_backward.
//
// With T teams, a CTA whose receiving warp is at round r has sent maps up to round r + T - 1, so
// another may be at r + T and send up to r + 2T - 1: maps of 2T rounds may be there at once.
//
// The receiving warp's wait for the cluster's maps is bounded (one second): when it gives up it sets
// kErrBitScan in the device error word and goes on without waiting for maps, so that the kernel ends;
// its outputs are then undefined.  It still keeps step with its own CTA: its arrival for a round at the
// barrier of the team's states must not come before the team has left that barrier's round before, which
// the round's maps tell where they have come and the sending warp's arrival at a barrier of their own
// where they have not.  No CTA of a cluster leaves before all have come to their end.
#pragma once

#include "scan.cuh"

namespace lapl {
namespace scan {
namespace pipe {

constexpr int kMaxCluster = 8;     // CTAs
// Rounds of maps that may have arrived: see above.
__host__ __device__ constexpr int slots_of(int teams) { return 2 * teams; }
// Teams, and worker warps of a team: with the chain's two warps 18 of up to 112 registers forward, 14
// of up to 128 backward.
constexpr int kForwardTeams = 4, kForwardWarps = 4, kBackwardTeams = 3, kBackwardWarps = 4;

// Bytes of a row of one tensor in shared memory, and from one run of kT rows to the next: a warp
// reads rows of 32 / kLanes runs at once, which lie side by side in the banks thanks to one row of
// space after each run.
template <int kLanes, int kBytes>
struct Tile {
  static constexpr int kRow = kLanes * kBytes;
  static constexpr int kRun = kT * kRow + (kLanes < 32 ? kRow : 0);
  static constexpr int kWarp = 32 / kLanes * kRun;       // of a warp's stage
  static constexpr int kPieces = kRow / 16;              // 16-byte pieces of a row
  static constexpr int kRows = 32 / kPieces;             // rows that a warp copies at once
  static constexpr int kCopies = 32 / kLanes * kT / kRows;   // of a thread for a stage
};

// Shared memory after the stages, in bytes: runs' maps, states that enter the teams' tiles, mbarriers,
// and for each CTA of the cluster the maps that have arrived.
struct Layout {
  unsigned runs, enters, bars, slots, a_cta;
  __host__ __device__ constexpr unsigned total(int cluster) const { return slots + a_cta * cluster; }
};
template <int V, int kLanes>
__host__ __device__ constexpr Layout layout_of(int teams, int warps, unsigned stage_bytes, int stages) {
  Layout l = {};
  l.runs = (unsigned)(teams * warps * stages) * stage_bytes;
  l.enters = l.runs + teams * warps * 32 * 2 * V * 4;
  l.bars = l.enters + teams * kLanes * V * 4;
  l.slots = l.bars + (slots_of(teams) * 8 + 15) / 16 * 16;
  l.a_cta = slots_of(teams) * kLanes * 2 * V * 4;
  return l;
}

using ops::smem_u32, ops::copy16, ops::copies_left;

__device__ __forceinline__ unsigned at_rank(unsigned addr, int rank) {
  unsigned r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// The same for a thread's own 4 or 8.
template <int kBytes>
__device__ __forceinline__ void copy_own(unsigned dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes),
               "n"(kBytes) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A map as it lies in shared memory: V factors, then V terms.
template <int V>
struct Map {
  Vec<V> a, b;
};
__device__ __forceinline__ void put_map(unsigned at, const Map<2>& m) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(m.a.f[0]), "f"(m.a.f[1]),
               "f"(m.b.f[0]), "f"(m.b.f[1]) : "memory");
}
__device__ __forceinline__ void put_map(unsigned at, const Map<1>& m) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(m.a.f[0]), "f"(m.b.f[0]) : "memory");
}
__device__ __forceinline__ void get_map(unsigned at, Map<2>& m) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(m.a.f[0]), "=f"(m.a.f[1]), "=f"(m.b.f[0]), "=f"(m.b.f[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ void get_map(unsigned at, Map<1>& m) {
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(m.a.f[0]), "=f"(m.b.f[0]) : "r"(at) : "memory");
}
// The same into a CTA of the cluster, counted by an mbarrier there.
__device__ __forceinline__ void send_map(unsigned at, unsigned bar, const Map<2>& m) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2, %3, %4, %5}, [%1];"
               ::"r"(at), "r"(bar), "f"(m.a.f[0]), "f"(m.a.f[1]), "f"(m.b.f[0]), "f"(m.b.f[1])
               : "memory");
}
__device__ __forceinline__ void send_map(unsigned at, unsigned bar, const Map<1>& m) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%2, %3}, [%1];"
               ::"r"(at), "r"(bar), "f"(m.a.f[0]), "f"(m.b.f[0]) : "memory");
}
__device__ __forceinline__ void put_state(unsigned at, const Vec<2>& v) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.f[0]), "f"(v.f[1]) : "memory");
}
__device__ __forceinline__ void put_state(unsigned at, const Vec<1>& v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v.f[0]) : "memory");
}
__device__ __forceinline__ void get_state(unsigned at, Vec<2>& v) {
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.f[0]), "=f"(v.f[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ void get_state(unsigned at, Vec<1>& v) {
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v.f[0]) : "r"(at) : "memory");
}

// A thread's channels of a token in a stage.
template <bool k16, int V>
__device__ __forceinline__ Raw<k16, V> read_raw(unsigned at) {
  Raw<k16, V> r;
  if constexpr (k16 && V == 1) {
    unsigned short t;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(t) : "r"(at) : "memory");
    r.w[0] = t;
  } else if constexpr (!k16 && V == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[V - 1]) : "r"(at) : "memory");
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.w[0]) : "r"(at) : "memory");
  }
  return r;
}

__device__ __forceinline__ unsigned long long nanoseconds() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// What a thread keeps of token k, V floats, where the warp's g and x were: 8 tokens in each of the two, of
// which one is `apart` bytes behind the other.  Whoever keeps the first of a half has met the warp after
// all of its threads read that half's words.
constexpr int kHalf = kT / 2;
template <int V>
__device__ __forceinline__ unsigned keep_at(unsigned warp_stage, unsigned apart, int k) {
  return warp_stage + (k < kHalf ? 0u : apart) + (k % kHalf * 32 + ((int)threadIdx.x & 31)) * (V * 4);
}

// Until the phase of the given parity is complete, or false after `bound` ns.
__device__ __forceinline__ bool wait_phase(unsigned bar, unsigned parity, unsigned long long bound) {
  const unsigned at_once = (unsigned)min(bound, 1000000ull);   // a look may last that long: up to 1 ms
  auto done = [&] {
    unsigned d;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(d) : "r"(bar), "r"(parity), "r"(at_once)
                 : "memory");
    return d != 0;
  };
  if (done()) return true;
  const unsigned long long t0 = nanoseconds();
  while (!done())
    if (nanoseconds() - t0 > bound) return false;
  return true;
}

// Named barriers: a team's runs are written; the states that enter its tile are; the sending warp has
// seen the runs.  (0 is __syncthreads'; there are 16.)
template <int kTeams>
__device__ __forceinline__ int runs_bar(int team) { return 1 + team; }
template <int kTeams>
__device__ __forceinline__ int states_bar(int team) { return 1 + kTeams + team; }
template <int kTeams>
__device__ __forceinline__ int seen_bar(int team) {
  static_assert(1 + 3 * kTeams <= 16, "named barriers");
  return 1 + 2 * kTeams + team;
}

// What a CTA works on.
template <int kLanes, int V>
struct Unit {
  long long s;
  int c0;             // first channel
  int rank, cluster, len;
  __device__ __forceinline__ explicit Unit(const Args& a) {
    cluster = a.geo.cluster;
    const int unit = blockIdx.x / cluster;
    rank = blockIdx.x - unit * cluster;
    s = unit / a.geo.blocks;
    c0 = (unit - (int)s * a.geo.blocks) * kLanes * V;
    len = a.n;
    if (a.lengths) len = max(0, min(a.n, a.lengths[s]));
  }
};

// Copies a warp's tokens of a round into a stage: rows of `first`.. in processing order, those from
// `len` on as zeros, and channels from C on too.  In 16-byte pieces, or with `fine` in the threads'
// own kBytes (4 or 8) where a row or the tensor does not start at a multiple of 16 bytes.
template <int kLanes, int kBytes, int kElem>
__device__ __forceinline__ void copy_stage(unsigned stage, const void* base, long long stride,
                                           const Args& a, long long s, int c0, int len,
                                           long long first, bool fine) {
  using T = Tile<kLanes, kBytes>;
  const int lane = threadIdx.x & 31;
  const int pieces = fine ? kLanes : T::kPieces;    // of a row
  const int row = fine ? lane / kLanes * kT : lane / T::kPieces, piece = lane & (pieces - 1);
  const int size = fine ? kBytes : 16;
  const int bytes = max(0, min(size, (a.c - c0) * kElem - piece * size));   // within C
  const long long i0 = first + row;
  const long long token = s * a.n + (a.reverse ? len - 1 - i0 : i0);
  const char* src = reinterpret_cast<const char*>(base) + (token * stride + c0) * kElem + piece * size;
  const int live = bytes ? (int)max(0ll, min((long long)len - i0, 64ll)) : 0;   // rows from i0 on
  const unsigned dst = stage + row * T::kRow + row / kT * (T::kRun - kT * T::kRow) + piece * size;
  if (!fine) {
    const long long by = (a.reverse ? -stride : stride) * (T::kRows * kElem);
#pragma unroll
    for (int k = 0; k < T::kCopies; ++k, src += by) {
      const bool in = k * T::kRows < live;
      copy16(dst + k * T::kRows * T::kRow + k * T::kRows / kT * (T::kRun - kT * T::kRow),
             in ? src : base, in ? bytes : 0);
    }
  } else if constexpr (kBytes >= 4) {
    // A thread copies what it will read itself: its run.
    const long long by = (a.reverse ? -stride : stride) * kElem;
#pragma unroll
    for (int k = 0; k < kT; ++k, src += by)
      copy_own<kBytes>(dst + k * T::kRow, k < live ? src : base, k < live ? bytes : 0);
  }
}

template <int V>
__device__ __forceinline__ Vec<V> shuffle(const Vec<V>& v, int from) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.f[i] = __shfl_sync(0xffffffffu, v.f[i], from);
  return r;
}

// The sending warp: composes the runs of every round's tile, sends the tile's map to all CTAs of
// the cluster, and leaves in each run's place the map of the runs before it.  Lanes 0 .. kLanes-1
// have the first kWarps runs in processing order, the next kLanes lanes the next.
template <int kLanes, int V, int kTeams, int kWarps, bool kDown>
__device__ __forceinline__ void send_chain(const Args& a, const Unit<kLanes, V>& u, unsigned smem,
                                           const Layout& l, unsigned bars) {
  constexpr int kMap = 2 * V * 4, kSets = 32 / kLanes, kRuns = kWarps * kSets;
  constexpr int kBy = (kDown ? -kLanes : kLanes) * kMap;   // from a lane's run to its next
  const int lane = threadIdx.x & 31, pos = lane & (kLanes - 1), set = lane / kLanes;
  const int first = (kDown ? kRuns - 1 - set * kWarps : set * kWarps) * kLanes + pos;
  // Fault injection: a round whose maps are not sent.
  const int lost_round = a.skip_last ? max(0, a.geo.tiles - a.skip_last) : -1;
  for (int r = 0; r < a.geo.tiles; ++r) {
    const int team = r % kTeams, slot = r % slots_of(kTeams);
    const unsigned runs = smem + l.runs + (team * kWarps * 32 + first) * kMap;
    bar_sync(runs_bar<kTeams>(team), kWarps * 32 + 32);
    bar_arrive(seen_bar<kTeams>(team), 64);
    Map<V> m[kWarps];
#pragma unroll
    for (int k = 0; k < kWarps; ++k) get_map(runs + k * kBy, m[k]);
    Map<V> all = m[0], before = {fill<V>(1.f), fill<V>(0.f)};
#pragma unroll
    for (int k = 1; k < kWarps; ++k) {
      all.b = fma(m[k].a, all.b, m[k].b);
      all.a = mul(m[k].a, all.a);
    }
    // Over the sets of lanes: `all` up to and with this one, `before` without it.
#pragma unroll
    for (int o = 1; o < kSets; o *= 2) {
      const Map<V> low = {shuffle(all.a, lane - o * kLanes), shuffle(all.b, lane - o * kLanes)};
      if (set >= o) {
        all.b = fma(all.a, low.b, all.b);
        all.a = mul(all.a, low.a);
      }
    }
    if constexpr (kSets > 1) {
      const Map<V> low = {shuffle(all.a, lane - kLanes), shuffle(all.b, lane - kLanes)};
      if (set > 0) before = low;
      all = {shuffle(all.a, 32 - kLanes + pos), shuffle(all.b, 32 - kLanes + pos)};
    }
    const unsigned to = smem + l.slots + ((slot * u.cluster + u.rank) * kLanes + pos) * kMap;
    if (r != lost_round)
      for (int k = set; k < u.cluster; k += kSets)
        send_map(at_rank(to, k), at_rank(bars + slot * 8, k), all);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      put_map(runs + k * kBy, before);
      before.b = fma(m[k].a, before.b, m[k].b);
      before.a = mul(m[k].a, before.a);
    }
    bar_arrive(states_bar<kTeams>(team), kWarps * 32 + 64);
  }
}

// The receiving warp's state before the first round.  Read before the cluster meets for the first
// time: its first CTA may write the last state over it, once all have sent their maps.
template <int kLanes, int V>
__device__ __forceinline__ Vec<V> first_state(const Args& a, const Unit<kLanes, V>& u, bool receives,
                                              const float* start) {
  const int c = u.c0 + ((int)threadIdx.x & (kLanes - 1)) * V;
  return receives && start && c < a.c ? widen(load_raw<false, V>(start + u.s * a.c + c))
                                      : fill<V>(0.f);
}

// The receiving warp: the state that enters every round's tile, from the tiles of the cluster.  True if
// a wait gave up.
template <int kLanes, int V, int kTeams, int kWarps, bool kDown>
__device__ __forceinline__ bool receive_chain(const Args& a, const Unit<kLanes, V>& u, unsigned smem,
                                              const Layout& l, unsigned bars, Vec<V> carry,
                                              float* finish, unsigned* err) {
  constexpr int kMap = 2 * V * 4;
  const int lane = threadIdx.x & 31, pos = lane & (kLanes - 1);
  const int c = u.c0 + pos * V;
  const bool on = lane < kLanes && c < a.c;
  bool lost = false;
  for (int r = 0; r < a.geo.tiles; ++r) {
    const int team = r % kTeams, slot = r % slots_of(kTeams);
    const unsigned bar = bars + slot * 8, bytes = u.cluster * kLanes * kMap;
    if (!lost) {
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                     ::"r"(bar), "r"(bytes) : "memory");
      lost = __any_sync(0xffffffffu, !wait_phase(bar, (r / slots_of(kTeams)) & 1, a.wait_ns));
    } else if (lane == 0) {
      // The slot's phase may have had its one arrival; the bytes that still come are counted off.
      asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;"
                   ::"r"(bar), "r"(bytes) : "memory");
    }
    // The sending warp has come by this round.  The round's maps, this CTA's among them, say so.
    if (lost) bar_sync(seen_bar<kTeams>(team), 64);
    else bar_arrive(seen_bar<kTeams>(team), 64);
    const unsigned slots = smem + l.slots + (slot * u.cluster * kLanes + pos) * kMap;
    Vec<V> enter = carry;
    for (int k = 0; k < u.cluster; ++k) {
      const int rank = kDown ? u.cluster - 1 - k : k;
      if (rank == u.rank) enter = carry;
      Map<V> m;
      get_map(slots + rank * kLanes * kMap, m);
      carry = fma(m.a, carry, m.b);
    }
    if (lane < kLanes) put_state(smem + l.enters + (team * kLanes + pos) * (V * 4), enter);
    bar_arrive(states_bar<kTeams>(team), kWarps * 32 + 64);
  }
  if (lost && lane == 0) atomicOr(err, kErrBitScan);
  if (finish && on && u.rank == 0) store_vec<false>(finish + u.s * a.c + c, carry);
  return lost;
}

__device__ __forceinline__ void start_barriers(unsigned bars, int slots) {
  if (threadIdx.x == 0) {
    for (int k = 0; k < slots; ++k)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + k * 8) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The end of a CTA.  One that gave up a wait may still be sent maps: all are on their way once the
// cluster has met, and it stays for 0.1 ms more (at most 10,000 looks at the clock), far longer than
// they take.
__device__ __forceinline__ void leave(bool lost) {
  cluster_sync();
  if (!lost) return;
  const unsigned long long t0 = nanoseconds();
  for (int k = 0; k < 10000 && nanoseconds() - t0 < 100000ull; ++k) __nanosleep(100);
}

template <bool kIn16, bool kOut16, bool kSig, int kLanes, int kStages, int kTeams, int kWarps>
__global__ void __launch_bounds__((kTeams * kWarps + 2) * 32, 1)
scan_forward_pipe_kernel(const Args a, unsigned* err) {
  constexpr int V = kIn16 ? 2 : 1, kElem = kIn16 ? 2 : 4, kOut = kOut16 ? 2 : 4;
  using T = Tile<kLanes, V * kElem>;
  constexpr unsigned kStage = 2 * T::kWarp;
  extern __shared__ __align__(128) unsigned char dynamic[];
  const unsigned smem = smem_u32(dynamic);
  constexpr Layout l = layout_of<V, kLanes>(kTeams, kWarps, kStage, kStages);
  const unsigned bars = smem + l.bars;
  const Unit<kLanes, V> unit(a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Vec<V> start = first_state(a, unit, warp == kTeams * kWarps + 1, a.h0);
  start_barriers(bars, slots_of(kTeams));
  cluster_sync();
  bool lost = false;   // in the receiving warp
  if (warp == kTeams * kWarps) {
    send_chain<kLanes, V, kTeams, kWarps, false>(a, unit, smem, l, bars);
  } else if (warp == kTeams * kWarps + 1) {
    lost = receive_chain<kLanes, V, kTeams, kWarps, false>(a, unit, smem, l, bars, start, a.final_state, err);
  } else {
    const int team = warp / kWarps, wt = warp - team * kWarps;   // place in the team
    const int run = wt * (32 / kLanes) + lane / kLanes;
    const int pos = lane & (kLanes - 1), c = unit.c0 + pos * V;
    const bool on = c < a.c;
    const int live = on ? unit.len : 0;
    const unsigned ring = smem + warp * kStages * kStage;
    const unsigned my = pos * (V * kElem) + (lane / kLanes) * T::kRun;   // within a stage
    const int tile = kWarps * (32 / kLanes) * kT;
    auto place = [&](int r, int k) {   // first token of run k of the team's tile in round r
      return ((long long)r * unit.cluster + unit.rank) * tile + k * kT;
    };
    auto ahead = [&](int r, int stage) {
      if (r < a.geo.tiles) {
        const long long first = place(r, wt * (32 / kLanes));
        copy_stage<kLanes, V * kElem, kElem>(ring + stage * kStage, a.g, a.g_stride, a, unit.s,
                                             unit.c0, unit.len, first, a.fine);
        copy_stage<kLanes, V * kElem, kElem>(ring + stage * kStage + T::kWarp, a.x, a.x_stride, a,
                                             unit.s, unit.c0, unit.len, first, a.fine);
      }
      ops::close_copies();
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) ahead(team + k * kTeams, k);
    int stage = 0;
    for (int r = team; r < a.geo.tiles; r += kTeams) {
      const long long start = place(r, run);
      const int i0 = (int)min(start, (long long)a.n);
      copies_left<kStages - 1>();
      __syncwarp();
      const unsigned from = ring + stage * kStage + my;
      Vec<V> decay[kT];
      Map<V> m = {{}, fill<V>(0.f)};
      Factor<kSig, V> factor;
      if constexpr (kSig) {
        Raw<kIn16, V> rg[kT];
#pragma unroll
        for (int k = 0; k < kT; ++k) rg[k] = read_raw<kIn16, V>(from + k * T::kRow);
        Raw<kIn16, V> rx[kT];
        gates<8, kIn16, V>(rg, i0, live, [&](int k, const Gate<V>& g) {
          if (k % kHalf == 0) {
#pragma unroll
            for (int u = k; u < k + kHalf; ++u) rx[u] = read_raw<kIn16, V>(from + T::kWarp + u * T::kRow);
            __syncwarp();
          }
          const Vec<V> b = mul(g.z, widen(rx[k]));
          factor.take(g);
          m.b = fma(g.a, m.b, b);
          put_state(keep_at<V>(ring + stage * kStage, T::kWarp, k), b);
          decay[k] = g.a;
        });
      } else {
#pragma unroll
        for (int k = 0; k < kT; ++k) decay[k] = widen(read_raw<kIn16, V>(from + k * T::kRow));
        if (i0 + kT > live) {
#pragma unroll
          for (int k = 0; k < kT; ++k)
            if (i0 + k >= live) decay[k] = fill<V>(1.f);
        }
#pragma unroll
        for (int k = 0; k < kT; ++k) {
          factor.take({decay[k], {}});
          m.b = fma(decay[k], m.b, widen(read_raw<kIn16, V>(from + T::kWarp + k * T::kRow)));
        }
      }
      m.a = factor.value();
      auto next = [&](int k, const Vec<V>& h) {
        Vec<V> b;
        if constexpr (kSig) {
          get_state(keep_at<V>(ring + stage * kStage, T::kWarp, k), b);
          return fma(decay[k], h, b);
        }
        return fma(decay[k], h, widen(read_raw<kIn16, V>(from + T::kWarp + k * T::kRow)));
      };
      put_map(smem + l.runs + (team * kWarps * 32 + wt * 32 + lane) * (2 * V * 4), m);
      bar_arrive(runs_bar<kTeams>(team), kWarps * 32 + 32);
      bar_sync(states_bar<kTeams>(team), kWarps * 32 + 64);
      Vec<V> h;
      get_state(smem + l.enters + (team * kLanes + pos) * (V * 4), h);
      get_map(smem + l.runs + (team * kWarps * 32 + wt * 32 + lane) * (2 * V * 4), m);
      h = fma(m.a, h, m.b);
      if (on && i0 < a.n) {
        if (a.states) store_vec<false>(a.states + (unit.s * a.chunks + i0 / kT) * a.c + c, h);
        const long long row = unit.s * a.n + (a.reverse ? unit.len - 1 - i0 : i0);
        char* q = reinterpret_cast<char*>(a.out) + (row * a.c + c) * kOut;
        const long long by = (a.reverse ? -(long long)a.c : (long long)a.c) * kOut;
        if (i0 + kT <= live) {
#pragma unroll
          for (int k = 0; k < kT; ++k, q += by) {
            h = next(k, h);
            store_vec<kOut16>(q, h);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kT; ++k, q += by) {
            const int i = i0 + k;
            h = next(k, h);
            if (i < live)
              store_vec<kOut16>(q, h);
            else if (i < a.n)
              store_vec<kOut16>(reinterpret_cast<char*>(a.out) + ((unit.s * a.n + i) * a.c + c) * kOut,
                                fill<V>(0.f));
          }
        }
      }
      // The stage is read: the team's round after the next one goes into it.
      __syncwarp();
      ahead(r + kStages * kTeams, stage);
      if (++stage == kStages) stage = 0;
    }
    copies_left<0>();
  }
  leave(lost);
}

template <bool kIn16, bool kGrad16, bool kSig, int kLanes, int kStages, int kTeams, int kWarps>
__global__ void __launch_bounds__((kTeams * kWarps + 2) * 32, 1)
scan_backward_pipe_kernel(const Args a, unsigned* err) {
  constexpr int V = kIn16 ? 2 : 1, kElem = kIn16 ? 2 : 4, kGrad = kGrad16 ? 2 : 4;
  using T = Tile<kLanes, V * kElem>;
  using TG = Tile<kLanes, V * kGrad>;
  constexpr unsigned kStage = 2 * T::kWarp + TG::kWarp;
  extern __shared__ __align__(128) unsigned char dynamic[];
  const unsigned smem = smem_u32(dynamic);
  constexpr Layout l = layout_of<V, kLanes>(kTeams, kWarps, kStage, kStages);
  const unsigned bars = smem + l.bars;
  const Unit<kLanes, V> unit(a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Vec<V> start = first_state(a, unit, warp == kTeams * kWarps + 1, a.dfinal);
  start_barriers(bars, slots_of(kTeams));
  cluster_sync();
  bool lost = false;   // in the receiving warp
  if (warp == kTeams * kWarps) {
    send_chain<kLanes, V, kTeams, kWarps, true>(a, unit, smem, l, bars);
  } else if (warp == kTeams * kWarps + 1) {
    lost = receive_chain<kLanes, V, kTeams, kWarps, true>(a, unit, smem, l, bars, start, a.dh0, err);
  } else {
    const int team = warp / kWarps, wt = warp - team * kWarps;
    const int run = wt * (32 / kLanes) + lane / kLanes;
    const int pos = lane & (kLanes - 1), c = unit.c0 + pos * V;
    const bool on = c < a.c;
    const int live = on ? unit.len : 0;
    const unsigned ring = smem + warp * kStages * kStage;
    const unsigned my = pos * (V * kElem) + (lane / kLanes) * T::kRun;
    const unsigned my_grad = 2 * T::kWarp + pos * (V * kGrad) + (lane / kLanes) * TG::kRun;
    const int tile = kWarps * (32 / kLanes) * kT;
    auto place = [&](int r, int k) {   // rounds go down the sequence
      return ((long long)(a.geo.tiles - 1 - r) * unit.cluster + unit.rank) * tile + k * kT;
    };
    auto ahead = [&](int r, int stage) {
      if (r < a.geo.tiles) {
        const long long first = place(r, wt * (32 / kLanes));
        const unsigned to = ring + stage * kStage;
        copy_stage<kLanes, V * kElem, kElem>(to, a.g, a.g_stride, a, unit.s, unit.c0, unit.len, first,
                                             a.fine);
        copy_stage<kLanes, V * kElem, kElem>(to + T::kWarp, a.x, a.x_stride, a, unit.s, unit.c0,
                                             unit.len, first, a.fine);
        copy_stage<kLanes, V * kGrad, kGrad>(to + 2 * T::kWarp, a.dout, a.c, a, unit.s, unit.c0,
                                             unit.len, first, a.fine_dout);
      }
      ops::close_copies();
    };
    auto state = [&](int r) {
      const long long i = place(r, run);
      if (r < a.geo.tiles && on && i < a.n)
        return widen(load_raw<false, V>(a.states + (unit.s * a.chunks + i / kT) * a.c + c));
      return fill<V>(0.f);
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) ahead(team + k * kTeams, k);
    Vec<V> next = state(team);
    int stage = 0;
    for (int r = team; r < a.geo.tiles; r += kTeams) {
      const int i0 = (int)min(place(r, run), (long long)a.n);
      copies_left<kStages - 1>();
      __syncwarp();
      const unsigned from = ring + stage * kStage;
      Vec<V> decay[kT], slope[kT], h = next;
      Factor<kSig, V> factor;
      if constexpr (kSig) {
        Raw<kIn16, V> rg[kT];
#pragma unroll
        for (int k = 0; k < kT; ++k) rg[k] = read_raw<kIn16, V>(from + my + k * T::kRow);
        Raw<kIn16, V> rx[kT];
        gates<kT, kIn16, V>(rg, i0, live, [&](int k, const Gate<V>& g) {
          if (k % kHalf == 0) {
#pragma unroll
            for (int u = k; u < k + kHalf; ++u)
              rx[u] = read_raw<kIn16, V>(from + my + T::kWarp + u * T::kRow);
            __syncwarp();
          }
          const Vec<V> x = widen(rx[k]);
          factor.take(g);
          slope[k] = mul(g.z, sub(h, x));
          h = fma(g.a, h, mul(g.z, x));
          put_state(keep_at<V>(from, T::kWarp, k), g.z);
          decay[k] = g.a;
        });
      } else {
#pragma unroll
        for (int k = 0; k < kT; ++k) decay[k] = widen(read_raw<kIn16, V>(from + my + k * T::kRow));
        if (i0 + kT > live) {
#pragma unroll
          for (int k = 0; k < kT; ++k)
            if (i0 + k >= live) decay[k] = fill<V>(1.f);
        }
      }
      next = state(r + kTeams);
      Map<V> m = {{}, fill<V>(0.f)};
#pragma unroll
      for (int k = kT - 1; k >= 0; --k) {
        if constexpr (!kSig) factor.take({decay[k], {}});
        m.b = mul(decay[k], add(widen(read_raw<kGrad16, V>(from + my_grad + k * TG::kRow)), m.b));
      }
      m.a = factor.value();
      put_map(smem + l.runs + (team * kWarps * 32 + wt * 32 + lane) * (2 * V * 4), m);
      bar_arrive(runs_bar<kTeams>(team), kWarps * 32 + 32);
      if constexpr (!kSig) {   // while the chain goes on
#pragma unroll
        for (int k = 0; k < kT; ++k) {
          slope[k] = h;
          h = fma(decay[k], h, widen(read_raw<kIn16, V>(from + my + T::kWarp + k * T::kRow)));
        }
      }
      bar_sync(states_bar<kTeams>(team), kWarps * 32 + 64);
      Vec<V> E;
      get_state(smem + l.enters + (team * kLanes + pos) * (V * 4), E);
      get_map(smem + l.runs + (team * kWarps * 32 + wt * 32 + lane) * (2 * V * 4), m);
      E = fma(m.a, E, m.b);
      if (on && i0 < a.n) {
        const int left = live - i0;
        const long long row = unit.s * a.n + (a.reverse ? unit.len - kT - i0 : i0 + kT - 1);
        char* qx = reinterpret_cast<char*>(a.dx) + (row * a.x_stride + c) * kGrad;
        char* qg = reinterpret_cast<char*>(a.dg) + (row * a.g_stride + c) * kGrad;
        const long long bx = (a.reverse ? a.x_stride : -a.x_stride) * kGrad;
        const long long bg = (a.reverse ? a.g_stride : -a.g_stride) * kGrad;
#pragma unroll
        for (int k = kT - 1; k >= 0; --k, qx += bx, qg += bg) {
          const Vec<V> D = add(widen(read_raw<kGrad16, V>(from + my_grad + k * TG::kRow)), E);
          E = mul(decay[k], D);
          Vec<V> z = {}, dx, dg;
          if constexpr (kSig) get_state(keep_at<V>(from, T::kWarp, k), z);
          step_gradients<kSig>(z, slope[k], D, E, dx, dg);
          if (k < left) {
            store_vec<kGrad16>(qx, dx);
            store_vec<kGrad16>(qg, dg);
          }
        }
        for (int i = max(i0, live); i < min(i0 + kT, a.n); ++i) {
          const long long at = unit.s * a.n + i;
          store_vec<kGrad16>(reinterpret_cast<char*>(a.dx) + (at * a.x_stride + c) * kGrad, fill<V>(0.f));
          store_vec<kGrad16>(reinterpret_cast<char*>(a.dg) + (at * a.g_stride + c) * kGrad, fill<V>(0.f));
        }
      }
      __syncwarp();
      ahead(r + kStages * kTeams, stage);
      if (++stage == kStages) stage = 0;
    }
    copies_left<0>();
  }
  leave(lost);
}

using PipeKernel = void (*)(Args, unsigned*);

// A kernel, its worker warps a team and its shared memory.
struct Pick {
  PipeKernel kernel;
  int teams, warps;
  Layout layout;
};
// For lanes of 32, 16 or 8.
Pick forward_f32(bool out16, bool sig, int lanes);
Pick forward_bf16(bool out16, bool sig, int lanes);
Pick backward_f32(bool grad16, bool sig, int lanes);
Pick backward_bf16(bool grad16, bool sig, int lanes);

}  // namespace pipe
}  // namespace scan
}  // namespace lapl
