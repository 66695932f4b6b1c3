// decay_tc.cu -- a pass of the linear attention with decays in chunks of 128 tokens on the tensor
// cores (decay.cuh has the formulas): bf16 rows, 64 columns of the state to a CTA.
//
// With g the head's decay, a chunk of n tokens (m = 0 .. n-1 in processing order) and the state S before
// it, the chunk's outputs and the state after it are
//   o_m = os ( sum_{j <= m} zs g^{m-j} (x_m . y_j) z_j  +  g^{m+1} x_m S ),
//   S' = g^n S + sum_j zs g^{n-1-j} y_j z_j^T.
// Four products of 128-row tiles (tcgen05, bf16 operands, fp32 sums in tensor memory):
//   scores  X Y^T          -> P = scores times decays, masked
//   inner   P Z            P from tensor memory
//   outer   X S
//   add     Y^T Z'         Z' = Z with each token's decay to the chunk's end
// x, y and z enter as they are.  What is computed is split into bf16 parts: Z' into three, which leave out
// 2^-24 of a value, as what the state loses is carried along (of 2 x 16 sequences of 4096 tokens of 64 x 128 the
// final state is 1.8e-7 off, root mean square).  P and S into three as well where outputs are fp32 (2.5e-7 off, of
// 128 x 128 3.1e-7; the formula in fp32 4.5e-7 and 4.7e-7), their smallest parts' products first: what is added in
// tensor memory is cut off by the sum so far (largest parts first 5.1e-7 and 8.1e-7).  Where outputs are bf16, P and
// S go into two parts, which leave out 2^-16: that alone makes outputs 2.5e-6 off, their rounding to bf16 1.7e-3,
// and both together as much as with three parts (1.65849e-3 either way).  The third part costs a stage of shared
// memory: 32 sequences of 16384 tokens of 64 x 64 with fp32 outputs 154 us, with two parts 130; 104 us with
// bf16 ones, with three parts 154.
//
// One CTA of an SM works through a segment of a sequence; its warps:
//   0-7    scores to P (warp w: rows 32 (w % 4) and up, every other block of 32 columns), and the
//          outputs: both accumulators, the decays, through shared memory to whole runs of rows.  Warp 0:
//          the copies of X, Y and Z tiles by TMA, 128-byte swizzle, a chunk ahead
//   8-11   the state, fp32 in registers: g^n S + add, and its parts as an operand
//   8-14   Z' from Z
//   15     the products
// (16 warps, so that each may have 128 registers: with 18 it was 96, and spills.)
// Before it, where a sequence has several segments: decay_sums_kernel forms each segment's own
// contribution to the state (add, with decays to the segment's end) and decay_carry_kernel the states
// before each.
//
// Bound by the chain of a chunk: scores, P, its product, the outputs, and beside them Z', its product, the
// state: 4,000 clocks, of which the products take 2,060 and the bytes, at 6.8 TB/s for all SMs, 2,790.  4 x 8
// sequences of 16384 tokens of 64 x 64 in bf16: 104 us (2.6 TB/s of 268 MB; 34 us the sums, 73 the
// outputs); the backward, three passes side by side, 260.  Of 128 x 128, 2 x 8 x 8192 tokens: 102 and 228,
// with room for one stage.
#include <algorithm>

#include "decay_tc.cuh"

namespace lapl {
namespace decay {
namespace {

using namespace tc;
using ops::Vec;

constexpr int kChunk = kTcChunk;
constexpr int kD = 64;                        // columns of a tile of X, Y or Z
constexpr unsigned kTile = kChunk * kD * 2;   // bytes of one, or of a part of Z'
constexpr int kParts = 3;                     // of Z'
constexpr int kPieces = kChunk * kD / 8;      // of a tile, of 16 bytes
constexpr int kAhead = 2;                     // chunks from a copy to the prefetch into L2 beside it
// kBoxes: tiles that rows of X and Y take, padded: 1 (up to 64 values) or 2 (up to 128).  Z is one, the
// pass's columns in steps of 64.
// kExact: P and S in three parts, for fp32 outputs.
// Stages of X, Y and Z, and of Z': of the longer rows, and with a third part of S, shared memory holds one.
constexpr int stages_of(int boxes, bool exact) { return boxes == 1 && !exact ? 2 : 1; }
constexpr int parts_of(bool exact) { return exact ? 3 : 2; }   // of P and S

// Columns of tensor memory.
constexpr unsigned kScores = 0, kInner = 256, kOuter = 320, kAdd = 384, kColumns = 512;

struct TcArgs {
  Args a;
  CUtensorMap x[kMaxPasses], y[kMaxPasses], z[kMaxPasses];
  unsigned* err;
  unsigned long long wait_ns;
  int skip_last;
};

// The chunks of a segment of one sequence, in processing order.
struct Chunks {
  int len, all;     // tokens of the sequence, its chunks
  int first, count; // the segment's chunks with tokens
  int reverse;
  __device__ __forceinline__ Chunks(const Args& a, const Pass& p, int bh, int segment) {
    len = Range(a, bh, segment).len;
    all = (len + kChunk - 1) / kChunk;
    const int per = a.per_segment / kChunk;
    first = segment * per;
    count = max(0, min(first + per, all) - first);
    reverse = p.reverse;
  }
  // Place in memory of the segment's chunk i, and its tokens.
  __device__ __forceinline__ int place(int i) const { return reverse ? all - 1 - first - i : first + i; }
  __device__ __forceinline__ int tokens(int i) const { return min(kChunk, len - place(i) * kChunk); }
};

// A place in a ring of stages, and the parity of the stage's current phase (kept by adding: a remainder by
// a number of stages that is no constant took the products' thread 100 clocks).
struct Ring {
  int stage = 0;
  unsigned phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// The tokens of Z, times late[row] and by, as kParts tiles; rows from n on as zeros, in Z and Y too, whose
// products with zeros would not be zeros for what is not finite there.  Pieces kFirst to kLast of 8 values,
// 8 to a row.
template <int kBoxes, int kThreads, int kFirst, int kLast>
__device__ __forceinline__ void weigh(unsigned char* y, unsigned char* z, unsigned char* to, int thread,
                                      int n, const float* late, float by) {
#pragma unroll 2
  for (int i = kFirst + thread; i < kLast; i += kThreads) {
    const int row = i >> 3;
    const unsigned at = (unsigned)row * 128u + ((unsigned)((i ^ row) & 7) << 4);
    uint4 part[kParts] = {};
    if (row < n) {
      const uint4 v = *reinterpret_cast<const uint4*>(z + at);
      const Vec<2> w = ops::fill<2>(late[row] * by);
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        Vec<2> f = ops::mul({{bf16_lo(in[e]), bf16_hi(in[e])}}, w);
#pragma unroll
        for (int k = 0; k < kParts; ++k) (&part[k].x)[e] = take(f);
      }
    } else {
      *reinterpret_cast<uint4*>(z + at) = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < kBoxes; ++k) *reinterpret_cast<uint4*>(y + k * kTile + at) = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k) *reinterpret_cast<uint4*>(to + k * kTile + at) = part[k];
  }
}

// add: D = Y^T Z' over a chunk, the first part in columns 0-63, the others' sum in 64-127.  With one box of Y
// rows 64 and up are rows 0 and up again (y's lbo = 0).
__device__ __forceinline__ void issue_add(unsigned d, uint64_t y, uint64_t parts) {
#pragma unroll
  for (int s = 0; s < kChunk / 16; ++s)
    mma(d, y + s * 2048 / 16, parts + s * 2048 / 16, instruction(2 * kD, true, true), s > 0);
#pragma unroll
  for (int s = 0; s < kChunk / 16; ++s)
    mma(d + kD, y + s * 2048 / 16, parts + (2 * kTile + s * 2048) / 16, instruction(kD, true, true),
        true);
}
constexpr unsigned kAddColumns = 2 * kD;
// A thread's part of the state: the row of its tensor-memory lane, all 64 columns of it, or with 64 rows, which
// the lanes hold twice, half of them.
template <int kBoxes>
struct Place {
  static constexpr int kCols = 32 * kBoxes;
  int row, col;
  __device__ __forceinline__ explicit Place(int lane)
      : row(kBoxes == 2 ? lane : lane & 63), col(kBoxes == 2 ? 0 : (lane >> 6) * 32) {}
};
// Calls use(16 columns at a time: which, both sums' sums in pairs) for kCols columns.
template <int kCols, class Use>
__device__ __forceinline__ void each_add(unsigned addr, Use use) {
#pragma unroll
  for (int q = 0; q < kCols / 16; ++q) {
    unsigned d[2][16];
    tmem_load16(addr + 16 * q, d[0]);
    tmem_load16(addr + kD + 16 * q, d[1]);
    tmem_loaded();
    Vec<2> sum[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      sum[c] = ops::add({{__uint_as_float(d[0][2 * c]), __uint_as_float(d[0][2 * c + 1])}},
                        {{__uint_as_float(d[1][2 * c]), __uint_as_float(d[1][2 * c + 1])}});
    use(q, sum);
  }
}

// ---- outputs ----------------------------------------------------------------------------

constexpr int kOutWarps = 16, kOutThreads = 32 * kOutWarps;
constexpr int kStateWarp = 8, kWeighWarp = 12, kIssueWarp = 15;
// Pieces of Z' that the warps from kWeighWarp on weigh; the state's warps weigh the rest, after the state.
constexpr int kWeighPieces = 640;

// Decays from a column of a block of 32 scores to a row, in processing order: within a block on the
// diagonal, near[31 + row - column], zero for columns after the row; in others g^(row - last column),
// times far[column].  (Last: of the block, in processing order; the order may be against the columns'.)
// late[row]: from a whole chunk's token to its end, times zs; of n tokens, late + 128 - n (late, against the
// order).
struct Decays {
  float far[32];
  float near[64];
  float late[kChunk];
  __device__ __forceinline__ void fill(float log2g, int reverse, float zs, int i) {   // i < kChunk
    if (i < 32) far[i] = power(log2g, reverse ? i : 31 - i);
    const int back = (i - 31) * (reverse ? -1 : 1);
    if (i < 64) near[i] = back >= 0 && i < 63 ? power(log2g, back) : 0.f;
    late[i] = zs * power(log2g, reverse ? i : kChunk - 1 - i);
  }
  __device__ __forceinline__ const float* late_of(int n, int reverse) const {
    return reverse ? late : late + kChunk - n;
  }
};

template <int kBoxes, bool kExact>
struct OutLayout {
  static constexpr int kStages = stages_of(kBoxes, kExact);
  static constexpr unsigned kStage = (2 * kBoxes + 1) * kTile;   // X, Y and Z
  static constexpr unsigned kState = kBoxes * kD * kD * 2;       // a part of S
  unsigned stage, parts, state, staging, decays, bars, total;
  __host__ __device__ OutLayout() {
    stage = 0;
    parts = kStages * kStage;
    state = parts + kStages * kParts * kTile;
    staging = state + parts_of(kExact) * kState;
    decays = staging + 8 * 2048;
    bars = decays + sizeof(Decays);
    total = bars + 8 * 32;
  }
};
enum Bar {
  kFull = 0, kScoresFull = kFull + 2, kPReady = kScoresFull + 2,
  kZReady = kPReady + 2, kOFull = kZReady + 2, kOFree, kAddFull, kAddFree,
  kSReady, kSFree, kDone, kBars
};
static_assert(kBars < 32, "room of the barriers");

template <int kBoxes, bool kExact>
__global__ void __launch_bounds__(kOutThreads, 1)
decay_chunks_kernel(const __grid_constant__ TcArgs t) {
  using Layout = OutLayout<kBoxes, kExact>;
  constexpr int kStages = Layout::kStages, kOutParts = parts_of(kExact);
  // P's third part lies over the other tile of scores, whose product waits for the next chunk's copies and
  // they for the end of what reads that part.
  static_assert(kOutParts == 2 || kStages == 1, "where P's third part is read, no scores are written");
  constexpr unsigned kStage = Layout::kStage, kState = Layout::kState;
  extern __shared__ unsigned char smem_raw[];
  const Args& a = t.a;
  const int which = blockIdx.z, col0 = blockIdx.y * kD;
  const Pass& p = a.pass[which];
  if (col0 >= p.b) return;   // (a pass with fewer columns than the launch's widest)
  const int bh = blockIdx.x / a.segments, segment = blockIdx.x % a.segments;
  const int lane = threadIdx.x & 31;
  // The products are issued beside the warps of the rows with the fewest scores: a scheduler's other warps
  // hold the issuing one up.
  int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  if (warp >= kWeighWarp && !p.reverse) warp = warp == kWeighWarp ? kIssueWarp : warp - 1;
  const Chunks chunks(a, p, bh, segment);
  const int n = chunks.count;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const Layout at;
  Decays& decays = *reinterpret_cast<Decays*>(smem + at.decays);
  const unsigned bars = smem_u32(smem + at.bars);
  auto bar = [&](int b) { return bars + 8u * (unsigned)b; };
  unsigned* slot = reinterpret_cast<unsigned*>(smem + at.bars + 8 * kBars);
  const float l = log_decay(a, bh), l2 = l * kLog2e;

  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kFull + s), 1);
      mbar_init(bar(kScoresFull + s), 1);
      mbar_init(bar(kPReady + s), 8);
      mbar_init(bar(kZReady + s), kIssueWarp - kStateWarp);
    }
    mbar_init(bar(kOFull), 1);
    mbar_init(bar(kOFree), 8);
    mbar_init(bar(kAddFull), 1);
    mbar_init(bar(kAddFree), 4);
    mbar_init(bar(kSReady), 4);
    mbar_init(bar(kSFree), 1);
    mbar_init(bar(kDone), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x >= 128 && threadIdx.x < 128 + kChunk)
    decays.fill(l2, p.reverse, p.zs, threadIdx.x - 128);
  fence_before();
  __syncthreads();
  fence_after();
  const unsigned tmem = *slot;
  bool ok = true;
  const unsigned long long wait_ns = t.wait_ns;

  // A chunk's stage, and the parity of its phase.
  auto stage_of = [](int i) { return kStages == 2 ? i & 1 : 0; };
  auto phase_of = [](int i) { return kStages == 2 ? (i >> 1) & 1 : i & 1; };
  // The copies of chunk i, by one lane of a warp; the chunks after the next are on their way into L2.
  auto copy = [&](int i, bool leader) {
    if (i >= n || (t.skip_last && i == n - 1)) return;   // (fault injection: never copied)
    if (leader) {
      const unsigned dst = smem_u32(smem + at.stage + stage_of(i) * kStage), full = bar(kFull + stage_of(i));
      const int token = chunks.place(i) * kChunk;
      mbar_expect_tx(full, kStage);
#pragma unroll
      for (int k = 0; k < kBoxes; ++k) {
        tma_load_3d(dst + k * kTile, &t.x[which], k * kD, token, bh, full);
        tma_load_3d(dst + (kBoxes + k) * kTile, &t.y[which], k * kD, token, bh, full);
      }
      tma_load_3d(dst + 2 * kBoxes * kTile, &t.z[which], col0, token, bh, full);
      if (i + kAhead < n) {
        const int later = chunks.place(i + kAhead) * kChunk;
#pragma unroll
        for (int k = 0; k < kBoxes; ++k) {
          tma_prefetch_3d(&t.x[which], k * kD, later, bh);
          tma_prefetch_3d(&t.y[which], k * kD, later, bh);
        }
        tma_prefetch_3d(&t.z[which], col0, later, bh);
      }
    }
  };
  // Z' of chunk i, by the warps from kStateWarp on.
  auto weigh_chunk = [&](int i) {
    const int b = stage_of(i);
    if (!warp_wait(bar(kFull + b), phase_of(i), wait_ns)) return false;
    // (All that read the Z' before in this place is done: what was copied for this one waited for it.)
    const int tokens = chunks.tokens(i);
    unsigned char* y = smem + at.stage + b * kStage + kBoxes * kTile;
    unsigned char* z = y + kBoxes * kTile;
    unsigned char* to = smem + at.parts + b * kParts * kTile;
    const float* late = decays.late_of(tokens, p.reverse);
    if (warp < kWeighWarp)
      weigh<kBoxes, 32 * (kWeighWarp - kStateWarp), kWeighPieces, kPieces>(
          y, z, to, threadIdx.x - 32 * kStateWarp, tokens, late, 1.f);
    else
      weigh<kBoxes, 32 * (kIssueWarp - kWeighWarp), 0, kWeighPieces>(
          y, z, to, 32 * (warp - kWeighWarp) + lane, tokens, late, 1.f);
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kZReady + b));
    return true;
  };

  if (warp < 8) {
    // ---------------- P and outputs ----------------
    const int quad = warp & 3, odd = warp >> 2;
    const unsigned lanes = (unsigned)(32 * quad) << 16;
    const int row = 32 * quad + lane;
    const float f = p.zs * p.os;
    const bool half = p.out_half;
    unsigned char* staging = smem + at.staging + warp * 2048;
    auto scores_to_p = [&](int i) {
      if (!warp_wait(bar(kScoresFull + (i & 1)), (i >> 1) & 1, wait_ns)) return false;
      fence_after();
      const unsigned base = tmem + kScores + 128u * (i & 1) + lanes;
      const unsigned third = tmem + kScores + 128u * ((i + 1) & 1) + lanes;
      const int tokens = chunks.tokens(i);
#pragma unroll 1
      for (int j = odd; j < 4; j += 2) {    // blocks of 32 columns
        unsigned part[kOutParts][16];
        const bool none = p.reverse ? j < quad : j > quad;
        if (none || 32 * j >= tokens) {
#pragma unroll
          for (int k = 0; k < kOutParts; ++k)
#pragma unroll
            for (int e = 0; e < 16; ++e) part[k][e] = 0u;
        } else {
          unsigned s[32];
          tmem_load32(base + 32 * j, s);
          Vec<2> v[16];
          if (j == quad) {
            const float* near = decays.near + 31 + lane;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = ops::mul({{near[-2 * e], near[-2 * e - 1]}}, ops::fill<2>(f));
          } else {
            const float g = f * power(l2, p.reverse ? 32 * j - row : row - (32 * j + 31));
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float4 w = *reinterpret_cast<const float4*>(decays.far + 2 * e);
              v[e] = ops::mul({{w.x, w.y}}, ops::fill<2>(g));
              v[e + 1] = ops::mul({{w.z, w.w}}, ops::fill<2>(g));
            }
          }
          tmem_loaded();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = ops::mul(v[e], {{__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])}});
          if (32 * j + 32 > tokens) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (32 * j + 2 * e >= tokens) v[e].f[0] = 0.f;
              if (32 * j + 2 * e + 1 >= tokens) v[e].f[1] = 0.f;
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
#pragma unroll
            for (int k = 0; k < kOutParts - 1; ++k) part[k][e] = take(v[e]);
            part[kOutParts - 1][e] = ops::pack_bf16(v[e].f[0], v[e].f[1]);
          }
        }
        tmem_store16(base + 32 * j, part[0]);
        tmem_store16(base + 32 * j + 16, part[1]);
        if constexpr (kExact) tmem_store16(third + 16 * j, part[2]);
      }
      tmem_stored();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kPReady + (i & 1)));
      return true;
    };
    // Outputs go through shared memory, 64 bytes of a row at a time (32 columns in bf16, or 16), to 8 rows at
    // once.
    const int piece = lane & 3, row0 = lane >> 2;
    auto stage = [&](const Vec<2>* o) {   // 32 bf16 columns, or 16
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          (&v.x)[e] = half ? ops::pack_bf16(o[4 * c + e].f[0], o[4 * c + e].f[1])
                           : __float_as_uint(o[2 * c + (e >> 1)].f[e & 1]);
        *reinterpret_cast<uint4*>(staging + (lane * 4 + (c ^ ((lane >> 1) & 3))) * 16) = v;
      }
      __syncwarp();
    };
    auto flush = [&](int i, int col) {
      const long long first = (long long)bh * a.tokens;
      const int size = half ? 2 : 4, token0 = chunks.place(i) * kChunk + 32 * quad;
      col += col0 + piece * (16 / size);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = row0 + 8 * k, token = token0 + r;
        const uint4 v =
            *reinterpret_cast<const uint4*>(staging + (r * 4 + (piece ^ ((r >> 1) & 3))) * 16);
        if (token < a.tokens && col < p.b)
          *reinterpret_cast<uint4*>(static_cast<char*>(p.out) + ((first + token) * p.b + col) * size) = v;
      }
      __syncwarp();
    };
    auto outputs = [&](int i) {
      if (!warp_wait(bar(kOFull), i & 1, wait_ns)) return false;
      fence_after();
      // All that reads the chunk's stage is done: the copies of the one after the next take it.
      if (warp == 0 && i + kStages < n) copy(i + kStages, elect());
      unsigned inner[32], outer[32];
      tmem_load32(tmem + kInner + 32 * odd + lanes, inner);
      tmem_load32(tmem + kOuter + 32 * odd + lanes, outer);
      const int tokens = chunks.tokens(i);
      const bool undecayed = p.undecayed && chunks.first + i == 0;
      const int steps = (p.reverse ? tokens - row : row + 1) - undecayed;
      const bool live = row < tokens;
      const Vec<2> g = ops::fill<2>(live ? p.os * power(l2, steps) : 0.f);
      tmem_loaded();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOFree));
      Vec<2> o[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        o[e] = ops::fma({{__uint_as_float(outer[2 * e]), __uint_as_float(outer[2 * e + 1])}}, g,
                        {{__uint_as_float(inner[2 * e]), __uint_as_float(inner[2 * e + 1])}});
        if (!live) o[e] = ops::fill<2>(0.f);
      }
      stage(o);
      if (!half) {
        flush(i, 32 * odd);
        stage(o + 8);
        flush(i, 32 * odd + 16);
      }
      return true;
    };
    // (bf16 rows leave shared memory after the next chunk's P, on which the products wait.)
    if (warp == 0)
      for (int i = 0; i < min(n, kStages); ++i) copy(i, elect());
    int done = 0;
    for (int i = 0; i < n && ok; ++i) {
      ok = scores_to_p(i);
      if (!ok) break;
      if (half && i > 0) flush(i - 1, 32 * odd);
      ok = outputs(i);
      if (ok) done = i + 1;
    }
    // Every copy lands before the CTA may finish: those of the chunks not done, made so far.
    if (!ok && warp == 0)
      for (int i = done; i < min(n, done + kStages); ++i)
        mbar_wait(bar(kFull + stage_of(i)), phase_of(i), wait_ns);
    if (half && ok && n > 0) flush(n - 1, 32 * odd);
  } else if (warp < 12) {
    // ---------------- the state ----------------
    const int tl = threadIdx.x - 256;
    using Mine = Place<kBoxes>;
    constexpr int kCols = Mine::kCols;
    const Mine place(tl);
    const int col = col0 + place.col;   // of the pass
    const unsigned lanes = (unsigned)(32 * (warp & 3)) << 16;
    Vec<2> S[kCols / 2];
    const float* from = nullptr;
    long long row_step = p.b, col_step = 1;
    if (p.states) await_last();   // the states before each segment are there
    if (p.states) {
      from = p.states + ((long long)bh * a.segments + segment) * p.a * p.b;
    } else if (p.first) {
      from = p.first + (long long)bh * p.a * p.b;
      if (p.first_across) row_step = 1, col_step = p.a;
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      S[c / 2].f[c & 1] = 0.f;
      if (from && place.row < p.a && col + c < p.b)
        S[c / 2].f[c & 1] = from[place.row * row_step + (col + c) * col_step];
    }
    unsigned char* operand_at = smem + at.state + place.row * 128;
    auto publish = [&] {
#pragma unroll
      for (int c = 0; c < kCols / 8; ++c) {
        uint4 part[kOutParts];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          Vec<2> v = S[4 * c + e];
#pragma unroll
          for (int k = 0; k < kOutParts - 1; ++k) (&part[k].x)[e] = take(v);
          (&part[kOutParts - 1].x)[e] = ops::pack_bf16(v.f[0], v.f[1]);
        }
        const unsigned piece = (unsigned)((place.col / 8 + c) ^ (place.row & 7)) << 4;
#pragma unroll
        for (int k = 0; k < kOutParts; ++k)
          *reinterpret_cast<uint4*>(operand_at + k * kState + piece) = part[k];
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSReady));
    };
    if (n > 0) {
      publish();
      ok = weigh_chunk(0);
    }
    for (int i = 0; i < n && ok; ++i) {
      ok = warp_wait(bar(kAddFull), i & 1, wait_ns);
      if (!ok) break;
      fence_after();
      const Fade fade(l, chunks.tokens(i) - (p.undecayed && chunks.first + i == 0));
      each_add<kCols>(tmem + kAdd + place.col + lanes, [&](int q, const Vec<2> (&add)[8]) {
#pragma unroll
        for (int c = 0; c < 8; ++c) S[8 * q + c] = ops::add(fade(S[8 * q + c]), add[c]);
      });
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kAddFree));
      if (i + 1 < n) {
        ok = warp_wait(bar(kSFree), i & 1, wait_ns);
        if (!ok) break;
        publish();
        ok = weigh_chunk(i + 1);
      }
    }
    if (ok && p.last && segment == a.segments - 1) {
      const float g = p.undecayed && chunks.len > 0 ? exp2f(l2) : 1.f;
      float* to = p.last + (long long)bh * p.a * p.b + (long long)place.row * p.b + col;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        if (place.row < p.a && col + c < p.b) to[c] = S[c / 2].f[c & 1] * g;
    }
  } else if (warp < kIssueWarp) {
    // ---------------- Z' ----------------
    for (int i = 0; i < n && ok; ++i) ok = weigh_chunk(i);
  } else {
    // ---------------- products ----------------
    const bool leader = elect();
    const unsigned stage0 = smem_u32(smem + at.stage);
    // k-th 16 values of rows of X or Y.
    auto step = [](int k) { return (uint64_t)((k / 4) * (kTile / 16) + 2 * (k % 4)); };
    auto scores = [&](int i) {
      if (!warp_wait(bar(kFull + stage_of(i)), phase_of(i), wait_ns)) return false;
      fence_after();
      if (leader) {
        const uint64_t x = operand(stage0 + stage_of(i) * kStage, 0);
#pragma unroll
        for (int s = 0; s < kBoxes * kD / 16; ++s)
          mma(tmem + kScores + 128u * (i & 1), x + step(s), x + kBoxes * (kTile / 16) + step(s),
              instruction(kChunk, false, false), s > 0);
        commit(bar(kScoresFull + (i & 1)));
      }
      return true;
    };
    const uint64_t state = operand(smem_u32(smem + at.state), 0);
    if (n > 0) ok = scores(0);
    for (int i = 0; i < n && ok; ++i) {
      const unsigned at_x = stage0 + stage_of(i) * kStage;
      const uint64_t x = operand(at_x, 0), z = x + 2 * kBoxes * (kTile / 16);
      const uint64_t y = operand(at_x + kBoxes * kTile, kBoxes == 2 ? kTile : 0);
      ok = warp_wait(bar(kZReady + stage_of(i)), phase_of(i), wait_ns) &&
           (i == 0 || warp_wait(bar(kAddFree), (i - 1) & 1, wait_ns));
      if (!ok) break;
      fence_after();
      if (leader) {
        issue_add(tmem + kAdd, y,
                  operand(smem_u32(smem + at.parts + stage_of(i) * kParts * kTile), kTile));
        commit(bar(kAddFull));
      }
      ok = warp_wait(bar(kSReady), i & 1, wait_ns) &&
           (i == 0 || warp_wait(bar(kOFree), (i - 1) & 1, wait_ns));
      if (!ok) break;
      fence_after();
      if (leader) {
#pragma unroll
        for (int k = kOutParts - 1; k >= 0; --k)   // (small parts first: what is added to later is cut off)
#pragma unroll
          for (int s = 0; s < kBoxes * kD / 16; ++s)
            mma(tmem + kOuter, x + step(s), state + (k * kState + s * 2048) / 16,
                instruction(kD, false, true), k < kOutParts - 1 || s > 0);
        commit(bar(kSFree));
      }
      ok = warp_wait(bar(kPReady + (i & 1)), (i >> 1) & 1, wait_ns);
      if (!ok) break;
      fence_after();
      if (leader) {
#pragma unroll
        for (int k = kOutParts - 1; k >= 0; --k)
#pragma unroll
          for (int s = 0; s < kChunk / 16; ++s) {
            const unsigned p_at = k < 2 ? 128u * (i & 1) + 32 * (s / 2) + 16 * k + 8 * (s & 1)
                                        : 128u * ((i + 1) & 1) + 8 * s;
            mma_tmem(tmem + kInner, tmem + kScores + p_at, z + s * 2048 / 16, instruction(kD, false, true),
                     k < kOutParts - 1 || s > 0);
          }
        commit(bar(kOFull));
      }
      // The next chunk's scores, whose tile of P the last chunk's product has read: kOFree told.
      ok = i + 1 == n || scores(i + 1);
    }
    if (leader) commit(bar(kDone));
  }

  // Agree on failures; then whatever the tensor core still does ends before its memory goes.
  ok = __syncthreads_and(ok ? 1 : 0) != 0;
  if (threadIdx.x == 0) {
    if (!mbar_wait(bar(kDone), 0, wait_ns)) ok = false;
    if (!ok) atomicOr(t.err, kErrBitDecay);
  }
  fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kColumns)
                 : "memory");
  }
  // Zeros for the chunks that are all padding.
  if (col0 == 0) {
    const long long row0 = (long long)bh * a.tokens;
    const int begin = max(segment * a.per_segment, chunks.all * kChunk);
    const int end = min((segment + 1) * a.per_segment, a.tokens);
    const int piece = p.out_half ? 8 : 4;
    uint4* out = static_cast<uint4*>(p.out);
    for (long long i = (row0 + begin) * (p.b / piece) + threadIdx.x; i < (row0 + end) * (p.b / piece);
         i += kOutThreads)
      out[i] = make_uint4(0, 0, 0, 0);
  }
}

// ---- segments' own states ------------------------------------------------------------------

constexpr int kSumWarps = 14, kSumThreads = 32 * kSumWarps;

template <int kBoxes>
struct SumLayout {
  static constexpr int kStages = kBoxes == 1 ? 4 : 2;
  static constexpr unsigned kStage = (kBoxes + 1) * kTile;   // Y and Z
  unsigned stage, parts, late, bars, total;
  __host__ __device__ SumLayout() {
    stage = 0;
    parts = kStages * kStage;
    late = parts + 2 * kParts * kTile;
    bars = late + kChunk * 4;
    total = bars + 8 * 32;
  }
};
enum SumBar {
  kSumFull = 0, kSumEmpty = kSumFull + 4, kSumReady = kSumEmpty + 4,
  kSumDone = kSumReady + 2, kSumFree = kSumDone + 2, kSumEnd = kSumFree + 2, kSumBars
};
static_assert(kSumBars < 32, "room of the barriers");

// Sum over a segment's tokens of y z^T with their decays to the segment's end.  Warps 0-7: Z'; 8-11: sums
// in registers (in tensor memory, whose adding cuts off, a chunk's products only); 12 copies, 13 issues.
template <int kBoxes>
__global__ void __launch_bounds__(kSumThreads, 1)
decay_sums_kernel(const __grid_constant__ TcArgs t) {
  using Layout = SumLayout<kBoxes>;
  constexpr int kSumStages = Layout::kStages;
  constexpr unsigned kStage = Layout::kStage;
  extern __shared__ unsigned char smem_raw[];
  const Args& a = t.a;
  const int which = blockIdx.z, col0 = blockIdx.y * kD;
  const Pass& p = a.pass[which];
  release_next();
  if (col0 >= p.b) return;   // (a pass with fewer columns than the launch's widest)
  const int bh = blockIdx.x / (a.segments - 1), segment = blockIdx.x % (a.segments - 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Chunks chunks(a, p, bh, segment);
  const int n = chunks.count;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const Layout at;
  const unsigned bars = smem_u32(smem + at.bars);
  auto bar = [&](int b) { return bars + 8u * (unsigned)b; };
  unsigned* slot = reinterpret_cast<unsigned*>(smem + at.bars + 8 * kSumBars);
  const float l2 = log_decay(a, bh) * kLog2e;
  constexpr unsigned kSumColumns = 2 * kAddColumns;

  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(kSumColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSumStages; ++s) {
      mbar_init(bar(kSumFull + s), 1);
      mbar_init(bar(kSumEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kSumReady + s), 8);
      mbar_init(bar(kSumDone + s), 1);
      mbar_init(bar(kSumFree + s), 4);
    }
    mbar_init(bar(kSumEnd), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  float* late = reinterpret_cast<float*>(smem + at.late);
  if (threadIdx.x >= 128 && threadIdx.x < 128 + kChunk) {
    const int i = threadIdx.x - 128;
    late[i] = p.zs * power(l2, p.reverse ? i : kChunk - 1 - i);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const unsigned tmem = *slot;
  bool ok = true;
  const unsigned long long wait_ns = t.wait_ns;

  if (warp < 8) {
    // Decays to the segment's end: to the chunk's, times those of the tokens after it.
    int after = 0;
    for (int i = 0; i < n; ++i) after += chunks.tokens(i);
    Ring ring;
    for (int i = 0; i < n; ++i, ring.next(kSumStages)) {
      const int tokens = chunks.tokens(i);
      after -= tokens;
      ok = warp_wait(bar(kSumFull + ring.stage), ring.phase, wait_ns);
      if (ok && i > 1) ok = warp_wait(bar(kSumDone + (i & 1)), ((i >> 1) - 1) & 1, wait_ns);
      if (!ok) break;
      unsigned char* y = smem + at.stage + ring.stage * kStage;
      weigh<kBoxes, 256, 0, kPieces>(
          y, y + kBoxes * kTile, smem + at.parts + (i & 1) * kParts * kTile, threadIdx.x, tokens,
                 p.reverse ? late : late + kChunk - tokens, power(l2, after));
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSumReady + (i & 1)));
    }
  } else if (warp < 12) {
    using Mine = Place<kBoxes>;
    constexpr int kCols = Mine::kCols;
    const Mine place(threadIdx.x - 256);
    const int col = col0 + place.col;   // of the pass
    const unsigned lanes = (unsigned)(32 * (warp & 3)) << 16;
    Vec<2> S[kCols / 2];
#pragma unroll
    for (int c = 0; c < kCols / 2; ++c) S[c] = ops::fill<2>(0.f);
    for (int i = 0; i < n; ++i) {
      ok = warp_wait(bar(kSumDone + (i & 1)), (i >> 1) & 1, wait_ns);
      if (!ok) break;
      fence_after();
      each_add<kCols>(tmem + kAddColumns * (i & 1) + place.col + lanes,
                      [&](int q, const Vec<2> (&add)[8]) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) S[8 * q + c] = ops::add(S[8 * q + c], add[c]);
                      });
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSumFree + (i & 1)));
    }
    float* to = p.states + (((long long)bh * a.segments + segment) * p.a + place.row) * p.b + col;
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      if (place.row < p.a && col + c < p.b) to[c] = S[c / 2].f[c & 1];
  } else if (warp == 12) {
    const bool leader = elect();
    int issued = 0;
    for (int i = 0; i < n; ++i) {
      const int s = i % kSumStages;
      if (t.skip_last && i == n - 1) break;   // (fault injection: never copied)
      if (i >= kSumStages) ok = warp_wait(bar(kSumEmpty + s), ((i / kSumStages) - 1) & 1, wait_ns);
      if (!ok) break;
      const unsigned dst = smem_u32(smem + at.stage + s * kStage);
      const int token = chunks.place(i) * kChunk;
      if (leader) {
        mbar_expect_tx(bar(kSumFull + s), kStage);
#pragma unroll
        for (int k = 0; k < kBoxes; ++k)
          tma_load_3d(dst + k * kTile, &t.y[which], k * kD, token, bh, bar(kSumFull + s));
        tma_load_3d(dst + kBoxes * kTile, &t.z[which], col0, token, bh, bar(kSumFull + s));
      }
      issued = i + 1;
    }
    for (int i = max(0, issued - kSumStages); i < issued; ++i)
      mbar_wait(bar(kSumFull + i % kSumStages), (i / kSumStages) & 1, wait_ns);
  } else {
    const bool leader = elect();
    for (int i = 0; i < n; ++i) {
      ok = warp_wait(bar(kSumReady + (i & 1)), (i >> 1) & 1, wait_ns) &&
           (i < 2 || warp_wait(bar(kSumFree + (i & 1)), ((i >> 1) - 1) & 1, wait_ns));
      if (!ok) break;
      fence_after();
      if (leader) {
        issue_add(tmem + kAddColumns * (i & 1),
                  operand(smem_u32(smem + at.stage + (i % kSumStages) * kStage), kBoxes == 2 ? kTile : 0),
                  operand(smem_u32(smem + at.parts + (i & 1) * kParts * kTile), kTile));
        commit(bar(kSumDone + (i & 1)));
        commit(bar(kSumEmpty + i % kSumStages));
      }
    }
    if (leader) commit(bar(kSumEnd));
  }

  ok = __syncthreads_and(ok ? 1 : 0) != 0;
  if (threadIdx.x == 0) {
    if (!mbar_wait(bar(kSumEnd), 0, wait_ns)) ok = false;
    if (!ok) atomicOr(t.err, kErrBitDecay);
  }
  fence_before();
  __syncthreads();
  if (warp == 13) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kSumColumns)
                 : "memory");
  }
}

constexpr unsigned kSmemMost = 227 * 1024;
static_assert(sizeof(Decays) == 896, "room of the decays");

bool encode(CUtensorMap* map, const void* base, int width, int tokens, int bh) {
  return tma_encode_3d_sw128(map, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)width,
                             (uint64_t)tokens, (uint64_t)bh, (uint64_t)width * 2,
                             (uint64_t)tokens * width * 2, kD, kChunk);
}

}  // namespace

bool tc_fits(const Args& a, int passes) {
  for (int i = 0; i < passes; ++i) {
    const Pass& p = a.pass[i];
    if (!p.x_half || !p.y_half || !p.z_half || p.a > 2 * kD || p.b > 2 * kD || p.a % 8 || p.b % 8) return false;
    for (const void* q : {p.x, p.y, p.z, static_cast<const void*>(p.out)})
      if (!ops::aligned(q, 16)) return false;
  }
  return true;
}

namespace {

template <int kBoxes, bool kExact>
cudaError_t launch_boxes(const TcArgs& t, int passes, int bh, int tiles, cudaStream_t st) {
  const Args& a = t.a;
  using Out = OutLayout<kBoxes, kExact>;
  const unsigned sums = SumLayout<kBoxes>().total + 1024, outs = Out().total + 1024;
  static_assert(Out::kStages * (Out::kStage + kParts * kTile) + parts_of(kExact) * Out::kState + 8 * 2048 +
                        896 + 256 + 1024 <= kSmemMost,
                "shared memory of the outputs' kernel");
  cudaError_t e = cudaSuccess;
  if (a.segments > 1) {
    e = cudaFuncSetAttribute(decay_sums_kernel<kBoxes>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemMost);
    if (e != cudaSuccess) return e;
    e = launch(decay_sums_kernel<kBoxes>,
               dim3((unsigned)(bh * (a.segments - 1)), (unsigned)tiles, (unsigned)passes), kSumThreads, sums,
               false, st, t);
    if (e == cudaSuccess) e = launch_carry(a, passes, bh, st);
    if (e != cudaSuccess) return e;
  }
  e = cudaFuncSetAttribute(decay_chunks_kernel<kBoxes, kExact>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemMost);
  if (e != cudaSuccess) return e;
  return launch(decay_chunks_kernel<kBoxes, kExact>,
                dim3((unsigned)(bh * a.segments), (unsigned)tiles, (unsigned)passes), kOutThreads, outs,
                a.segments > 1, st, t);
}

}  // namespace

cudaError_t launch_tc(const Args& a, int passes, int bh, unsigned* err, unsigned long long wait_ns,
                      int skip_last, cudaStream_t st) {
  TcArgs t;
  t.a = a;
  t.err = err;
  t.wait_ns = wait_ns;
  t.skip_last = skip_last;
  int rows = 0, cols = 0;
  bool exact = false;
  for (int i = 0; i < passes; ++i) {
    const Pass& p = a.pass[i];
    exact = exact || !p.out_half;
    rows = std::max(rows, p.a);
    cols = std::max(cols, p.b);
    if (!encode(&t.x[i], p.x, p.a, a.tokens, bh) || !encode(&t.y[i], p.y, p.a, a.tokens, bh) ||
        !encode(&t.z[i], p.z, p.b, a.tokens, bh))
      return cudaErrorInvalidValue;
  }
  const int tiles = (cols + kD - 1) / kD;
  if (exact)
    return rows <= kD ? launch_boxes<1, true>(t, passes, bh, tiles, st)
                      : launch_boxes<2, true>(t, passes, bh, tiles, st);
  return rows <= kD ? launch_boxes<1, false>(t, passes, bh, tiles, st)
                    : launch_boxes<2, false>(t, passes, bh, tiles, st);
}

}  // namespace decay
}  // namespace lapl
