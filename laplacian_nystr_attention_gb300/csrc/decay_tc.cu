// decay_tc.cu -- a pass of the linear attention with decays in chunks of 128 tokens on the tensor
// cores (decay.cuh has the formulas): bf16 rows of up to 64 values.
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
// x, y and z enter as they are.  What is computed is split into bf16 parts, so that no product loses
// what fp32 holds: P and S into two (2^-17 of a value is left out, against 2^-9 of the output's own
// rounding), Z' into three (2^-25), as the state's errors are carried along.
//
// One CTA of an SM works through a segment of a sequence; its warps:
//   0-7    scores to P (warp w: rows 32 (w % 4) and up, every other block of 32 columns), and the
//          outputs: both accumulators, the decays, through shared memory to whole runs of rows
//   8-11   the state, fp32 in registers: g^n S + add, and its two parts as an operand
//   12-15  Z' from Z
//   16     copies: X, Y and Z tiles by TMA, 128-byte swizzle, up to 3 chunks ahead
//   17     one thread issues the products
// Before it, where a sequence has several segments: decay_sums_kernel forms each segment's own
// contribution to the state (add, with decays to the segment's end) and decay_carry_kernel the states
// before each.
#include <algorithm>

#include "decay_tc.cuh"

namespace lapl {
namespace decay {
namespace {

using namespace tc;
using ops::Vec;

constexpr int kChunk = kTcChunk;
constexpr int kD = 64;                        // padded row length
constexpr unsigned kTile = kChunk * kD * 2;   // bytes of a tile of X, Y, Z or a part of Z'
constexpr unsigned kState = kD * kD * 2;      // bytes of a part of S
constexpr int kParts = 3;                     // of Z'
constexpr int kMaxStages = 4;
constexpr int kPowers = 32;

// Columns of tensor memory.
constexpr unsigned kScores = 0, kInner = 256, kOuter = 320, kAdd = 384, kColumns = 512;

struct TcArgs {
  Args a;
  CUtensorMap x[kMaxPasses], y[kMaxPasses], z[kMaxPasses];
  unsigned* err;
  unsigned long long wait_ns;
  int skip_last;
  int stages;
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

// The tokens of Z, times weight(row), as kParts tiles; rows from n on as zeros, in Z and Y too, whose
// products with zeros would not be zeros for what is not finite there.  A thread has 16 / kShare pieces
// of 8 values of a row of 64.
template <int kShare, class Weight>
__device__ __forceinline__ void weigh(unsigned char* y, unsigned char* z, unsigned char* to, int row,
                                      int share, int n, Weight weight) {
  const float w = weight(row);
  const Vec<2> w2 = ops::fill<2>(w);
  const unsigned at = (unsigned)row * 128u;
#pragma unroll
  for (int c = 0; c < 8 / kShare; ++c) {
    const unsigned piece = at + ((unsigned)((share * (8 / kShare) + c) ^ (row & 7)) << 4);
    uint4 part[kParts] = {};
    if (row < n) {
      const uint4 v = *reinterpret_cast<const uint4*>(z + piece);
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        Vec<2> f = ops::mul({{bf16_lo(in[e]), bf16_hi(in[e])}}, w2);
#pragma unroll
        for (int k = 0; k < kParts; ++k) (&part[k].x)[e] = take(f);
      }
    } else {
      *reinterpret_cast<uint4*>(z + piece) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(y + piece) = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k) *reinterpret_cast<uint4*>(to + k * kTile + piece) = part[k];
  }
}

// add: D = Y^T Z' over a chunk; rows 64 and up of D are rows 0 and up again (lbo = 0).
__device__ __forceinline__ void issue_add(unsigned d, unsigned y, unsigned parts) {
#pragma unroll
  for (int k = 0; k < kParts; ++k)
#pragma unroll
    for (int s = 0; s < kChunk / 16; ++s)
      mma(d, operand(y + s * 2048, 0), operand(parts + k * kTile + s * 2048, 0),
          instruction(kD, true, true), k > 0 || s > 0);
}

// A state's values of tensor-memory lane `lane`: row lane % 64, columns from 32 (lane / 64) on.
struct Place64 {
  int row, col;
  __device__ __forceinline__ explicit Place64(int lane) : row(lane & 63), col((lane >> 6) * 32) {}
};

// ---- outputs ----------------------------------------------------------------------------

constexpr int kOutWarps = 18, kOutThreads = 32 * kOutWarps;
constexpr int kCopyWarp = 16, kIssueWarp = 17;

struct OutLayout {
  unsigned stage, parts, state, staging, powers, bars, total;
  __host__ __device__ OutLayout(int stages, bool out_half) {
    stage = 0;
    parts = stages * 3 * kTile;
    state = parts + kParts * kTile;
    staging = state + 2 * kState;
    powers = staging + 8 * 32 * 32 * (out_half ? 2 : 4);
    bars = powers + kPowers * 4;
    total = bars + 8 * 32;
  }
};
enum Bar {
  kFull = 0, kEmpty = kFull + kMaxStages, kScoresFull = kEmpty + kMaxStages, kPReady = kScoresFull + 2,
  kOFull = kPReady + 2, kOFree, kZReady, kAddFull, kAddFree, kSReady, kSFree, kDone, kBars
};
static_assert(kBars < 32, "room of the barriers");

__global__ void __launch_bounds__(kOutThreads, 1)
decay_chunks_kernel(const __grid_constant__ TcArgs t) {
  extern __shared__ unsigned char smem_raw[];
  const Args& a = t.a;
  const int which = blockIdx.z;
  const Pass& p = a.pass[which];
  const int bh = blockIdx.x / a.segments, segment = blockIdx.x % a.segments;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Chunks chunks(a, p, bh, segment);
  const int n = chunks.count, stages = t.stages;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const OutLayout at(stages, p.out_half);
  float* powers = reinterpret_cast<float*>(smem + at.powers);
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
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(bar(kFull + s), 1);
      mbar_init(bar(kEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kScoresFull + s), 1);
      mbar_init(bar(kPReady + s), 8);
    }
    mbar_init(bar(kOFull), 1);
    mbar_init(bar(kOFree), 8);
    mbar_init(bar(kZReady), 4);
    mbar_init(bar(kAddFull), 1);
    mbar_init(bar(kAddFree), 4);
    mbar_init(bar(kSReady), 4);
    mbar_init(bar(kSFree), 1);
    mbar_init(bar(kDone), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kPowers)
    powers[threadIdx.x - 32] = power(l2, threadIdx.x - 32);
  fence_before();
  __syncthreads();
  fence_after();
  const unsigned tmem = *slot;
  bool ok = true;
  const unsigned long long wait_ns = t.wait_ns;

  if (warp < 8) {
    // ---------------- P and outputs ----------------
    const int quad = warp & 3, odd = warp >> 2;
    const unsigned lanes = (unsigned)(32 * quad) << 16;
    const int row = 32 * quad + lane;
    const float f = p.zs * p.os;
    const bool half = p.out_half;
    unsigned char* staging = smem + at.staging + warp * (half ? 2048 : 4096);
    auto scores_to_p = [&](int i) {
      if (!warp_wait(bar(kScoresFull + (i & 1)), (i >> 1) & 1, wait_ns)) return false;
      fence_after();
      const unsigned base = tmem + kScores + 128u * (i & 1) + lanes;
      const int tokens = chunks.tokens(i);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int j = 2 * b + odd;          // block of 32 columns
        unsigned hi[16], lo[16];
        const bool none = p.reverse ? j < quad : j > quad;
        if (none || 32 * j >= tokens) {
#pragma unroll
          for (int e = 0; e < 16; ++e) hi[e] = lo[e] = 0u;
        } else {
          unsigned s[32];
          tmem_load32(base + 32 * j, s);
          // A block off the diagonal: g^(row - its last column) g^(last column - column).
          const int ahead = p.reverse ? 32 * j - row : row - (32 * j + 31);
          const float rowf = j == quad ? f : f * power(l2, ahead);
          tmem_loaded();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            Vec<2> v = {{__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])}};
            Vec<2> w;
            if (j == quad) {
              const int d0 = p.reverse ? 2 * e - lane : lane - 2 * e;
              const int d1 = p.reverse ? d0 + 1 : d0 - 1;
              w = ops::mul({{powers[d0 & 31], powers[d1 & 31]}}, ops::fill<2>(rowf));
              v = ops::mul(v, w);
              if (d0 < 0) v.f[0] = 0.f;
              if (d1 < 0) v.f[1] = 0.f;
            } else {
              w = p.reverse ? Vec<2>{{powers[2 * e], powers[2 * e + 1]}}
                            : Vec<2>{{powers[31 - 2 * e], powers[30 - 2 * e]}};
              v = ops::mul(v, ops::mul(w, ops::fill<2>(rowf)));
            }
            if (tokens < kChunk) {
              if (32 * j + 2 * e >= tokens) v.f[0] = 0.f;
              if (32 * j + 2 * e + 1 >= tokens) v.f[1] = 0.f;
            }
            hi[e] = take(v);
            lo[e] = ops::pack_bf16(v.f[0], v.f[1]);
          }
        }
        tmem_store16(base + 32 * j, hi);
        tmem_store16(base + 32 * j + 16, lo);
      }
      tmem_stored();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kPReady + (i & 1)));
      return true;
    };
    auto outputs = [&](int i) {
      if (!warp_wait(bar(kOFull), i & 1, wait_ns)) return false;
      fence_after();
      unsigned inner[32], outer[32];
      tmem_load32(tmem + kInner + 32 * odd + lanes, inner);
      tmem_load32(tmem + kOuter + 32 * odd + lanes, outer);
      const int tokens = chunks.tokens(i), place = chunks.place(i) * kChunk;
      const bool undecayed = p.undecayed && chunks.first + i == 0;
      const int steps = (p.reverse ? tokens - row : row + 1) - undecayed;
      const float g = row < tokens ? p.os * power(l2, steps) : 0.f;
      tmem_loaded();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOFree));
      const bool live = row < tokens;
      if (half) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 8 * c + 2 * e;
            const Vec<2> o = ops::fma({{__uint_as_float(outer[k]), __uint_as_float(outer[k + 1])}},
                                      ops::fill<2>(g),
                                      {{__uint_as_float(inner[k]), __uint_as_float(inner[k + 1])}});
            (&v.x)[e] = live ? ops::pack_bf16(o.f[0], o.f[1]) : 0u;
          }
          *reinterpret_cast<uint4*>(staging + (lane * 4 + (c ^ ((lane >> 1) & 3))) * 16) = v;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 4 * c + e;
            v[e] = live ? fmaf(__uint_as_float(outer[k]), g, __uint_as_float(inner[k])) : 0.f;
          }
          *reinterpret_cast<float4*>(staging + (lane * 8 + (c ^ (lane & 7))) * 16) =
              make_float4(v[0], v[1], v[2], v[3]);
        }
      }
      __syncwarp();
      // 64 or 128 bytes of a row at a time, rows side by side.
      const int pieces = half ? 4 : 8, per = half ? 8 : 4;
      const int piece = lane % pieces, row0 = lane / pieces;
      const int col = 32 * odd + piece * per;
      const long long first = (long long)bh * a.tokens;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= pieces) break;
        const int r = row0 + k * (32 / pieces);
        const int sw = half ? piece ^ ((r >> 1) & 3) : piece ^ (r & 7);
        const uint4 v = *reinterpret_cast<const uint4*>(staging + (r * pieces + sw) * 16);
        const int token = place + 32 * quad + r;
        if (token < a.tokens && col < p.b) {
          const long long to = ((first + token) * p.b + col) * (half ? 2 : 4);
          *reinterpret_cast<uint4*>(static_cast<char*>(p.out) + to) = v;
        }
      }
      __syncwarp();
      return true;
    };
    for (int i = 0; i <= n && ok; ++i) {
      if (i < n) ok = scores_to_p(i);
      if (ok && i > 0) ok = outputs(i - 1);
    }
  } else if (warp < 12) {
    // ---------------- the state ----------------
    const int tl = threadIdx.x - 256;
    const Place64 place(tl);
    const unsigned lanes = (unsigned)(32 * (warp & 3)) << 16;
    float S[32];
    const float* from = nullptr;
    long long row_step = p.b, col_step = 1;
    if (p.states) {
      from = p.states + ((long long)bh * a.segments + segment) * p.a * p.b;
    } else if (p.first) {
      from = p.first + (long long)bh * p.a * p.b;
      if (p.first_across) row_step = 1, col_step = p.a;
    }
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      S[c] = 0.f;
      if (from && place.row < p.a && place.col + c < p.b)
        S[c] = from[place.row * row_step + (place.col + c) * col_step];
    }
    unsigned char* operand_at = smem + at.state + place.row * 128;
    auto publish = [&] {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          Vec<2> v = {{S[8 * c + 2 * e], S[8 * c + 2 * e + 1]}};
          (&hi.x)[e] = take(v);
          (&lo.x)[e] = ops::pack_bf16(v.f[0], v.f[1]);
        }
        const unsigned piece = (unsigned)((place.col / 8 + c) ^ (place.row & 7)) << 4;
        *reinterpret_cast<uint4*>(operand_at + piece) = hi;
        *reinterpret_cast<uint4*>(operand_at + kState + piece) = lo;
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSReady));
    };
    if (n > 0) publish();
    for (int i = 0; i < n; ++i) {
      ok = warp_wait(bar(kAddFull), i & 1, wait_ns);
      if (!ok) break;
      fence_after();
      unsigned d[32];
      tmem_load32(tmem + kAdd + place.col + lanes, d);
      const Fade fade(l, chunks.tokens(i) - (p.undecayed && chunks.first + i == 0));
      tmem_loaded();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kAddFree));
#pragma unroll
      for (int c = 0; c < 32; ++c) S[c] = fade(S[c]) + __uint_as_float(d[c]);
      if (i + 1 < n) {
        ok = warp_wait(bar(kSFree), i & 1, wait_ns);
        if (!ok) break;
        publish();
      }
    }
    if (ok && p.last && segment == a.segments - 1) {
      const float g = p.undecayed && chunks.len > 0 ? exp2f(l2) : 1.f;
      float* to = p.last + (long long)bh * p.a * p.b + (long long)place.row * p.b + place.col;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (place.row < p.a && place.col + c < p.b) to[c] = S[c] * g;
    }
  } else if (warp < 16) {
    // ---------------- Z' ----------------
    const int row = threadIdx.x - 384;
    const float whole = p.zs * power(l2, p.reverse ? row : kChunk - 1 - row);
    for (int i = 0; i < n; ++i) {
      const int s = i % stages, tokens = chunks.tokens(i);
      ok = warp_wait(bar(kFull + s), (i / stages) & 1, wait_ns);
      if (ok && i > 0) ok = warp_wait(bar(kAddFull), (i - 1) & 1, wait_ns);
      if (!ok) break;
      unsigned char* stage = smem + at.stage + s * 3 * kTile;
      weigh<1>(stage + kTile, stage + 2 * kTile, smem + at.parts, row, 0, tokens, [&](int r) {
        return tokens == kChunk || p.reverse ? whole : p.zs * power(l2, max(0, tokens - 1 - r));
      });
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kZReady));
    }
  } else if (warp == kCopyWarp) {
    // ---------------- copies ----------------
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i % stages;
        if (i >= stages && !mbar_wait(bar(kEmpty + s), ((i / stages) - 1) & 1, wait_ns)) {
          ok = false;
          break;
        }
        if (t.skip_last && i == n - 1) break;   // fault injection: never copied
        const unsigned dst = smem_u32(smem + at.stage + s * 3 * kTile);
        const int token = chunks.place(i) * kChunk;
        mbar_expect_tx(bar(kFull + s), 3 * kTile);
        tma_load_3d(dst, &t.x[which], 0, token, bh, bar(kFull + s));
        tma_load_3d(dst + kTile, &t.y[which], 0, token, bh, bar(kFull + s));
        tma_load_3d(dst + 2 * kTile, &t.z[which], 0, token, bh, bar(kFull + s));
        issued = i + 1;
      }
      // Every copy lands before the CTA may finish.
      for (int i = max(0, issued - stages); i < issued; ++i)
        mbar_wait(bar(kFull + i % stages), (i / stages) & 1, wait_ns);
    }
  } else if (lane == 0) {
    // ---------------- products ----------------
    auto stage_at = [&](int i) { return smem_u32(smem + at.stage + (i % stages) * 3 * kTile); };
    auto scores = [&](int i) {
      if (!mbar_wait(bar(kFull + i % stages), (i / stages) & 1, wait_ns)) return false;
      // The tile of P that the scores overwrite: its product is done.
      if (i >= 2 && !mbar_wait(bar(kOFull), (i - 2) & 1, wait_ns)) return false;
      fence_after();
      const unsigned x = stage_at(i);
#pragma unroll
      for (int s = 0; s < kD / 16; ++s)
        mma(tmem + kScores + 128u * (i & 1), operand(x + s * 32, 0), operand(x + kTile + s * 32, 0),
            instruction(kChunk, false, false), s > 0);
      commit(bar(kScoresFull + (i & 1)));
      return true;
    };
    const unsigned parts = smem_u32(smem + at.parts), state = smem_u32(smem + at.state);
    if (n > 0) ok = scores(0);
    for (int i = 0; i < n && ok; ++i) {
      const unsigned x = stage_at(i), y = x + kTile, z = x + 2 * kTile;
      ok = mbar_wait(bar(kZReady), i & 1, wait_ns) &&
           (i == 0 || mbar_wait(bar(kAddFree), (i - 1) & 1, wait_ns));
      if (!ok) break;
      fence_after();
      issue_add(tmem + kAdd, y, parts);
      commit(bar(kAddFull));
      if (i + 1 < n) ok = scores(i + 1);
      ok = ok && mbar_wait(bar(kSReady), i & 1, wait_ns) &&
           (i == 0 || mbar_wait(bar(kOFree), (i - 1) & 1, wait_ns));
      if (!ok) break;
      fence_after();
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < kD / 16; ++s)
          mma(tmem + kOuter, operand(x + s * 32, 0), operand(state + k * kState + s * 2048, 0),
              instruction(kD, false, true), k > 0 || s > 0);
      commit(bar(kSFree));
      ok = mbar_wait(bar(kPReady + (i & 1)), (i >> 1) & 1, wait_ns);
      if (!ok) break;
      fence_after();
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < kChunk / 16; ++s)
          mma_tmem(tmem + kInner, tmem + kScores + 128u * (i & 1) + 32 * (s / 2) + 16 * k + 8 * (s & 1),
                   operand(z + s * 2048, 0), instruction(kD, false, true), k > 0 || s > 0);
      commit(bar(kOFull));
      commit(bar(kEmpty + i % stages));
    }
    commit(bar(kDone));
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
  {
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
constexpr int kSumStages = 4;

struct SumLayout {
  unsigned stage, parts, bars, total;
  __host__ __device__ SumLayout() {
    stage = 0;
    parts = kSumStages * 2 * kTile;
    bars = parts + 2 * kParts * kTile;
    total = bars + 8 * 32;
  }
};
enum SumBar {
  kSumFull = 0, kSumEmpty = kSumFull + kSumStages, kSumReady = kSumEmpty + kSumStages,
  kSumDone = kSumReady + 2, kSumFree = kSumDone + 2, kSumEnd = kSumFree + 2, kSumBars
};
static_assert(kSumBars < 32, "room of the barriers");

// Sum over a segment's tokens of y z^T with their decays to the segment's end.  Warps 0-7: Z'; 8-11: sums
// in registers (a chunk's products in tensor memory, whose adding rounds down, only); 12 copies, 13 issues.
__global__ void __launch_bounds__(kSumThreads, 1)
decay_sums_kernel(const __grid_constant__ TcArgs t) {
  extern __shared__ unsigned char smem_raw[];
  const Args& a = t.a;
  const int which = blockIdx.z;
  const Pass& p = a.pass[which];
  const int bh = blockIdx.x / (a.segments - 1), segment = blockIdx.x % (a.segments - 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Chunks chunks(a, p, bh, segment);
  const int n = chunks.count;
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const SumLayout at;
  const unsigned bars = smem_u32(smem + at.bars);
  auto bar = [&](int b) { return bars + 8u * (unsigned)b; };
  unsigned* slot = reinterpret_cast<unsigned*>(smem + at.bars + 8 * kSumBars);
  const float l2 = log_decay(a, bh) * kLog2e;
  constexpr unsigned kSumColumns = 128;

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
  fence_before();
  __syncthreads();
  fence_after();
  const unsigned tmem = *slot;
  bool ok = true;
  const unsigned long long wait_ns = t.wait_ns;

  if (warp < 8) {
    const int row = threadIdx.x >> 1, share = threadIdx.x & 1;
    int after = 0;   // tokens of the segment after the chunk
    for (int i = 0; i < n; ++i) after += chunks.tokens(i);
    for (int i = 0; i < n; ++i) {
      const int s = i % kSumStages, tokens = chunks.tokens(i);
      after -= tokens;
      ok = warp_wait(bar(kSumFull + s), (i / kSumStages) & 1, wait_ns);
      if (ok && i > 1) ok = warp_wait(bar(kSumDone + (i & 1)), ((i >> 1) - 1) & 1, wait_ns);
      if (!ok) break;
      unsigned char* stage = smem + at.stage + s * 2 * kTile;
      weigh<2>(stage, stage + kTile, smem + at.parts + (i & 1) * kParts * kTile, row, share, tokens,
               [&](int r) {
                 return p.zs * power(l2, after + (p.reverse ? r : max(0, tokens - 1 - r)));
               });
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSumReady + (i & 1)));
    }
  } else if (warp < 12) {
    const Place64 place(threadIdx.x - 256);
    const unsigned lanes = (unsigned)(32 * (warp & 3)) << 16;
    float S[32] = {};
    for (int i = 0; i < n; ++i) {
      ok = warp_wait(bar(kSumDone + (i & 1)), (i >> 1) & 1, wait_ns);
      if (!ok) break;
      fence_after();
      unsigned d[32];
      tmem_load32(tmem + 64u * (i & 1) + place.col + lanes, d);
      tmem_loaded();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSumFree + (i & 1)));
#pragma unroll
      for (int c = 0; c < 32; ++c) S[c] += __uint_as_float(d[c]);
    }
    float* to = p.states + (((long long)bh * a.segments + segment) * p.a + place.row) * p.b + place.col;
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (place.row < p.a && place.col + c < p.b) to[c] = S[c];
  } else if (warp == 12) {
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i % kSumStages;
        if (i >= kSumStages && !mbar_wait(bar(kSumEmpty + s), ((i / kSumStages) - 1) & 1, wait_ns)) {
          ok = false;
          break;
        }
        if (t.skip_last && i == n - 1) break;   // fault injection: never copied
        const unsigned dst = smem_u32(smem + at.stage + s * 2 * kTile);
        const int token = chunks.place(i) * kChunk;
        mbar_expect_tx(bar(kSumFull + s), 2 * kTile);
        tma_load_3d(dst, &t.y[which], 0, token, bh, bar(kSumFull + s));
        tma_load_3d(dst + kTile, &t.z[which], 0, token, bh, bar(kSumFull + s));
        issued = i + 1;
      }
      for (int i = max(0, issued - kSumStages); i < issued; ++i)
        mbar_wait(bar(kSumFull + i % kSumStages), (i / kSumStages) & 1, wait_ns);
    }
  } else if (lane == 0) {
    for (int i = 0; i < n; ++i) {
      ok = mbar_wait(bar(kSumReady + (i & 1)), (i >> 1) & 1, wait_ns) &&
           (i < 2 || mbar_wait(bar(kSumFree + (i & 1)), ((i >> 1) - 1) & 1, wait_ns));
      if (!ok) break;
      fence_after();
      issue_add(tmem + 64u * (i & 1), smem_u32(smem + at.stage + (i % kSumStages) * 2 * kTile),
                smem_u32(smem + at.parts + (i & 1) * kParts * kTile));
      commit(bar(kSumDone + (i & 1)));
      commit(bar(kSumEmpty + i % kSumStages));
    }
    commit(bar(kSumEnd));
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

bool encode(CUtensorMap* map, const void* base, int width, int tokens, int bh) {
  return tma_encode_3d_sw128(map, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)width,
                             (uint64_t)tokens, (uint64_t)bh, (uint64_t)width * 2,
                             (uint64_t)tokens * width * 2, kD, kChunk);
}

}  // namespace

bool tc_fits(const Args& a, int passes) {
  for (int i = 0; i < passes; ++i) {
    const Pass& p = a.pass[i];
    if (!p.x_half || !p.y_half || !p.z_half || p.a > kD || p.b > kD || p.a % 8 || p.b % 8) return false;
    for (const void* q : {p.x, p.y, p.z, static_cast<const void*>(p.out)})
      if (!ops::aligned(q, 16)) return false;
  }
  return true;
}

cudaError_t launch_tc(const Args& a, int passes, int bh, unsigned* err, unsigned long long wait_ns,
                      int skip_last, cudaStream_t st) {
  TcArgs t;
  t.a = a;
  t.err = err;
  t.wait_ns = wait_ns;
  t.skip_last = skip_last;
  bool out_half = true;
  for (int i = 0; i < passes; ++i) {
    const Pass& p = a.pass[i];
    out_half = out_half && p.out_half;
    if (!encode(&t.x[i], p.x, p.a, a.tokens, bh) || !encode(&t.y[i], p.y, p.a, a.tokens, bh) ||
        !encode(&t.z[i], p.z, p.b, a.tokens, bh))
      return cudaErrorInvalidValue;
  }
  t.stages = 3;
  while (t.stages > 2 && OutLayout(t.stages, out_half).total + 1024 > kSmemMost) --t.stages;
  cudaError_t e = cudaSuccess;
  if (a.segments > 1) {
    t.skip_last = 0;   // (the outputs' kernel is the one that is told to)
    const unsigned smem = SumLayout().total + 1024;
    e = cudaFuncSetAttribute(decay_sums_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
    if (e != cudaSuccess) return e;
    decay_sums_kernel<<<dim3((unsigned)(bh * (a.segments - 1)), 1, (unsigned)passes), kSumThreads, smem,
                        st>>>(t);
    e = cudaGetLastError();
    t.skip_last = skip_last;
  }
  if (e == cudaSuccess && a.pass[0].states) e = launch_carry(a, passes, bh, st);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(decay_chunks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
  if (e != cudaSuccess) return e;
  decay_chunks_kernel<<<dim3((unsigned)(bh * a.segments), 1, (unsigned)passes), kOutThreads,
                        OutLayout(t.stages, out_half).total + 1024, st>>>(t);
  return cudaGetLastError();
}

}  // namespace decay
}  // namespace lapl
