// decay.cuh -- what the kernels of the linear attention with decays share (lapl_decay_* of
// include/lapl_ops.h).
//
// One pass.  With rows x, y of `a` values and z of `b` values for every token, in processing order:
//   S_i = g S_{i-1} + zs y_i z_i^T,   o_i = os x_i S_i                                       (a x b)
// The forward is the pass with (x, y, z) = (q, k, v).  The gradients are passes, too: of the forward's
// o_i = os sum_{j <= i} g^{i-j} (q_i . k_j) v_j follow
//   dq_i = os sum_{j <= i} g^{i-j} (do_i . v_j) k_j         (do, v, k), in the forward's order;
//   dk_j = os sum_{i >= j} g^{i-j} (v_j . do_i) q_i         (v, do, q), in the opposite one;
//   dv_j = os sum_{i >= j} g^{i-j} (k_j . q_i) do_i         (k, q, do), in the opposite one.
// There the final state's gradient is the state to start from, which the first token meets undecayed
// (`undecayed`), and what is left after all tokens, decayed once more, is the first state's.
//
// A sequence is worked on in segments side by side: a first launch forms each segment's own
// contribution to the state, a second the state before each segment, a third the outputs.
#pragma once

#include "ops_common.cuh"

namespace lapl {

namespace decay {

// Smallest log_decay: it underflows at the first step, and stays finite times any length.
constexpr float kLeastLog = -1e30f;
constexpr float kLog2e = 1.4426950408889634f;

struct Pass {
  const void* x;          // [BH,N,a]
  const void* y;          // [BH,N,a]
  const void* z;          // [BH,N,b]
  void* out;              // [BH,N,b]
  const float* first;     // state to start from, [BH,a,b], or [BH,b,a] if first_across; or null
  float* last;            // state after all tokens, or null
  float* states;          // workspace: [BH,segments,a,b]; null (one segment): the state is `first`
  int a, b;
  int x_half, y_half, z_half, out_half;   // bf16
  int reverse;
  int first_across;
  int undecayed;
  float zs, os;
};

constexpr int kMaxPasses = 3;
constexpr int kTcChunk = 128;   // tokens of a chunk on the tensor cores
constexpr int kRowsStep = 16;   // token by token, segments are multiples of this
constexpr int kMostSegments = 128;
struct Args {
  Pass pass[kMaxPasses];
  const float* log_decay;   // [H]
  const int* lengths;       // [B] or null
  int heads, tokens;
  int segments, per_segment;   // tokens of a segment (in chunks: a multiple of kTcChunk)
  int chunks;   // 1: chunks lie in memory as they do from the first token on, in either order
};

// A segment of one sequence.
struct Range {
  int len;         // tokens of the sequence
  int begin, end;  // of the segment, in processing order (padding among them)
  __device__ __forceinline__ Range(const Args& a, int bh, int segment) {
    len = a.tokens;
    if (a.lengths) len = min(max(a.lengths[bh / a.heads], 0), a.tokens);
    begin = segment * a.per_segment;
    end = min(begin + a.per_segment, a.tokens);
  }
  // Tokens of the segment that are no padding.
  __device__ __forceinline__ int live(const Args& a, const Pass& p) const {
    if (!a.chunks || !p.reverse) return max(0, min(end, len) - begin);
    // From the last chunk on, which may be short.
    const int all = (len + kTcChunk - 1) / kTcChunk, per = a.per_segment / kTcChunk;
    const int segment = begin / a.per_segment;
    const int top = all - segment * per, bottom = max(0, top - per);
    return top <= 0 ? 0 : min(len, top * kTcChunk) - bottom * kTcChunk;
  }
};

// g^n, with log2g = log2(g).
__device__ __forceinline__ float power(float log2g, int n) { return exp2f(log2g * (float)n); }
// The logarithm of a head's decay, at most 0, or NaN.
__device__ __forceinline__ float log_decay(const Args& a, int bh) {
  const float l = a.log_decay[bh % a.heads];
  return l > 0.f ? 0.f : l < kLeastLog ? kLeastLog : l;   // (fmaxf and fminf drop a NaN)
}
// A state's decay over n tokens, s -> s exp(l n).  With a decay near 1 that factor's own rounding, the
// same at every step, would add up over as many steps as the state remembers: there it is s + s m with
// m = exp(l n) - 1, whose rounding counts for less.
struct Fade {
  float factor, less;   // less: m, or 0 where the factor is used
  Fade() = default;
  __device__ __forceinline__ Fade(float l, int n) {
    const float x = n == 0 ? 0.f : l * (float)n;   // (no token: nothing fades, by a NaN either)
    factor = exp2f(x * kLog2e);
    less = x > -0.5f ? expm1f(x) : 0.f;
    if (x > -0.5f) factor = 1.f;
  }
  __device__ __forceinline__ float operator()(float s) const { return fmaf(s, less, s * factor); }
  __device__ __forceinline__ ops::Vec<2> operator()(const ops::Vec<2>& s) const {
    return ops::fma(s, ops::fill<2>(less), ops::mul(s, ops::fill<2>(factor)));
  }
};

// The next launch's CTAs may be placed from here on; they wait themselves for what they need.
__device__ __forceinline__ void release_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Until the launch before has ended, where this one was placed early.
__device__ __forceinline__ void await_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// early: placed while the launch before runs.
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, bool early, cudaStream_t st,
                   const A&... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a...);
}

// CTAs of four warps of the kernel that goes token by token that an SM has registers for, with as many padded
// rows and columns of a lane.
constexpr int rows_ctas(int rows, int cols) { return rows * cols <= 256 ? 4 : rows * cols <= 384 ? 3 : 2; }
// How that kernel takes a pass's rows: as it pads them, a warp's columns, a CTA's warps, and those that an SM has
// room for.  A lane has 8 columns where that is no more than half of them padding, and where it has registers.
struct RowsShape {
  int rows, cols, warps, room;
};
inline RowsShape rows_shape(int rows, int cols) {
  const int padded = rows <= 64 ? (rows + 15) / 16 * 16 : rows <= 80 ? 80 : rows <= 96 ? 96 : 128;
  const int wide = cols > 32 && padded <= 32 ? 64 : 32;
  return {padded, wide, (cols + wide - 1) / wide, 4 * rows_ctas(padded, wide / 8)};
}
// Passes from the i-th on that one launch takes: those of the same padded rows.
template <class Rows>
int rows_together(int i, int passes, Rows rows) {
  int n = 1;
  while (i + n < passes && rows_shape(rows(i + n), 1).rows == rows_shape(rows(i), 1).rows) ++n;
  return n;
}

// All launches of the passes token by token, for any sizes and types (decay_rows.cu).
cudaError_t launch_rows(const Args& a, int passes, int bh, cudaStream_t st);
// The launch, right after that of the segments' own states, that turns them into those before each.
cudaError_t launch_carry(const Args& a, int passes, int bh, cudaStream_t st);
// All launches of the passes in chunks on the tensor cores (decay_tc.cu), where types, sizes and
// alignment allow that.
bool tc_fits(const Args& a, int passes);
cudaError_t launch_tc(const Args& a, int passes, int bh, unsigned* err, unsigned long long wait_ns,
                      int skip_last, cudaStream_t st);

}  // namespace decay
}  // namespace lapl
