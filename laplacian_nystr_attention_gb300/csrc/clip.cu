// clip.cu -- global norm of many gradient tensors and clipping: lapl_clip_* of
// include/lapl_ops.h.
//
// The tensors are cut into pieces of 2048 to 65536 values, as large as leaves no CTA much longer at
// work than the others (33 tensors of 18.8 million values together: clipped in 19 us, 36 with four
// pieces or more for each CTA); the table of tensors travels as a kernel parameter (no table in
// device memory, nothing to upload), for up to kTable tensors a launch.  First pass:
// CTA b sums the squares of pieces b, b + grid, ... and writes one partial.  Second pass: every CTA
// sums all partials in the same order, so each has the same norm to the last bit, and scales its
// pieces.  HBM-bound: the first pass reads every value, the second reads and writes it.  Measured:
// 2^28 values (540 MB of bf16 and fp32) 82 us for the norm (the copy's rate), 258 us to clip
// them into other tensors, of which 239 are the bytes of both passes at that rate; 24 tensors of 2^20
// values together 7.7 us, the latency of two launches.
//
// Squares.  fp32 holds values over 2^-149 .. 2^128, whose squares need twice that range.  There are
// three sums: of (x 2^35)^2, and for where that vanishes or overflows of (x 2^86)^2 and (x 2^-72)^2.  Their
// squares are normal numbers from |x| = 2^-98, 2^-149 and 2^9 on.  The first is used if it comes out at
// 2^-86 or more, against which the 2^-150 that each value may have lost is nothing even for 2^40
// values.  If it does not, the second cannot overflow, and loses nothing.  If it overflows, all squares
// together are more than 2^58, of which the third loses 2^-6 for each value at most, 2^-24 for 2^40 of
// them.  A CTA sums the first alone, and the others are that times a power of two, unless it may have lost
// something that counts, or nearly overflows: then the CTA goes through its pieces again for the other
// two.  (All three for every value: 90 us instead of 79 for 2^28 bf16 values.)  Partial sums are fp32
// over the 128 values at most that a thread has of a piece, in two chains, then pairs of floats.
#include <algorithm>
#include <new>
#include <type_traits>
#include <vector>

#include "ops_common.cuh"

namespace lapl {
namespace clip {

using ops::Pair;

constexpr int kThreads = 512;
constexpr int kCtas = 4;             // of an SM, all resident at once: 32 registers a thread
constexpr int kMinPiece = 2048, kMaxPiece = 65536;   // values, powers of two
constexpr int kStart = 2048;   // values that a CTA streams while it starts on a piece
constexpr int kUnroll = 4;           // 16-byte loads of a thread in flight, or 2 kUnroll of a value
constexpr int kTable = 1000;         // tensors of a launch: 20 KB of its 32 KB of parameters
constexpr int kSmallTable = 64;
constexpr float kLow = 34359738368.f;                // 2^35
constexpr float kTiny = 77371252455336267181195264.f;   // 2^86
// A sum of squares times kLow^2 that is used.
constexpr float kLowUsed = 1.292469707114106e-26f;      // 2^-86
// A thread's sum for one piece: 128 values may be off by 2^-143 together, 2^-25 of this.
constexpr float kLowLeast = 3.009265538105056e-36f;     // 2^-118
// A thread's sum for all its pieces, below which a CTA's does not overflow.
constexpr float kLowMost = 8.307674973655724e34f;       // 2^116
constexpr float kHigh = 2.117582368135751e-22f;      // 2^-72

template <int N>
struct Table {
  const void* in[N];
  void* out[N];
  int first[N + 1];     // first piece of each tensor, and the number of pieces
  int last[N];          // values of its last piece
  unsigned char kind[N];   // lapl_dtype
  int tensors;
  int piece;            // values of the others
};

// One piece: where it is and how many values it has.
struct Piece {
  const char* in;
  char* out;
  int count;
  bool half;   // bf16
};
template <int N>
__device__ __forceinline__ Piece piece_of(const Table<N>& t, int i) {
  int lo = 0, hi = t.tensors;   // first[lo] <= i < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= i) lo = mid; else hi = mid;
  }
  Piece p;
  p.half = t.kind[lo] == LAPL_BF16;
  const long long off = (long long)(i - t.first[lo]) * t.piece * (p.half ? 2 : 4);
  p.in = reinterpret_cast<const char*>(t.in[lo]) + off;
  p.out = t.out[lo] ? reinterpret_cast<char*>(t.out[lo]) + off : nullptr;
  p.count = i + 1 == t.first[lo + 1] ? t.last[lo] : t.piece;
  return p;
}

// Squares of even and odd values times scale, and whether there is anything but zeros.
struct Sums {
  ops::Vec<2> sum;
  uint32_t bits;
  __device__ __forceinline__ void add(const ops::Vec<2>& x, float scale) {
    const ops::Vec<2> v = ops::mul(x, ops::fill<2>(scale));
    sum = ops::fma(v, v, sum);
  }
  template <bool kHalf>
  __device__ __forceinline__ void add(const uint4& v, float scale) {
    bits |= v.x | v.y;
    bits |= v.z | v.w;
    if constexpr (kHalf) {
      add({bf16_lo(v.x), bf16_hi(v.x)}, scale);
      add({bf16_lo(v.y), bf16_hi(v.y)}, scale);
      add({bf16_lo(v.z), bf16_hi(v.z)}, scale);
      add({bf16_lo(v.w), bf16_hi(v.w)}, scale);
    } else {
      add({__uint_as_float(v.x), __uint_as_float(v.y)}, scale);
      add({__uint_as_float(v.z), __uint_as_float(v.w)}, scale);
    }
  }
};

// Calls use(k, v) for each of n values or vectors at p (k: its index), kAtOnce of a thread's loads at
// a time.
template <int kAtOnce, class T, class Use>
__device__ __forceinline__ void each(const T* p, int n, Use use) {
  int k = threadIdx.x;
  for (; k + (kAtOnce - 1) * kThreads < n; k += kAtOnce * kThreads) {
    T v[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) v[u] = p[k + u * kThreads];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) use(k + u * kThreads, v[u]);
  }
  for (; k < n; k += kThreads) use(k, p[k]);
}

struct Pairs {
  Pair of[3];   // low, tiny, high
};
// Sum over the CTA in thread 0 (fixed order).
__device__ __forceinline__ Pair block_sum(Pair s, Pair* sm) {
  auto across = [](Pair s, int n) {
    for (int o = n / 2; o > 0; o >>= 1) {
      const float hi = __shfl_down_sync(0xffffffffu, s.hi, o);
      s.add(hi, __shfl_down_sync(0xffffffffu, s.lo, o));
    }
    return s;
  };
  s = across(s, 32);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) s = across(sm[threadIdx.x & (kThreads / 32 - 1)], kThreads / 32);
  return s;
}

// The squares of one piece.
template <bool kHalf>
__device__ __forceinline__ Sums squares(const Piece& p, float scale) {
  constexpr int kBytes = kHalf ? 2 : 4;
  // Values before the first 16-byte boundary, 16 bytes at a time, and the rest.
  const int head = min(p.count, (int)((16 - ((uintptr_t)p.in & 15)) & 15) / kBytes);
  const int vectors = (p.count - head) * kBytes / 16;
  Sums s = {};
  each<kUnroll>(reinterpret_cast<const uint4*>(p.in + head * kBytes), vectors,
              [&](int, const uint4& v) { s.add<kHalf>(v, scale); });
  const int body = vectors * 16 / kBytes;
  for (int k = threadIdx.x; k < p.count - body; k += kThreads) {
    const int e = k < head ? k : k + body;
    const float v = kHalf ? ops::bf16_bits(reinterpret_cast<const uint16_t*>(p.in)[e])
                          : reinterpret_cast<const float*>(p.in)[e];
    s.bits |= __float_as_uint(v);
    s.add({v, 0.f}, scale);
  }
  return s;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas)
clip_norm_kernel(const __grid_constant__ Table<N> t, Pairs* part) {
  __shared__ Pair sm[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int pieces = t.first[t.tensors];
  Pairs& mine = part[blockIdx.x];
  // One pass, or three.
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const float scale = pass == 0 ? kLow : pass == 1 ? kTiny : kHigh;
    Pair sum = {};
    bool unsure = false;
    for (int i = blockIdx.x; i < pieces; i += gridDim.x) {
      const Piece p = piece_of(t, i);
      const Sums s = p.half ? squares<true>(p, scale) : squares<false>(p, scale);
      const float v = s.sum.f[0] + s.sum.f[1];
      unsure |= v < kLowLeast && (s.bits & (p.half ? 0x7fff7fffu : 0x7fffffffu)) != 0u;
      sum.add(v);
    }
    const bool more = __syncthreads_or(unsure || !(sum.hi < kLowMost)) || pass > 0;
    sum = block_sum(sum, sm);
    if (threadIdx.x == 0) mine.of[pass] = sum;
    if (!more) {
      constexpr float kUp = (kTiny / kLow) * (kTiny / kLow), kDown = kHigh / kLow;   // kDown twice
      if (threadIdx.x == 0) {
        mine.of[1] = {sum.hi * kUp, sum.lo * kUp};
        mine.of[2] = {sum.hi * kDown * kDown, sum.lo * kDown * kDown};
      }
      return;
    }
  }
}

// The norm from all partials, the same in every thread.
__device__ __forceinline__ float norm_of(const Pairs* part, int parts) {
  __shared__ Pair sm[kThreads / 32];
  __shared__ float norm;
  __shared__ int next;
  // The first sum, and where that is of no use another.
#pragma unroll 1
  for (int which = 0;;) {
    Pair s = {};
    for (int k = threadIdx.x; k < parts; k += kThreads) s.add(part[k].of[which].hi, part[k].of[which].lo);
    s = block_sum(s, sm);
    if (threadIdx.x == 0) {
      const float v = s.value();
      norm = sqrtf(v) * (which == 0 ? 1.f / kLow : which == 1 ? 1.f / kTiny : 1.f / kHigh);
      next = which > 0 || (v >= kLowUsed && v < INFINITY) ? 0 : v < kLowUsed ? 1 : 2;
    }
    __syncthreads();
    which = next;
    if (which == 0) return norm;
  }
}

__global__ void __launch_bounds__(kThreads)
clip_finish_kernel(const Pairs* part, int parts, float* norm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are written
  const float v = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = v;
}

// One piece to its output, times scale where kScale.
template <bool kHalf, bool kScale>
__device__ __forceinline__ void copy_piece(const Piece& p, float scale) {
  constexpr int kBytes = kHalf ? 2 : 4;
  auto scaled = [&](uint32_t w) {
    if constexpr (!kScale) return w;
    else if constexpr (kHalf) return ops::pack_bf16(bf16_lo(w) * scale, bf16_hi(w) * scale);
    else return __float_as_uint(__uint_as_float(w) * scale);
  };
  using Word = typename std::conditional<kHalf, uint16_t, uint32_t>::type;
  const Word* in = reinterpret_cast<const Word*>(p.in);
  Word* out = reinterpret_cast<Word*>(p.out);
  if (((uintptr_t)p.in ^ (uintptr_t)p.out) & 15) {   // no vector of one is one of the other
    each<2 * kUnroll>(in, p.count, [&](int k, Word w) { out[k] = (Word)scaled(w); });
    return;
  }
  const int head = min(p.count, (int)((16 - ((uintptr_t)p.in & 15)) & 15) / kBytes);
  const int vectors = (p.count - head) * kBytes / 16;
  uint4* to = reinterpret_cast<uint4*>(out + head);
  each<kUnroll>(reinterpret_cast<const uint4*>(in + head), vectors, [&](int k, const uint4& v) {
    to[k] = make_uint4(scaled(v.x), scaled(v.y), scaled(v.z), scaled(v.w));
  });
  const int body = vectors * 16 / kBytes;
  for (int k = threadIdx.x; k < p.count - body; k += kThreads) {
    const int e = k < head ? k : k + body;
    out[e] = (Word)scaled(in[e]);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
clip_scale_kernel(const __grid_constant__ Table<N> t, const Pairs* part, int parts, float max_norm,
                  float* norm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are written
  const float v = norm_of(part, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = v;
  const bool clip = isfinite(v) && v > max_norm;
  const float scale = clip ? max_norm / v : 1.f;
  const int pieces = t.first[t.tensors];
  // Last pieces first: those the first pass has left in L2.
  for (int i = pieces - 1 - (int)blockIdx.x; i >= 0; i -= gridDim.x) {
    const Piece p = piece_of(t, i);
    if (clip) {
      if (p.half) copy_piece<true, true>(p, scale);
      else copy_piece<false, true>(p, scale);
    } else if (p.in != p.out) {
      if (p.half) copy_piece<true, false>(p, scale);
      else copy_piece<false, false>(p, scale);
    }
  }
}

}  // namespace clip
}  // namespace lapl

struct lapl_clip_plan {
  std::vector<long long> counts;
  std::vector<int> dtypes;
  struct Batch {       // the tensors of one launch
    std::vector<int> index;   // those with values
    int piece;                // values of a piece
    int pieces, grid, first_part;
  };
  std::vector<Batch> batches;
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;   // scratch of the overlap check
  int parts;           // partials of all launches
  int device;
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

lapl_status validate(const lapl_clip_config* c) {
  if (!c || c->tensors < 0) return LAPL_ERR_INVALID_ARG;
  if (c->tensors > 0 && (!c->counts || !c->dtypes)) return LAPL_ERR_INVALID_ARG;
  for (int i = 0; i < c->tensors; ++i) {
    if (c->counts[i] < 0 || !ops::is_float_dtype(c->dtypes[i])) return LAPL_ERR_INVALID_ARG;
    if (c->counts[i] > (1LL << 40)) return LAPL_ERR_UNSUPPORTED;
  }
  return LAPL_OK;
}

// Fills the table of one batch.
template <int N>
void fill(const lapl_clip_plan& p, const lapl_clip_plan::Batch& b, const void* const* in,
          void* const* out, clip::Table<N>* t) {
  int first = 0, k = 0;
  for (const int i : b.index) {
    t->in[k] = in[i];
    t->out[k] = out ? out[i] : nullptr;
    t->first[k] = first;
    const long long pieces = (p.counts[i] - 1) / b.piece + 1;
    first += (int)pieces;
    t->last[k] = (int)(p.counts[i] - (pieces - 1) * b.piece);
    t->kind[k] = (unsigned char)p.dtypes[i];
    ++k;
  }
  t->first[k] = first;
  t->tensors = k;
  t->piece = b.piece;
}

// dependent: placed before the kernel before it has ended, for whose end it waits itself.
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), int grid, bool dependent, cudaStream_t st, const A&... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(clip::kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a...);
}

template <int N>
cudaError_t launch_norm(const lapl_clip_plan& p, const lapl_clip_plan::Batch& b,
                        const void* const* in, clip::Pairs* part, cudaStream_t st) {
  clip::Table<N> t;
  fill(p, b, in, nullptr, &t);
  return launch(clip::clip_norm_kernel<N>, b.grid, false, st, t, part + b.first_part);
}
template <int N>
cudaError_t launch_scale(const lapl_clip_plan& p, const lapl_clip_plan::Batch& b,
                         const void* const* in, void* const* out, const clip::Pairs* part,
                         float max_norm, float* norm, bool dependent, cudaStream_t st) {
  clip::Table<N> t;
  fill(p, b, in, out, &t);
  return launch(clip::clip_scale_kernel<N>, b.grid, dependent, st, t, part, p.parts, max_norm, norm);
}

lapl_status check_pointers(const lapl_clip_plan& p, const void* const* a) {
  for (size_t i = 0; i < p.counts.size(); ++i) {
    if (p.counts[i] == 0) continue;
    if (!a[i]) return LAPL_ERR_INVALID_ARG;
    if (!ops::aligned(a[i], ops::dtype_bytes(p.dtypes[i]))) return LAPL_ERR_ALIGNMENT;
  }
  return LAPL_OK;
}

// Whether outputs overlap each other, or an input that is not their own.
bool overlapping(lapl_clip_plan* p, const void* const* in, void* const* out) {
  auto& s = p->spans;
  s.clear();
  for (size_t i = 0; i < p->counts.size(); ++i) {
    if (p->counts[i] == 0) continue;
    const uintptr_t bytes = (uintptr_t)p->counts[i] * ops::dtype_bytes(p->dtypes[i]);
    // An output's end is odd-tagged: spans are doubled to make room for the tag.
    const uintptr_t o = (uintptr_t)out[i], a = (uintptr_t)in[i];
    s.emplace_back(o, (o + bytes) * 2 + 1);
    if (a != o) s.emplace_back(a, (a + bytes) * 2);
  }
  std::sort(s.begin(), s.end());
  uintptr_t end = 0, out_end = 0;   // furthest end so far, of all spans and of outputs
  for (const auto& v : s) {
    const bool is_out = v.second & 1;
    if (v.first < (is_out ? end : out_end)) return true;
    end = std::max(end, v.second / 2);
    if (is_out) out_end = std::max(out_end, v.second / 2);
  }
  return false;
}

// The norm's partials of every launch.
cudaError_t partials(const lapl_clip_plan& p, const void* const* in, clip::Pairs* part, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  for (const auto& b : p.batches) {
    e = (int)b.index.size() <= clip::kSmallTable
            ? launch_norm<clip::kSmallTable>(p, b, in, part, st)
            : launch_norm<clip::kTable>(p, b, in, part, st);
    if (e != cudaSuccess) break;
  }
  return e;
}

lapl_status check(lapl_clip_plan* p, const void* const* grads, float* norm, void* workspace,
                  size_t workspace_bytes, const char* where) {
  if (!grads && !p->counts.empty()) return LAPL_ERR_INVALID_ARG;
  if (!norm || !workspace) return LAPL_ERR_INVALID_ARG;
  if (!ops::aligned(norm, 4) || !ops::aligned(workspace, 16)) return LAPL_ERR_ALIGNMENT;
  size_t need = 0;
  lapl_clip_workspace_size(p, &need);
  if (workspace_bytes < need) return LAPL_ERR_WORKSPACE;
  const lapl_status st = check_pointers(*p, grads);
  if (st != LAPL_OK) return st;
  return ops::check_device(p->device, p->last_error, where);
}

lapl_status create(const lapl_clip_config* cfg, int sms, int device, lapl_clip_plan** out) {
  lapl_clip_plan* p = new lapl_clip_plan();
  *out = p;
  p->device = device;
  p->counts.assign(cfg->counts, cfg->counts + cfg->tensors);
  p->dtypes.assign(cfg->dtypes, cfg->dtypes + cfg->tensors);
  p->spans.reserve(2 * p->counts.size());
  p->parts = 0;
  // Tensors with values, kTable to a launch and at most 2^30 of the largest pieces.
  long long pieces = 0;
  for (int i = 0; i < cfg->tensors; ++i) {
    if (p->counts[i] == 0) continue;
    const long long more = (p->counts[i] - 1) / clip::kMaxPiece + 1;
    if (p->batches.empty() || (int)p->batches.back().index.size() == clip::kTable ||
        pieces + more > (1LL << 30)) {
      p->batches.emplace_back();
      pieces = 0;
    }
    p->batches.back().index.push_back(i);
    pieces += more;
  }
  const long long ctas = (long long)clip::kCtas * sms;
  for (auto& b : p->batches) {
    // The piece with the least on the longest path: rounds of pieces, and starting on each.  (Of any
    // size, one or two for each CTA, large ones took up to 5% longer.)
    long long best = 0;
    for (int piece = clip::kMaxPiece; piece >= clip::kMinPiece; piece /= 2) {
      long long n = 0;
      for (const int i : b.index) n += (p->counts[i] - 1) / piece + 1;
      const long long cost = (n + ctas - 1) / ctas * (piece + clip::kStart);
      if (best != 0 && (cost >= best || n > (1LL << 30))) continue;
      best = cost;
      b.piece = piece;
      b.pieces = (int)n;
    }
    b.grid = (int)std::min<long long>(b.pieces, ctas);
    b.first_part = p->parts;
    p->parts += b.grid;
  }
  return LAPL_OK;
}

}  // namespace

extern "C" {

lapl_status lapl_clip_create(const lapl_clip_config* cfg, lapl_clip_handle* out) {
  if (!out) return LAPL_ERR_INVALID_ARG;
  *out = nullptr;
  const lapl_status st = validate(cfg);
  if (st != LAPL_OK) return st;
  int sms = 0, device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return LAPL_ERR_CUDA;
  lapl_clip_plan* p = nullptr;
  try {
    create(cfg, sms, device, &p);
  } catch (const std::exception&) {   // out of host memory
    delete p;
    return LAPL_ERR_INVALID_ARG;
  }
  *out = p;
  return LAPL_OK;
}

lapl_status lapl_clip_workspace_size(lapl_clip_handle p, size_t* bytes) {
  if (!p || !bytes) return LAPL_ERR_INVALID_ARG;
  *bytes = align_up((size_t)std::max(p->parts, 1) * sizeof(clip::Pairs), kAlign);
  return LAPL_OK;
}

lapl_status lapl_clip_norm(lapl_clip_handle p, const void* const* grads, float* norm,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  const lapl_status st = check(p, grads, norm, workspace, workspace_bytes, "clip_norm/device");
  if (st != LAPL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  clip::Pairs* part = static_cast<clip::Pairs*>(workspace);
  cudaError_t e = partials(*p, grads, part, s);
  if (e == cudaSuccess) {
    e = launch(clip::clip_finish_kernel, 1, p->batches.size() == 1, s,
               static_cast<const clip::Pairs*>(part), p->parts, norm);
  }
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "clip_norm");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

lapl_status lapl_clip_apply(lapl_clip_handle p, const void* const* grads, void* const* outs,
                            float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  if (!(max_norm >= 0.f) || !isfinite(max_norm)) return LAPL_ERR_INVALID_ARG;
  lapl_status st = check(p, grads, norm, workspace, workspace_bytes, "clip_apply/device");
  if (st != LAPL_OK) return st;
  void* const* to = outs ? outs : const_cast<void* const*>(grads);
  st = check_pointers(*p, to);
  if (st != LAPL_OK) return st;
  if (overlapping(p, grads, to)) return LAPL_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  clip::Pairs* part = static_cast<clip::Pairs*>(workspace);
  cudaError_t e = partials(*p, grads, part, s);
  // One launch after one: the second may be placed early.  (Of several, a later one would only wait
  // for the one just before it.)
  const bool alone = p->batches.size() == 1;
  for (size_t k = 0; k < p->batches.size() && e == cudaSuccess; ++k) {
    const auto& b = p->batches[k];
    float* out_norm = k == 0 ? norm : nullptr;
    e = (int)b.index.size() <= clip::kSmallTable
            ? launch_scale<clip::kSmallTable>(*p, b, grads, to, part, max_norm, out_norm, alone, s)
            : launch_scale<clip::kTable>(*p, b, grads, to, part, max_norm, out_norm, alone, s);
  }
  if (e == cudaSuccess && p->batches.empty()) e = cudaMemsetAsync(norm, 0, sizeof(float), s);
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "clip_apply");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

const char* lapl_clip_last_error(lapl_clip_handle p) { return p ? p->last_error : ""; }

lapl_status lapl_clip_destroy(lapl_clip_handle p) {
  delete p;
  return LAPL_OK;
}

}  // extern "C"
