// adamw.cu -- AdamW over many tensors in one launch: lapl_adamw_* of include/lapl_ops.h.
//
// The tensors are cut into pieces of whole 256-value blocks; the table of tensors travels as a kernel
// parameter, for up to kTable tensors a launch.  CTA b takes pieces b, b + grid, ...; a warp takes a
// block: a lane has values 4 lane .. 4 lane + 3 of each half, so that every access of a warp is one
// run of memory, and a block's largest value is one reduction over the warp.  Blocks that end early
// and tensors off 16 bytes (8-bit states: off 4) go value by value, lane by lane.
// HBM-bound: every value's weight, gradient and states are read and written once (28 bytes with fp32
// states, 16 with 8-bit ones, of fp32 weights).  Measured, of 6.8 TB/s, from HBM: 2^20 fp32 values in 24 tensors 9.4 us
// (3.1 TB/s: one round of loads, that of the table among them); with fp32 states 2^26 fp32 weights 297 us and 2^26
// bf16 ones with masters 299 (6.3 TB/s); 2^27 bf16 weights with masters and 8-bit states 450 us (4.8 TB/s), with
// instructions issued in three quarters of the cycles: roots, divisions and conversions of 8-bit states.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "ops_common.cuh"

namespace lapl {
namespace adamw {

constexpr int kThreads = 256;
constexpr int kBlock = LAPL_ADAMW_BLOCK;
constexpr int kPer = kBlock / 32;    // values of a lane
constexpr int kTable = 400;          // tensors of a launch: 29 KB of its 32 KB of parameters
constexpr int kSmallTable = 64;
constexpr int kMinPiece = 2048, kMaxPiece = 32768;   // values, powers of two
constexpr int kStart = 2048;         // values that a CTA streams while it starts on a piece
constexpr int kCtas = 4;             // of an SM
constexpr float kF8Max = 448.f, kF8Least = 0.001953125f;   // e4m3's largest and smallest
constexpr float kAmaxFloor = 7.888609052210118e-31f;       // 2^-100

template <int N>
struct Table {
  void* param[N];
  const void* grad[N];
  float* master[N];
  void* m[N];
  void* v[N];
  float* m_scale[N];
  float* v_scale[N];
  float weight_decay[N];
  int first[N + 1];     // first piece of each tensor, and the number of pieces
  int last[N];          // values of its last piece
  unsigned char kind[N];   // bit 0: bf16 parameter, bit 1: bf16 gradient, bit 2: whole vectors
  int tensors;
  int piece;            // values of the others
};

struct Step {
  float beta1, beta2, one_beta1, one_beta2;   // 1 - beta rounded from double
  float eps, down_by;   // the update's divisors are held times down_by, eps among them
  double log_beta1, log_beta2;
  float lr, late1, late2;        // late: 1 - beta^t
  const float* lr_device;
  const long long* step_device;
  const float* norm;
  float max_norm;
};

// What a lane holds of a block.
struct Lane {
  float w[kPer], g[kPer], m[kPer], v[kPer];
};

// Value i of a lane's: in fours, or one by one.
template <bool kVector>
__device__ __forceinline__ int place(int i, int lane) {
  return kVector ? (i >> 2) * 128 + lane * 4 + (i & 3) : i * 32 + lane;
}

template <bool kVector>
__device__ __forceinline__ void load_f32(float (&x)[kPer], const float* p, int lane, int n) {
#pragma unroll
  for (int i = 0; i < kPer; i += kVector ? 4 : 1) {
    const int at = place<kVector>(i, lane);
    if constexpr (kVector) {
      const float4 f = *reinterpret_cast<const float4*>(p + at);
      x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
    } else {
      x[i] = at < n ? p[at] : 0.f;
    }
  }
}
template <bool kVector>
__device__ __forceinline__ void load_bf16(float (&x)[kPer], const uint16_t* p, int lane, int n) {
#pragma unroll
  for (int i = 0; i < kPer; i += kVector ? 4 : 1) {
    const int at = place<kVector>(i, lane);
    if constexpr (kVector) {
      const uint2 f = *reinterpret_cast<const uint2*>(p + at);
      x[i] = bf16_lo(f.x), x[i + 1] = bf16_hi(f.x), x[i + 2] = bf16_lo(f.y), x[i + 3] = bf16_hi(f.y);
    } else {
      x[i] = at < n ? ops::bf16_bits(p[at]) : 0.f;
    }
  }
}
// e4m3 codes as floats.
__device__ __forceinline__ float2 decode2(uint16_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint16_t encode2(float lo, float hi) {
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(hi), "f"(lo));
  return two;
}
template <bool kVector>
__device__ __forceinline__ void load_f8(float (&x)[kPer], const uint8_t* p, int lane, int n) {
#pragma unroll
  for (int i = 0; i < kPer; i += kVector ? 4 : 1) {
    const int at = place<kVector>(i, lane);
    if constexpr (kVector) {
      const uint32_t f = *reinterpret_cast<const uint32_t*>(p + at);
      const float2 a = decode2((uint16_t)f), b = decode2((uint16_t)(f >> 16));
      x[i] = a.x, x[i + 1] = a.y, x[i + 2] = b.x, x[i + 3] = b.y;
    } else {
      x[i] = at < n ? decode2(p[at]).x : 0.f;
    }
  }
}
template <bool kVector>
__device__ __forceinline__ void store_f32(float* p, const float (&x)[kPer], int lane, int n) {
#pragma unroll
  for (int i = 0; i < kPer; i += kVector ? 4 : 1) {
    const int at = place<kVector>(i, lane);
    if constexpr (kVector) {
      *reinterpret_cast<float4*>(p + at) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else if (at < n) {
      p[at] = x[i];
    }
  }
}
template <bool kVector>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&x)[kPer], int lane, int n) {
#pragma unroll
  for (int i = 0; i < kPer; i += kVector ? 4 : 1) {
    const int at = place<kVector>(i, lane);
    if constexpr (kVector) {
      *reinterpret_cast<uint2*>(p + at) =
          make_uint2(ops::pack_bf16(x[i], x[i + 1]), ops::pack_bf16(x[i + 2], x[i + 3]));
    } else if (at < n) {
      p[at] = (uint16_t)ops::pack_bf16(x[i], 0.f);
    }
  }
}

// Largest absolute value of the warp's, and at least `least`; a NaN among them wins, as its bits are larger
// than any number's.
__device__ __forceinline__ float block_max(const float (&x)[kPer], float least) {
  unsigned top = __float_as_uint(least);
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}
__device__ __forceinline__ float fast_sqrt(float v) {   // off by a unit
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// x, or with kRoot the root of x, as codes with a scale; kRoot: what is above zero gets a code above zero.
// Where x / scale falls is clear from x (or its root, off by a unit) times the scale's reciprocal, off by 4
// units together at most, but next to the middle between two codes, and where codes have fewer bits: there
// the root and the division are formed exactly.  (For each code they were half of the kernel's
// instructions, whose issue bounds it: 2^27 values 490 us and 715, root and divisions for each, before
// blocks were fetched ahead.)
template <bool kVector, bool kRoot>
__device__ __forceinline__ void store_f8(uint8_t* p, float* scale_at, const float (&x)[kPer],
                                         const float (&root)[kPer], int lane, int n) {
  // The root of the largest is the largest root.
  const float top = block_max(x, kRoot ? 0.f : kAmaxFloor);
  // (The root of anything above zero is above the floor.)
  const float most = !kRoot ? top : top > 0.f ? __fsqrt_rn(top) : isnan(top) ? top : kAmaxFloor;
  const float scale = __fmul_rn(most, 1.f / kF8Max);
  if (lane == 0) *scale_at = scale;
  const float inverse = 1.f / scale;   // (scale is at least 2^-109)
  float q[kPer];
  bool exactly = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = (kRoot ? root[i] : x[i]) * inverse;
    const int off = (int)(__float_as_uint(q[i]) & 0xFFFFFu) - (0x80000 - 8);
    exactly |= (unsigned)off <= 16u || (q[i] != 0.f && fabsf(q[i]) < 0.015626f);
  }
  if (exactly) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) q[i] = __fdiv_rn(kRoot ? __fsqrt_rn(x[i]) : x[i], scale);
  }
  if (kRoot) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (x[i] > 0.f) q[i] = fmaxf(q[i], kF8Least);
  }
#pragma unroll
  for (int i = 0; i < kPer; i += kVector ? 4 : 1) {
    const int at = place<kVector>(i, lane);
    if constexpr (kVector) {
      *reinterpret_cast<uint32_t*>(p + at) =
          (uint32_t)encode2(q[i], q[i + 1]) | (uint32_t)encode2(q[i + 2], q[i + 3]) << 16;
    } else if (at < n) {
      p[at] = (uint8_t)encode2(q[i], 0.f);
    }
  }
}

// A lane's 8 of the values from `at` on, into L2.
__device__ __forceinline__ void prefetch(const void* p, long long at, int bytes, int lane) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const unsigned char*>(p) +
                                                (at + kPer * lane) * bytes));
}

// The block of n values (256 of kVector) that starts at value `at` of a tensor; block: its number.
template <bool k8, bool kVector, int N>
__device__ __forceinline__ void update(const Table<N>& t, int k, long long at, long long block, int n,
                                       const Step& s, float clip, float a, float root, float keep) {
  const int lane = threadIdx.x & 31;
  const bool half = t.kind[k] & 1, grad_half = t.kind[k] & 2;
  float* master = t.master[k];
  Lane x;
  if (master) load_f32<kVector>(x.w, master + at, lane, n);
  else if (half) load_bf16<kVector>(x.w, static_cast<const uint16_t*>(t.param[k]) + at, lane, n);
  else load_f32<kVector>(x.w, static_cast<const float*>(t.param[k]) + at, lane, n);
  if (grad_half) load_bf16<kVector>(x.g, static_cast<const uint16_t*>(t.grad[k]) + at, lane, n);
  else load_f32<kVector>(x.g, static_cast<const float*>(t.grad[k]) + at, lane, n);
  float m_scale = 1.f, v_scale = 1.f;
  if constexpr (k8) {
    m_scale = t.m_scale[k][block];
    v_scale = t.v_scale[k][block];
    load_f8<kVector>(x.m, static_cast<const uint8_t*>(t.m[k]) + at, lane, n);
    load_f8<kVector>(x.v, static_cast<const uint8_t*>(t.v[k]) + at, lane, n);
  } else {
    load_f32<kVector>(x.m, static_cast<const float*>(t.m[k]) + at, lane, n);
    load_f32<kVector>(x.v, static_cast<const float*>(t.v[k]) + at, lane, n);
  }
  float r[kPer];
  // The states' products and sums are rounded one by one, as the formulas read, and not contracted: a code
  // next to a border must not depend on how a compiler joins them.  (Packed instructions of two values do
  // get joined.)
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if constexpr (k8) {
      x.m[i] = __fmul_rn(x.m[i], m_scale);
      x.v[i] = __fmul_rn(x.v[i], v_scale);
      x.v[i] = __fmul_rn(x.v[i], x.v[i]);
    }
    const float g = __fmul_rn(x.g[i], clip);
    x.m[i] = __fadd_rn(__fmul_rn(s.beta1, x.m[i]), __fmul_rn(s.one_beta1, g));
    x.v[i] = __fadd_rn(__fmul_rn(s.beta2, x.v[i]), __fmul_rn(__fmul_rn(s.one_beta2, g), g));
    r[i] = fast_sqrt(x.v[i]);
    // lr m / late1 / (sqrt(v / late2) + eps), with a = lr / late1 and root = 1 / sqrt(late2), both times
    // down_by.  (Root and quotient, off by 2 units each, are the step's alone: no state is made of them.  The
    // quotient by more than 2^126 would be zero.)
    x.w[i] = x.w[i] * keep - __fdividef(a * x.m[i], fmaf(r[i], root, s.eps));
  }
  if (master) store_f32<kVector>(master + at, x.w, lane, n);
  if (half) store_bf16<kVector>(static_cast<uint16_t*>(t.param[k]) + at, x.w, lane, n);
  else store_f32<kVector>(static_cast<float*>(t.param[k]) + at, x.w, lane, n);
  if constexpr (k8) {
    store_f8<kVector, false>(static_cast<uint8_t*>(t.m[k]) + at, t.m_scale[k] + block, x.m, r, lane, n);
    store_f8<kVector, true>(static_cast<uint8_t*>(t.v[k]) + at, t.v_scale[k] + block, x.v, r, lane, n);
  } else {
    store_f32<kVector>(static_cast<float*>(t.m[k]) + at, x.m, lane, n);
    store_f32<kVector>(static_cast<float*>(t.v[k]) + at, x.v, lane, n);
  }
}

// Weights, gradients and codes of a whole block with 8-bit states, into L2, while a block is worked on, which
// registers have no room for.  (2^27 bf16 weights 450 us and 490 without.  With fp32 states, which wait for
// bandwidth and not for latency: 2^26 values 320 us and 295
// without; with the scales 470.)
template <int N>
__device__ __forceinline__ void fetch(const Table<N>& t, int k, long long at) {
  const int lane = threadIdx.x & 31;
  if (t.master[k]) prefetch(t.master[k], at, 4, lane);
  else prefetch(t.param[k], at, t.kind[k] & 1 ? 2 : 4, lane);
  prefetch(t.grad[k], at, t.kind[k] & 2 ? 2 : 4, lane);
  prefetch(t.m[k], at, 1, lane);
  prefetch(t.v[k], at, 1, lane);
}

template <bool k8, int N>
__global__ void __launch_bounds__(kThreads, kCtas)
adamw_kernel(const __grid_constant__ Table<N> t, const __grid_constant__ Step s) {
  float clip = 1.f;
  if (s.norm) {
    const float norm = *s.norm;
    if (!isfinite(norm)) return;
    // (Norms below 2^-128 have no reciprocal.)
    const float inverse = 1.f / norm;
    if (norm > s.max_norm) clip = isfinite(inverse) ? s.max_norm * inverse : s.max_norm / norm;
  }
  const float lr = s.lr_device ? *s.lr_device : s.lr;
  float late1 = s.late1, late2 = s.late2;
  if (s.step_device) {
    // 1 - beta^t = -expm1(t ln beta), the product in double.
    const double step = (double)*s.step_device;
    late1 = -expm1f((float)(step * s.log_beta1));
    late2 = -expm1f((float)(step * s.log_beta2));
  }
  const float a = lr / late1 * s.down_by, root = s.down_by / sqrtf(late2);
  const int pieces = t.first[t.tensors];
  const int warp = threadIdx.x >> 5;
  for (int i = blockIdx.x; i < pieces; i += gridDim.x) {
    int lo = 0, hi = t.tensors;   // first[lo] <= i < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (t.first[mid] <= i) lo = mid; else hi = mid;
    }
    const long long start = (long long)(i - t.first[lo]) * t.piece;
    const int count = i + 1 == t.first[lo + 1] ? t.last[lo] : t.piece;
    const float keep = 1.f - lr * t.weight_decay[lo];
    const bool vector = t.kind[lo] & 4;
    for (int b = warp * kBlock; b < count; b += kThreads / 32 * kBlock) {
      const int n = min(kBlock, count - b);
      if (k8 && b + kThreads / 32 * kBlock + kBlock <= count)
        fetch(t, lo, start + b + kThreads / 32 * kBlock);
      if (vector && n == kBlock)
        update<k8, true>(t, lo, start + b, (start + b) / kBlock, n, s, clip, a, root, keep);
      else
        update<k8, false>(t, lo, start + b, (start + b) / kBlock, n, s, clip, a, root, keep);
    }
  }
}

}  // namespace adamw
}  // namespace lapl

struct lapl_adamw_plan {
  std::vector<long long> counts;
  std::vector<int> dtypes, grad_dtypes;
  std::vector<float> weight_decay;
  lapl::adamw::Step step;
  double beta1, beta2;
  bool f8;
  struct Batch {       // the tensors of one launch
    std::vector<int> index;   // those with values
    int piece;                // values of a piece
    int pieces, grid;
  };
  std::vector<Batch> batches;
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;   // scratch of the overlap check
  int device;
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

lapl_status validate(const lapl_adamw_config* c) {
  if (!c || c->tensors < 0) return LAPL_ERR_INVALID_ARG;
  if (c->tensors > 0 && (!c->counts || !c->dtypes || !c->grad_dtypes || !c->weight_decay))
    return LAPL_ERR_INVALID_ARG;
  if (!(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0))
    return LAPL_ERR_INVALID_ARG;
  if (!((float)c->eps > 0.f) || !std::isfinite((float)c->eps)) return LAPL_ERR_INVALID_ARG;
  if (c->state_bits != 32 && c->state_bits != 8) return LAPL_ERR_INVALID_ARG;
  for (int i = 0; i < c->tensors; ++i) {
    if (c->counts[i] < 0 || !ops::is_float_dtype(c->dtypes[i]) ||
        !ops::is_float_dtype(c->grad_dtypes[i]))
      return LAPL_ERR_INVALID_ARG;
    if (!(c->weight_decay[i] >= 0.f) || !std::isfinite(c->weight_decay[i]))
      return LAPL_ERR_INVALID_ARG;
    if (c->counts[i] > (1LL << 40)) return LAPL_ERR_UNSUPPORTED;
  }
  return LAPL_OK;
}

// 1 - beta^t.
double late(double beta, long long t) { return -std::expm1((double)t * std::log(beta)); }

void create(const lapl_adamw_config* cfg, int sms, lapl_adamw_plan* p) {
  const int T = cfg->tensors;
  p->counts.assign(cfg->counts, cfg->counts + T);
  p->dtypes.assign(cfg->dtypes, cfg->dtypes + T);
  p->grad_dtypes.assign(cfg->grad_dtypes, cfg->grad_dtypes + T);
  p->weight_decay.assign(cfg->weight_decay, cfg->weight_decay + T);
  p->spans.reserve(7 * (size_t)T + 3);
  p->f8 = cfg->state_bits == 8;
  // In double: 1 - beta of a float near 1 would have few bits (0.999f is 1 - 0.00100005).
  p->beta1 = cfg->beta1;
  p->beta2 = cfg->beta2;
  adamw::Step& s = p->step;
  s = {};
  s.beta1 = (float)cfg->beta1;
  s.beta2 = (float)cfg->beta2;
  s.one_beta1 = (float)(1.0 - p->beta1);
  s.one_beta2 = (float)(1.0 - p->beta2);
  s.log_beta1 = std::log(p->beta1);
  s.log_beta2 = std::log(p->beta2);
  // Roots are below 2^64, and with their correction below 2^91.
  s.down_by = (float)cfg->eps > 0x1p62f ? 0x1p-64f : 1.f;
  s.eps = (float)cfg->eps * s.down_by;
  long long pieces = 0;
  for (int i = 0; i < T; ++i) {
    if (p->counts[i] == 0) continue;
    const long long more = (p->counts[i] - 1) / adamw::kMaxPiece + 1;
    if (p->batches.empty() || (int)p->batches.back().index.size() == adamw::kTable ||
        pieces + more > (1LL << 30)) {
      p->batches.emplace_back();
      pieces = 0;
    }
    p->batches.back().index.push_back(i);
    pieces += more;
  }
  const long long ctas = (long long)adamw::kCtas * sms;
  for (auto& b : p->batches) {
    // The piece with the least on the longest path: rounds of pieces, and starting on each.
    long long best = 0;
    for (int piece = adamw::kMaxPiece; piece >= adamw::kMinPiece; piece /= 2) {
      long long n = 0;
      for (const int i : b.index) n += (p->counts[i] - 1) / piece + 1;
      const long long cost = (n + ctas - 1) / ctas * (piece + adamw::kStart);
      if (best != 0 && (cost >= best || n > (1LL << 30))) continue;
      best = cost;
      b.piece = piece;
      b.pieces = (int)n;
    }
    b.grid = (int)std::min<long long>(b.pieces, ctas);
  }
}

struct Arrays {
  void* const* params;
  const void* const* grads;
  float* const* masters;
  void* const* m;
  void* const* v;
  float* const* m_scales;
  float* const* v_scales;
  float* master(int i) const { return masters ? masters[i] : nullptr; }
};

template <int N>
void fill(const lapl_adamw_plan& p, const lapl_adamw_plan::Batch& b, const Arrays& a,
          adamw::Table<N>* t) {
  int first = 0, k = 0;
  for (const int i : b.index) {
    t->param[k] = a.params[i];
    t->grad[k] = a.grads[i];
    t->master[k] = a.master(i);
    t->m[k] = a.m[i];
    t->v[k] = a.v[i];
    t->m_scale[k] = p.f8 ? a.m_scales[i] : nullptr;
    t->v_scale[k] = p.f8 ? a.v_scales[i] : nullptr;
    t->weight_decay[k] = p.weight_decay[i];
    t->first[k] = first;
    const long long pieces = (p.counts[i] - 1) / b.piece + 1;
    first += (int)pieces;
    t->last[k] = (int)(p.counts[i] - (pieces - 1) * b.piece);
    const bool half = p.dtypes[i] == LAPL_BF16, grad_half = p.grad_dtypes[i] == LAPL_BF16;
    const bool vector = ops::aligned(a.params[i], half ? 8 : 16) &&
                        ops::aligned(a.grads[i], grad_half ? 8 : 16) &&
                        ops::aligned(a.master(i), 16) && ops::aligned(a.m[i], p.f8 ? 4 : 16) &&
                        ops::aligned(a.v[i], p.f8 ? 4 : 16);
    t->kind[k] = (unsigned char)(half | grad_half << 1 | vector << 2);
    ++k;
  }
  t->first[k] = first;
  t->tensors = k;
  t->piece = b.piece;
}

template <int N>
cudaError_t launch(const lapl_adamw_plan& p, const lapl_adamw_plan::Batch& b, const Arrays& a,
                   const adamw::Step& s, cudaStream_t st) {
  adamw::Table<N> t;
  fill(p, b, a, &t);
  if (p.f8) adamw::adamw_kernel<true, N><<<b.grid, adamw::kThreads, 0, st>>>(t, s);
  else adamw::adamw_kernel<false, N><<<b.grid, adamw::kThreads, 0, st>>>(t, s);
  return cudaGetLastError();
}

// scalars: lr_device, step_device and norm, which every CTA reads whenever it starts.
lapl_status check_arrays(lapl_adamw_plan* p, const Arrays& a, const void* const (&scalars)[3]) {
  auto& spans = p->spans;
  spans.clear();
  // A written span's end is odd-tagged: spans are doubled to make room for the tag.
  auto add = [&](const void* at, long long n, int size, bool written) {
    if (!at) return LAPL_ERR_INVALID_ARG;
    if (!ops::aligned(at, size)) return LAPL_ERR_ALIGNMENT;
    spans.emplace_back((uintptr_t)at, ((uintptr_t)at + (uintptr_t)n * size) * 2 + written);
    return LAPL_OK;
  };
  for (int i = 0; i < 3; ++i)
    if (scalars[i]) {
      const lapl_status st = add(scalars[i], 1, i == 1 ? 8 : 4, false);
      if (st != LAPL_OK) return st;
    }
  for (size_t i = 0; i < p->counts.size(); ++i) {
    const long long n = p->counts[i];
    if (n == 0) continue;
    lapl_status st = add(a.params[i], n, ops::dtype_bytes(p->dtypes[i]), true);
    if (st == LAPL_OK) st = add(a.grads[i], n, ops::dtype_bytes(p->grad_dtypes[i]), false);
    if (st == LAPL_OK && a.master((int)i)) st = add(a.master((int)i), n, 4, true);
    if (st == LAPL_OK) st = add(a.m[i], n, p->f8 ? 1 : 4, true);
    if (st == LAPL_OK) st = add(a.v[i], n, p->f8 ? 1 : 4, true);
    if (p->f8) {
      const long long blocks = (n - 1) / adamw::kBlock + 1;
      if (st == LAPL_OK) st = add(a.m_scales[i], blocks, 4, true);
      if (st == LAPL_OK) st = add(a.v_scales[i], blocks, 4, true);
    }
    if (st != LAPL_OK) return st;
  }
  std::sort(spans.begin(), spans.end());
  uintptr_t end = 0, written_end = 0;   // furthest end so far, of all spans and of written ones
  for (const auto& s : spans) {
    const bool written = s.second & 1;
    if (s.first < (written ? end : written_end)) return LAPL_ERR_INVALID_ARG;
    end = std::max(end, s.second / 2);
    if (written) written_end = std::max(written_end, s.second / 2);
  }
  return LAPL_OK;
}

}  // namespace

extern "C" {

lapl_status lapl_adamw_create(const lapl_adamw_config* cfg, lapl_adamw_handle* out) {
  if (!out) return LAPL_ERR_INVALID_ARG;
  *out = nullptr;
  const lapl_status st = validate(cfg);
  if (st != LAPL_OK) return st;
  int sms = 0, device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return LAPL_ERR_CUDA;
  lapl_adamw_plan* p = nullptr;
  try {
    p = new lapl_adamw_plan();
    p->device = device;
    create(cfg, sms, p);
  } catch (const std::exception&) {   // out of host memory
    delete p;
    return LAPL_ERR_INVALID_ARG;
  }
  *out = p;
  return LAPL_OK;
}

lapl_status lapl_adamw_step(lapl_adamw_handle p, void* const* params, const void* const* grads,
                            float* const* masters, void* const* m, void* const* v,
                            float* const* m_scales, float* const* v_scales, float lr,
                            const float* lr_device, long long step, const long long* step_device,
                            const float* norm, float max_norm, void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  if (!p->counts.empty()) {
    if (!params || !grads || !m || !v) return LAPL_ERR_INVALID_ARG;
    if (p->f8 != (m_scales != nullptr) || p->f8 != (v_scales != nullptr)) return LAPL_ERR_INVALID_ARG;
  }
  if (!lr_device && !std::isfinite(lr)) return LAPL_ERR_INVALID_ARG;
  if (!step_device && step < 1) return LAPL_ERR_INVALID_ARG;
  if (norm && (!(max_norm >= 0.f) || !std::isfinite(max_norm))) return LAPL_ERR_INVALID_ARG;
  const Arrays a = {params, grads, masters, m, v, m_scales, v_scales};
  lapl_status st = check_arrays(p, a, {lr_device, step_device, norm});
  if (st != LAPL_OK) return st;
  st = ops::check_device(p->device, p->last_error, "adamw_step/device");
  if (st != LAPL_OK) return st;
  adamw::Step s = p->step;
  s.lr = lr;
  s.lr_device = lr_device;
  s.step_device = step_device;
  if (!step_device) {
    s.late1 = (float)late(p->beta1, step);
    s.late2 = (float)late(p->beta2, step);
  }
  s.norm = norm;
  s.max_norm = max_norm;
  cudaError_t e = cudaSuccess;
  for (const auto& b : p->batches) {
    e = (int)b.index.size() <= adamw::kSmallTable
            ? launch<adamw::kSmallTable>(*p, b, a, s, static_cast<cudaStream_t>(stream))
            : launch<adamw::kTable>(*p, b, a, s, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) break;
  }
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "adamw_step");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

const char* lapl_adamw_last_error(lapl_adamw_handle p) { return p ? p->last_error : ""; }

lapl_status lapl_adamw_destroy(lapl_adamw_handle p) {
  delete p;
  return LAPL_OK;
}

}  // extern "C"
