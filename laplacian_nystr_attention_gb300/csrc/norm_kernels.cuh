// norm_kernels.cuh -- residual addition + root-mean-square norm (lapl_norm_* of
// include/lapl_ops.h): what its kernels share, and the forward kernel, compiled for each output type
// by norm_f32.cu, norm_bf16.cu and norm_f8.cu.
//
// Per row (token) of W = H d values, s = x + residual:
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
// and backward, with t = dy w and n = s rstd,
//   d = rstd (t - n mean(t n)) + dsum,  dw = sum over rows dy n.
//
// Every value is read once and held in registers between the row's sum and its use.  A row
// belongs to G threads, each with NV vectors of 8 values, vector j of thread t at columns
// (j G + t) 8: whole 16- or 32-byte pieces, neighbours side by side.  G up to 32 is a power of two,
// with several rows side by side in a CTA, each summed by shuffles alone; a longer row has a CTA of
// whole warps to itself and is summed through shared memory.  The CTAs are as many
// as the GPU holds and go through the rows in strides, so a thread's columns stay its own: its
// weights and its part of dweight are in registers, and the next row's values are on their way
// while this row is summed and written.
// x comes head by head ([B,H,N,d]); a vector never straddles a head (d a multiple of 8), so
// merging the heads costs only where the pieces are read from.
// Rows of a length that is no multiple of 8 start anywhere among the vectors of the whole tensor.
// There a CTA takes only rows that start at the same place, every 8th, 4th or 2nd one, so its threads'
// columns still stay their own; a row's first and last vector are shared with its neighbours and
// written value by value, and heads of such a length are read and written so.  What is left (a
// pointer off 16 bytes) runs with vectors of one value, a row to a CTA.
//
// HBM-bound.  Measured (of 6.78 TB/s): the attention's fp32 output at 4 x 8 x 16384 x 64 with a bf16
// residual 52 us (6.5 TB/s, 95%); rows of 4096 bf16 values to e4m3 by groups of 128 38.3 us (91%; a
// value's conversions and division keep issue at 68%).
#pragma once

#include "ops_common.cuh"

namespace lapl {
namespace norm {

constexpr int kMaxWidth = 16384;
constexpr int kThreads = 256;        // of a CTA whose rows have at most as many
constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100
constexpr float kE4m3Max = 448.f;

constexpr int kMaxThreads = 512;

// Division by an invariant (Granlund and Montgomery): l = ceil(log2 n),
// mul = floor(2^32 (2^l - n) / n) + 1, v / n = (umulhi(mul, v) + v) >> l for v below 2^31.
struct Divisor {
  unsigned mul;
  int shift;
  __device__ __forceinline__ unsigned operator()(unsigned v) const {
    return (__umulhi(mul, v) + v) >> shift;
  }
};

struct Args {
  const void* x;        // forward: [B,H,N,d]
  const void* res;      // forward: residual; backward: sum
  const float* weight;
  void* sum;
  float* rstd;
  void* y;
  float* scales;
  const void* dy;
  const void* dsum;
  void* dx;
  void* dres;
  float* part;          // [CTAs, W] partial dweight
  unsigned rows;
  int period;           // rows r, r + period, ... start at the same place among the vectors
  int n, d, heads, width;
  Divisor by_n, by_d;
  int g;                // threads of a row
  int per_log2;         // rows side by side in a CTA (one where g > 32)
  int group_log2;       // values that share a scale, -1: the whole row
  float eps, inv_width;
};

// Offset of a row's head 0 in [B,H,N,d], and of a column's head and channel from there.
__device__ __forceinline__ long long head_row(const Args& a, unsigned row) {
  if (a.heads == 1) return (long long)row * a.width;
  const unsigned b = a.by_n(row);
  return (long long)b * a.n * a.width + (long long)(row - b * a.n) * a.d;
}
__device__ __forceinline__ long long head_col(const Args& a, int col) {
  if (a.heads == 1) return col;
  const int h = (int)a.by_d((unsigned)col);
  return (long long)h * a.n * a.d + (col - h * a.d);
}

// VEC values as they lie in memory (VEC = 8 or 1), and widened.
template <bool k16, int VEC>
struct Raw {
  uint32_t w[VEC == 8 ? (k16 ? 4 : 8) : 1];
};
template <bool k16, int VEC>
__device__ __forceinline__ void load(Raw<k16, VEC>& r, const void* base, long long e) {
  if constexpr (VEC == 8) {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) +
                                                    e * (k16 ? 2 : 4));
    const uint4 a = *p;
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    if constexpr (!k16) {
      const uint4 b = p[1];
      r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    }
  } else if constexpr (k16) {
    r.w[0] = reinterpret_cast<const uint16_t*>(base)[e];
  } else {
    r.w[0] = reinterpret_cast<const uint32_t*>(base)[e];
  }
}
template <bool k16, int VEC>
__device__ __forceinline__ void zero(Raw<k16, VEC>& r) {
#pragma unroll
  for (uint32_t& w : r.w) w = 0u;
}
// Value i alone: set to zero, or loaded (for VEC = 8, into a vector of zeros).
template <bool k16, int VEC>
__device__ __forceinline__ void clear(Raw<k16, VEC>& r, int i) {
  if constexpr (!k16) r.w[i] = 0u;
  else r.w[i / 2] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
}
template <bool k16, int VEC>
__device__ __forceinline__ void load_one(Raw<k16, VEC>& r, const void* base, long long e, int i) {
  if constexpr (!k16) r.w[i] = reinterpret_cast<const uint32_t*>(base)[e + i];
  else r.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(base)[e + i] << (16 * (i & 1));
}
// A vector of bf16 from shared memory.
__device__ __forceinline__ void read_copy(Raw<true, 8>& r, unsigned at) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(at) : "memory");
}

// Values are worked on two at a time (packed fp32 instructions), or one where vectors have one.
template <int VEC>
struct Values {
  static constexpr int kW = VEC == 8 ? 2 : 1, kN = VEC / kW;
  ops::Vec<kW> v[kN];
};
template <bool k16, int VEC>
__device__ __forceinline__ ops::Vec<Values<VEC>::kW> get(const Raw<k16, VEC>& r, int i) {
  ops::Vec<Values<VEC>::kW> v;
  if constexpr (VEC == 1) {
    v.f[0] = k16 ? bf16_lo(r.w[0]) : __uint_as_float(r.w[0]);
  } else if constexpr (k16) {
    v.f[0] = bf16_lo(r.w[i]);
    v.f[Values<VEC>::kW - 1] = bf16_hi(r.w[i]);
  } else {
    v.f[0] = __uint_as_float(r.w[2 * i]);
    v.f[Values<VEC>::kW - 1] = __uint_as_float(r.w[2 * i + 1]);
  }
  return v;
}
template <int VEC>
__device__ __forceinline__ float at(const Values<VEC>& x, int i) {
  return x.v[i / Values<VEC>::kW].f[i % Values<VEC>::kW];
}
template <bool k16, int VEC>
__device__ __forceinline__ void store(void* base, long long e, const Values<VEC>& x) {
  if constexpr (VEC == 8) {
    uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<char*>(base) + e * (k16 ? 2 : 4));
    if constexpr (k16) {
      *p = make_uint4(ops::pack_bf16(at(x, 0), at(x, 1)), ops::pack_bf16(at(x, 2), at(x, 3)),
                      ops::pack_bf16(at(x, 4), at(x, 5)), ops::pack_bf16(at(x, 6), at(x, 7)));
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(at(x, 0), at(x, 1), at(x, 2), at(x, 3));
      reinterpret_cast<float4*>(p)[1] = make_float4(at(x, 4), at(x, 5), at(x, 6), at(x, 7));
    }
  } else if constexpr (k16) {
    reinterpret_cast<uint16_t*>(base)[e] = (uint16_t)ops::pack_bf16(at(x, 0), 0.f);
  } else {
    reinterpret_cast<float*>(base)[e] = at(x, 0);
  }
}

// The larger one, or NaN if either is.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum or largest over the G threads of a row, the same value in each.  `scratch`: one float for
// each warp of the CTA, of this reduction alone until the next __syncthreads.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, int g, float* scratch) {
  for (int o = min(g, 32) >> 1; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? larger(v, other) : v + other;
  }
  if (g > 32) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (g >> 5) ? scratch[lane] : 0.f;     // sums and largest magnitudes: 0 changes neither
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, v, o);
      v = kMax ? larger(v, other) : v + other;
    }
  }
  return v;
}

// A thread's place in its row, and its row's in the CTA.
__device__ __forceinline__ int place_in_row(const Args& a) {
  return a.g > 32 ? (int)threadIdx.x : (int)threadIdx.x & (a.g - 1);
}
__device__ __forceinline__ unsigned row_in_cta(const Args& a) {
  return a.g > 32 ? 0u : threadIdx.x / (unsigned)a.g;
}

// The e4m3 values of up to 8 floats, in bytes.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo =
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi =
      __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// v / by from inv, 1 / by rounded to nearest: the product, and what is left of v by a fused step, which
// corrects it (Markstein's division).  y times 1 / scale alone, or times 448 / largest, would put
// values near the middle of two e4m3 ones on the wrong side.
__device__ __forceinline__ float quotient(float v, float by, float inv) {
  const float q = v * inv;
  return fmaf(fmaf(-by, q, v), inv, q);
}
template <int V>
__device__ __forceinline__ ops::Vec<V> quotient(const ops::Vec<V>& v, float by, float inv) {
  const ops::Vec<V> q = ops::mul(v, ops::fill<V>(inv));
  return ops::fma(ops::fma(ops::fill<V>(-by), q, v), ops::fill<V>(inv), q);
}

// A row's values one after the other where the heads' lengths are no multiple of 8.
struct Walk {
  long long at;
  int left;   // of the head
  __device__ __forceinline__ Walk(const Args& a, long long row, int col) {
    const unsigned c = (unsigned)max(col, 0), h = a.by_d(c);
    at = row + (long long)h * a.n * a.d + (c - h * a.d);
    left = a.d - (int)(c - h * a.d);
  }
  __device__ __forceinline__ long long next(const Args& a) {
    const long long now = at;
    ++at;
    if (--left == 0) {
      left = a.d;
      at += (long long)(a.n - 1) * a.d;
    }
    return now;
  }
};

// Shared memory of a thread for its weights.
constexpr int weight_bytes(int vec, int nv) { return vec == 8 && nv > 2 ? nv * 32 : 0; }

// A thread's columns: vector j is columns col(j) .. col(j) + VEC - 1, of which those from 0 to W - 1
// are the row's (kShift: col(0) of thread 0 is -shift).
template <int VEC, int NV, bool kShift>
struct Columns {
  static constexpr bool kHeads = VEC == 8 && !kShift;
  // Weights in registers, or (longer rows) in shared memory, a thread's 16-byte pieces beside its
  // neighbours' (read from global memory for each row: 2^24 bf16 values in rows of 8191 forward 63
  // instead of 33 us).
  static constexpr bool kWeights = NV * VEC <= 16, kShared = !kWeights && VEC == 8;
  int first, step, width;
  long long place[kHeads ? NV : 1];              // in [B,H,N,d]
  Values<VEC> w[kWeights ? NV : 1];
  unsigned shared;
  // room: of shared memory, weight_bytes(NV) for each of the CTA's threads.
  __device__ __forceinline__ void init(const Args& a, int t, int shift, void* room) {
    shared = kShared ? ops::smem_u32(room) + threadIdx.x * 16 : 0u;
    first = t * VEC - (kShift ? shift : 0);
    step = a.g * VEC;
    width = a.width;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (kHeads) place[j] = in(j) ? head_col(a, col(j)) : 0;
      if constexpr (kWeights)
#pragma unroll
        for (int i = 0; i < Values<VEC>::kN; ++i) w[j].v[i] = load_weight(a, j, i);
      if constexpr (kShared)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const auto lo = load_weight(a, j, 2 * k), hi = load_weight(a, j, 2 * k + 1);
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(piece(j, k)), "f"(lo.f[0]),
                       "f"(lo.f[1]), "f"(hi.f[0]), "f"(hi.f[1]) : "memory");
        }
    }
  }
  __device__ __forceinline__ int col(int j) const { return first + j * step; }
  __device__ __forceinline__ bool in(int j) const { return col(j) < width; }
  __device__ __forceinline__ bool valid(int j, int i) const {
    return kShift ? (unsigned)(col(j) + i) < (unsigned)width : in(j);
  }
  __device__ __forceinline__ bool whole(int j) const {
    return !kShift || (col(j) >= 0 && col(j) + VEC <= width);
  }
  __device__ __forceinline__ ops::Vec<Values<VEC>::kW> load_weight(const Args& a, int j, int i) const {
    constexpr int kW = Values<VEC>::kW;
    ops::Vec<kW> r;
#pragma unroll
    for (int k = 0; k < kW; ++k)
      r.f[k] = a.weight && valid(j, i * kW + k) ? __ldg(a.weight + col(j) + i * kW + k) : 1.f;
    return r;
  }
  __device__ __forceinline__ long long head(const Args& a, int j) const {
    if constexpr (kHeads) return place[j];
    else return head_col(a, col(j));
  }
  __device__ __forceinline__ unsigned piece(int j, int k) const {
    return shared + (2 * j + k) * blockDim.x * 16;
  }
  __device__ __forceinline__ Values<VEC> weights(const Args& a, int j) const {
    Values<VEC> r;
    if constexpr (kWeights) {
      r = w[j];
    } else if constexpr (kShared) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(r.v[2 * k].f[0]), "=f"(r.v[2 * k].f[1]), "=f"(r.v[2 * k + 1].f[0]),
                       "=f"(r.v[2 * k + 1].f[1]) : "r"(piece(j, k)) : "memory");
    } else {
      r.v[0] = load_weight(a, j, 0);
    }
    return r;
  }
  // Vector j at element e of a tensor that ends at `end`, with its neighbours' values where it is
  // not the row's (trim() clears them when the values are used: the load is not waited for here).
  template <bool k16>
  __device__ __forceinline__ void fetch(Raw<k16, VEC>& r, const void* base, int j, long long e,
                                        long long end) const {
    if (!kShift || e + VEC <= end) {
      load(r, base, e);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (valid(j, i)) load_one(r, base, e, i);
    }
  }
  // The same of a tensor by heads, whose row starts at element `row`.
  template <bool k16>
  __device__ __forceinline__ void gather(Raw<k16, VEC>& r, const void* base, const Args& a, int j,
                                         long long row, long long end) const {
    if (!kShift || a.heads == 1) {
      fetch(r, base, j, row + head(a, j), end);
    } else {
      Walk w(a, row, col(j));
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (valid(j, i)) load_one(r, base, w.next(a) - i, i);
    }
  }
  // The same of bf16 into shared memory; zeros where `on` is not set, and behind `end`.
  __device__ __forceinline__ void copy(unsigned to, const void* base, bool on, long long e,
                                       long long end) const {
    ops::copy16(to, reinterpret_cast<const char*>(base) + e * 2,
                on ? (int)max(0LL, min(8LL, end - e)) * 2 : 0);
  }
  template <bool k16>
  __device__ __forceinline__ void trim(Raw<k16, VEC>& r, int j) const {
    if (!whole(j)) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (!valid(j, i)) clear(r, i);
    }
  }
  template <bool k16>
  __device__ __forceinline__ void put(void* base, int j, long long e, const Values<VEC>& x) const {
    if (whole(j)) {
      store<k16, VEC>(base, e, x);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (valid(j, i)) store<k16, 1>(base, e + i, Values<1>{{{at(x, i)}}});
    }
  }
  template <bool k16>
  __device__ __forceinline__ void scatter(void* base, const Args& a, int j, long long row,
                                          const Values<VEC>& x) const {
    if (!kShift || a.heads == 1) {
      put<k16>(base, j, row + head(a, j), x);
    } else {
      Walk w(a, row, col(j));
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (valid(j, i)) store<k16, 1>(base, w.next(a), Values<1>{{{at(x, i)}}});
    }
  }
};

// The rows that a group of G threads goes through.
template <bool kShift>
struct Rows {
  unsigned row, first, stride;   // `first`: of the CTA's first group, the same for all its threads
  int shift;                     // place of the rows' start in their first vector
  __device__ __forceinline__ Rows(const Args& a) {
    const unsigned per = 1u << a.per_log2, mine = row_in_cta(a);
    if constexpr (kShift) {
      const unsigned p = (unsigned)a.period, k = blockIdx.x % p;
      first = k + blockIdx.x / p * per * p;
      row = first + mine * p;
      stride = gridDim.x * per;   // gridDim.x is a multiple of the period
      shift = (int)((unsigned long long)k * (unsigned)a.width & 7u);
    } else {
      first = blockIdx.x * per;
      row = first + mine;
      stride = gridDim.x * per;
      shift = 0;
    }
  }
};

enum Out { kF32, kBf16, kF8 };

template <bool kX16, bool kRes16, int kOut, int VEC, int NV, bool kShift>
__global__ void __launch_bounds__(kMaxThreads)
norm_forward_kernel(const Args a) {
  __shared__ float scratch[2][2][kMaxThreads / 32];
  extern __shared__ __align__(16) float room[];
  __shared__ float seg[VEC == 1 && kOut == kF8 ? 2 : 1][VEC == 1 && kOut == kF8 ? kMaxWidth / 32 : 1];
  // Registers for a row ahead: where a thread's part of a row is small.
  constexpr bool kAhead = NV * ((kX16 ? 4 : 8) + (kRes16 ? 4 : 8)) * VEC / 8 <= 32;
  const int t = place_in_row(a);
  Rows<kShift> rows(a);
  Columns<VEC, NV, kShift> cols;
  cols.init(a, t, rows.shift, room);
  const long long end = (long long)a.rows * a.width;
  Raw<kX16, VEC> rx[NV];
  Raw<kRes16, VEC> rr[NV];
  auto fetch = [&](unsigned r) {
    const long long xr = head_row(a, r), rr0 = (long long)r * a.width;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      zero(rx[j]);
      zero(rr[j]);
      if (r < a.rows && cols.in(j)) {
        cols.template gather<kX16>(rx[j], a.x, a, j, xr, end);
        if (a.res) cols.template fetch<kRes16>(rr[j], a.res, j, rr0 + cols.col(j), end);
      }
    }
  };
  if constexpr (kAhead) fetch(rows.row);
  int parity = 0;
  // The bound is the CTA's: its threads leave together.
  for (; rows.first < a.rows; rows.first += rows.stride, rows.row += rows.stride, parity ^= 1) {
    const unsigned row = rows.row;
    if constexpr (!kAhead) fetch(row);
    const bool live = row < a.rows;
    const long long row0 = (long long)row * a.width;
    using X = Values<VEC>;
    X s[NV];
    ops::Vec<X::kW> sums = ops::fill<X::kW>(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      cols.template trim<kX16>(rx[j], j);
      cols.template trim<kRes16>(rr[j], j);
#pragma unroll
      for (int i = 0; i < X::kN; ++i) {
        s[j].v[i] = ops::add(get(rx[j], i), get(rr[j], i));
        sums = ops::fma(s[j].v[i], s[j].v[i], sums);
      }
    }
    float sq = sums.f[0];
    if constexpr (X::kW == 2) sq += sums.f[X::kW - 1];
    if constexpr (kAhead) fetch(row + rows.stride);
    if (a.sum) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (live && cols.in(j)) cols.template put<kRes16>(a.sum, j, row0 + cols.col(j), s[j]);
    }
    sq = row_reduce<false>(sq, a.g, scratch[parity][0]);
    const float rstd = rsqrtf(fmaf(sq, a.inv_width, a.eps));
    if (a.rstd && live && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const X w = cols.weights(a, j);
#pragma unroll
      for (int i = 0; i < X::kN; ++i)
        s[j].v[i] = ops::mul(s[j].v[i], ops::mul(w.v[i], ops::fill<X::kW>(rstd)));
    }
    if constexpr (kOut != kF8) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (live && cols.in(j))
          cols.template put<kOut == kBf16>(a.y, j, row0 + cols.col(j), s[j]);
    } else {
      float top[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        top[j] = 0.f;
        if (cols.in(j))
#pragma unroll
          for (int i = 0; i < VEC; ++i) top[j] = larger(top[j], fabsf(at(s[j], i)));
      }
      if (a.group_log2 < 0) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) m = larger(m, top[j]);
        m = row_reduce<true>(m, a.g, scratch[parity][1]);
#pragma unroll
        for (int j = 0; j < NV; ++j) top[j] = m;
      } else if constexpr (VEC == 8) {
        // 4, 8 or 16 neighbouring threads share a group.
#pragma unroll
        for (int o = 1; o < 16; o <<= 1)
          if (o < (1 << a.group_log2) / 8)
#pragma unroll
            for (int j = 0; j < NV; ++j)
              top[j] = larger(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
      } else {
        // A warp has 32 columns side by side; a row has the CTA to itself.
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float m = top[j];
          for (int o = 16; o > 0; o >>= 1) m = larger(m, __shfl_xor_sync(0xffffffffu, m, o));
          if ((t & 31) == 0 && cols.in(j)) seg[parity][cols.col(j) >> 5] = m;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (cols.in(j)) {
            const int each = 1 << (a.group_log2 - 5);
            const int from = (cols.col(j) >> a.group_log2) * each;
            for (int k = 0; k < each; ++k) top[j] = larger(top[j], seg[parity][from + k]);
          }
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!(live && cols.in(j))) continue;
        const int col = cols.col(j);
        const float scale = quotient(larger(top[j], kAmaxFloor), kE4m3Max, 1.f / kE4m3Max);
        const float inv = __frcp_rn(scale);
        if (a.group_log2 < 0) {
          if (t == 0 && j == 0) a.scales[row] = scale;
        } else if ((col & ((1 << a.group_log2) - 1)) == 0) {
          a.scales[(row0 + col) >> a.group_log2] = scale;
        }
        unsigned char* p = reinterpret_cast<unsigned char*>(a.y) + row0 + col;
        if constexpr (VEC == 8) {
#pragma unroll
          for (int i = 0; i < X::kN; ++i) s[j].v[i] = quotient(s[j].v[i], scale, inv);
          const uint2 q = make_uint2(pack_e4m3(at(s[j], 0), at(s[j], 1), at(s[j], 2), at(s[j], 3)),
                                     pack_e4m3(at(s[j], 4), at(s[j], 5), at(s[j], 6), at(s[j], 7)));
          if (cols.whole(j)) {
            *reinterpret_cast<uint2*>(p) = q;
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (cols.valid(j, i)) p[i] = (unsigned char)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
          }
        } else {
          *p = (unsigned char)pack_e4m3(quotient(at(s[j], 0), scale, inv), 0.f, 0.f, 0.f);
        }
      }
    }
  }
}

using Kernel = void (*)(Args);

// How rows are cut: values one by one, vectors that rows start with, or vectors of the whole tensor.
enum Cut { kValues, kVectors, kShifted, kCuts };

template <bool X, bool R, int O, bool kShift>
Kernel forward_vectors(int nv) {
  switch (nv) {
    case 1: return norm_forward_kernel<X, R, O, 8, 1, kShift>;
    case 2: return norm_forward_kernel<X, R, O, 8, 2, kShift>;
  }
  return norm_forward_kernel<X, R, O, 8, 4, kShift>;
}
template <bool X, bool R, int O>
Kernel forward_kernel(Cut cut, int nv) {
  if (cut == kVectors) return forward_vectors<X, R, O, false>(nv);
  if (cut == kShifted) return forward_vectors<X, R, O, true>(nv);
  return nv == 4 ? norm_forward_kernel<X, R, O, 1, 4, false> : norm_forward_kernel<X, R, O, 1, 32, false>;
}

// The forward kernel for an output type: of x and residual types, of the cut and of nv vectors.
template <int O>
Kernel forward_for(bool x16, bool r16, Cut cut, int nv) {
  return x16 ? (r16 ? forward_kernel<true, true, O>(cut, nv) : forward_kernel<true, false, O>(cut, nv))
             : (r16 ? forward_kernel<false, true, O>(cut, nv) : forward_kernel<false, false, O>(cut, nv));
}
Kernel forward_f32(bool x16, bool r16, Cut cut, int nv);
Kernel forward_bf16(bool x16, bool r16, Cut cut, int nv);
Kernel forward_f8(bool x16, bool r16, Cut cut, int nv);

}  // namespace norm
}  // namespace lapl
