// norm.cu -- residual addition + root-mean-square norm: lapl_norm_* of include/lapl_ops.h.
//
// Per row (token) of W = H d values, s = x + residual:
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
// and backward, with t = dy w and n = s rstd,
//   d = rstd (t - n mean(t n)) + dsum,  dw = sum over rows dy n.
//
// Every value is read once and held in registers between the row's sum and its use.  A row
// belongs to G threads (a power of two), each with NV vectors of 8 values, vector j of thread t at
// columns (j G + t) 8: whole 16- or 32-byte pieces, neighbours side by side.  Rows of up to 32
// threads are summed by shuffles alone, longer ones through shared memory.  The CTAs are as many
// as the GPU holds and go through the rows in strides, so a thread's columns stay its own: its
// weights and its part of dweight are in registers, and the next row's values are on their way
// while this row is summed and written.
// x comes head by head ([B,H,N,d]); a vector never straddles a head (d a multiple of 8), so
// merging the heads costs only where the pieces are read from.
// Where a row's pieces cannot be vectors (d not a multiple of 8, or a pointer off 16 bytes), the
// same kernels run with vectors of one value, a row to a CTA.
#include <algorithm>
#include <new>

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
  int n, d, heads, width;
  Divisor by_n, by_d;
  int g, g_log2;        // threads of a row
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
template <bool k16, int VEC>
__device__ __forceinline__ float get(const Raw<k16, VEC>& r, int i) {
  if constexpr (!k16) return __uint_as_float(r.w[i]);
  else return (i & 1) ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
}
template <bool k16, int VEC>
__device__ __forceinline__ void store(void* base, long long e, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<char*>(base) + e * (k16 ? 2 : 4));
    if constexpr (k16) {
      *p = make_uint4(ops::pack_bf16(f[0], f[1]), ops::pack_bf16(f[2], f[3]),
                      ops::pack_bf16(f[4], f[5]), ops::pack_bf16(f[6], f[7]));
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else if constexpr (k16) {
    reinterpret_cast<uint16_t*>(base)[e] = (uint16_t)ops::pack_bf16(f[0], 0.f);
  } else {
    reinterpret_cast<float*>(base)[e] = f[0];
  }
}

// Sum or largest over the G threads of a row, the same value in each.  `scratch`: one float for
// each warp of the CTA, of this reduction alone until the next __syncthreads.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, int g, float* scratch) {
  for (int o = min(g, 32) >> 1; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, other) : v + other;
  }
  if (g > 32) {
    const int warp = threadIdx.x >> 5, per = g >> 5;
    if ((threadIdx.x & 31) == 0) scratch[warp] = v;
    __syncthreads();
    const int first = warp & ~(per - 1);
    v = scratch[first];
    for (int k = 1; k < per; ++k) v = kMax ? fmaxf(v, scratch[first + k]) : v + scratch[first + k];
  }
  return v;
}

// The e4m3 values of up to 8 floats, in bytes.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo =
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi =
      __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// A thread's columns: which are within the row, where they lie in [B,H,N,d] and their weights, in
// registers where those are few.
template <int VEC, int NV>
struct Columns {
  static constexpr bool kHeads = VEC == 8, kWeights = NV * VEC <= 16;
  bool in[NV];
  long long at[kHeads ? NV : 1];
  float w[kWeights ? NV : 1][kWeights ? VEC : 1];
  __device__ __forceinline__ void init(const Args& a, int t) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * a.g + t) * VEC;
      in[j] = col < a.width;
      if constexpr (kHeads) at[j] = in[j] ? head_col(a, col) : 0;
      if constexpr (kWeights)
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[j][i] = a.weight && in[j] ? a.weight[col + i] : 1.f;
    }
  }
  __device__ __forceinline__ long long head(const Args& a, int t, int j) const {
    if constexpr (kHeads) return at[j];
    else return head_col(a, j * a.g + t);
  }
  __device__ __forceinline__ float weight(const Args& a, int t, int j, int i) const {
    if constexpr (kWeights) return w[j][i];
    else return a.weight && in[j] ? __ldg(a.weight + (j * a.g + t) * VEC + i) : 1.f;
  }
};

enum Out { kF32, kBf16, kF8 };

template <bool kX16, bool kRes16, int kOut, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
norm_forward_kernel(const Args a) {
  __shared__ float scratch[2][2][kMaxThreads / 32];
  __shared__ float seg[VEC == 1 && kOut == kF8 ? 2 : 1][VEC == 1 && kOut == kF8 ? kMaxWidth / 32 : 1];
  // Registers for a row ahead: where a thread's part of a row is small.
  constexpr bool kAhead = NV * VEC <= 16;
  const int t = threadIdx.x & (a.g - 1);
  const unsigned per = blockDim.x >> a.g_log2, stride = gridDim.x * per;
  unsigned row = blockIdx.x * per + (threadIdx.x >> a.g_log2);
  Columns<VEC, NV> cols;
  cols.init(a, t);
  const auto& in = cols.in;
  Raw<kX16, VEC> rx[NV];
  Raw<kRes16, VEC> rr[NV];
  auto fetch = [&](unsigned r) {
    const long long xr = head_row(a, r), rr0 = (long long)r * a.width;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      zero(rx[j]);
      zero(rr[j]);
      if (r < a.rows && in[j]) {
        load(rx[j], a.x, xr + cols.head(a, t, j));
        if (a.res) load(rr[j], a.res, rr0 + (j * a.g + t) * VEC);
      }
    }
  };
  if constexpr (kAhead) fetch(row);
  int parity = 0;
  // The bound is the CTA's: its threads leave together.
  for (unsigned first = blockIdx.x * per; first < a.rows; first += stride, row += stride, parity ^= 1) {
    if constexpr (!kAhead) fetch(row);
    const bool live = row < a.rows;
    const long long at = (long long)row * a.width;
    float s[NV][VEC];
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        s[j][i] = get(rx[j], i) + get(rr[j], i);
        sq = fmaf(s[j][i], s[j][i], sq);
      }
    if constexpr (kAhead) fetch(row + stride);
    if (a.sum) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (live && in[j]) store<kRes16, VEC>(a.sum, at + (j * a.g + t) * VEC, s[j]);
    }
    sq = row_reduce<false>(sq, a.g, scratch[parity][0]);
    const float rstd = rsqrtf(fmaf(sq, a.inv_width, a.eps));
    if (a.rstd && live && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[j][i] *= rstd * cols.weight(a, t, j, i);
    if constexpr (kOut != kF8) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (live && in[j]) store<kOut == kBf16, VEC>(a.y, at + (j * a.g + t) * VEC, s[j]);
    } else {
      float top[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        top[j] = 0.f;
        if (in[j])
#pragma unroll
          for (int i = 0; i < VEC; ++i) top[j] = fmaxf(top[j], fabsf(s[j][i]));
      }
      if (a.group_log2 < 0) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) m = fmaxf(m, top[j]);
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
              top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
      } else {
        // A warp has 32 columns side by side; a row has the CTA to itself.
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float m = top[j];
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if ((t & 31) == 0 && in[j]) seg[parity][(j * a.g + t) >> 5] = m;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (in[j]) {
            const int each = 1 << (a.group_log2 - 5);
            const int from = ((j * a.g + t) >> a.group_log2) * each;
            for (int k = 0; k < each; ++k) top[j] = fmaxf(top[j], seg[parity][from + k]);
          }
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!(live && in[j])) continue;
        const int col = (j * a.g + t) * VEC;
        const float m = fmaxf(top[j], kAmaxFloor);
        const float inv = kE4m3Max / m;
        if (a.group_log2 < 0) {
          if (col == 0) a.scales[row] = m * (1.f / kE4m3Max);
        } else if ((col & ((1 << a.group_log2) - 1)) == 0) {
          a.scales[(at + col) >> a.group_log2] = m * (1.f / kE4m3Max);
        }
        unsigned char* p = reinterpret_cast<unsigned char*>(a.y) + at + col;
        if constexpr (VEC == 8) {
          *reinterpret_cast<uint2*>(p) =
              make_uint2(pack_e4m3(s[j][0] * inv, s[j][1] * inv, s[j][2] * inv, s[j][3] * inv),
                         pack_e4m3(s[j][4] * inv, s[j][5] * inv, s[j][6] * inv, s[j][7] * inv));
        } else {
          *p = (unsigned char)pack_e4m3(s[j][0] * inv, 0.f, 0.f, 0.f);
        }
      }
    }
  }
}

template <bool kRes16, bool kGrad16, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
norm_backward_kernel(const Args a) {
  __shared__ float scratch[2][kMaxThreads / 32];
  extern __shared__ float sums[];   // [rows side by side, W]
  constexpr bool kAhead = NV * VEC <= 8;
  // The kernel that sums the partials may be placed now; it waits for this grid's end.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x & (a.g - 1);
  const unsigned per = blockDim.x >> a.g_log2, mine = threadIdx.x >> a.g_log2;
  const unsigned stride = gridDim.x * per;
  unsigned row = blockIdx.x * per + mine;
  Columns<VEC, NV> cols;
  cols.init(a, t);
  const auto& in = cols.in;
  float dw[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[j][i] = 0.f;
  Raw<kRes16, VEC> rs[NV];
  Raw<kGrad16, VEC> ry[NV], rd[NV];
  float next_rstd = 0.f;
  auto fetch = [&](unsigned r) {
    const long long at = (long long)r * a.width;
    next_rstd = r < a.rows ? a.rstd[r] : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      zero(rs[j]);
      zero(ry[j]);
      zero(rd[j]);
      if (r < a.rows && in[j]) {
        load(rs[j], a.res, at + (j * a.g + t) * VEC);
        load(ry[j], a.dy, at + (j * a.g + t) * VEC);
        if (a.dsum) load(rd[j], a.dsum, at + (j * a.g + t) * VEC);
      }
    }
  };
  if constexpr (kAhead) fetch(row);
  int parity = 0;
  for (unsigned first = blockIdx.x * per; first < a.rows; first += stride, row += stride, parity ^= 1) {
    if constexpr (!kAhead) fetch(row);
    const bool live = row < a.rows;
    const long long at = (long long)row * a.width;
    const float rstd = next_rstd;
    Raw<kRes16, VEC> cs[NV];
    Raw<kGrad16, VEC> cy[NV], cd[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      cs[j] = rs[j];
      cy[j] = ry[j];
      cd[j] = rd[j];
    }
    if constexpr (kAhead) fetch(row + stride);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float dyn = get(cy[j], i) * (get(cs[j], i) * rstd);
        dw[j][i] += dyn;
        dot = fmaf(dyn, cols.weight(a, t, j, i), dot);
      }
    dot = row_reduce<false>(dot, a.g, scratch[parity]);
    const float back = -rstd * rstd * dot * a.inv_width;   // of s
    const long long hr = a.dx ? head_row(a, row) : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!(live && in[j])) continue;
      float d[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        d[i] = fmaf(rstd, get(cy[j], i) * cols.weight(a, t, j, i), fmaf(back, get(cs[j], i), get(cd[j], i)));
      if (a.dres) store<kGrad16, VEC>(a.dres, at + (j * a.g + t) * VEC, d);
      if (a.dx) store<kGrad16, VEC>(a.dx, hr + cols.head(a, t, j), d);
    }
  }
  if (!a.part) return;
  // The rows side by side in the CTA, one after the other.
  float* part = a.part + (size_t)blockIdx.x * a.width;
  if (per > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (in[j])
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          sums[(size_t)mine * a.width + (j * a.g + t) * VEC + i] = dw[j][i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
      float v = 0.f;
      for (unsigned k = 0; k < per; ++k) v += sums[(size_t)k * a.width + c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (in[j]) store<false, VEC>(part, (j * a.g + t) * VEC, dw[j]);
  }
}

// dweight[c] = sum over the CTAs' partials in a fixed order: 32 columns by 32 slices a CTA.
__global__ void __launch_bounds__(1024)
norm_dweight_kernel(const float* part, float* dweight, int ctas, int width) {
  __shared__ float sm[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are written
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int k = threadIdx.y; k < ctas; k += 32) v += part[(size_t)k * width + c];
  }
  sm[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  // Column threadIdx.y's 32 slices, one a lane.
  v = sm[threadIdx.x][threadIdx.y];
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int mine = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && mine < width) dweight[mine] = v;
}

// ---- host --------------------------------------------------------------------------------

using Kernel = void (*)(Args);

Divisor divisor(unsigned long long n) {
  Divisor d = {0, 0};
  while ((1ull << d.shift) < n) ++d.shift;
  d.mul = (unsigned)((((1ull << d.shift) - n) << 32) / n + 1);
  return d;
}

// Threads of a row and vectors of a thread.
struct Shape {
  int g, g_log2, nv, threads, per;
};
Shape shape_of(int width, int vec, bool backward) {
  const int vectors = (width + vec - 1) / vec;
  Shape s;
  if (vec == 8) {
    // One warp where up to 4 (forward) or 2 (backward) vectors a thread do: no exchange between
    // warps.  Longer rows: 2 vectors (forward) or 1 for as long as 512 threads do.
    const int most = backward ? 2 : 4;
    s.nv = 1;
    s.g = 32;
    if (vectors <= 32) {
      s.g = 1;
      while (s.g < vectors) s.g *= 2;
    } else if (vectors <= 32 * most) {
      while (32 * s.nv < vectors) s.nv *= 2;
    } else {
      s.nv = backward ? 1 : 2;
      while (s.g * s.nv < vectors && s.g < kMaxThreads) s.g *= 2;
      while (s.g * s.nv < vectors) s.nv *= 2;
    }
    s.threads = std::max(s.g, kThreads);
  } else {
    // A row has a CTA of whole warps to itself, 8 values a thread in rows up to 4096.
    s.g = 32;
    while (s.g * 8 < vectors && s.g < kMaxThreads) s.g *= 2;
    s.nv = s.g * 2 >= vectors ? 2 : s.g * 8 >= vectors ? 8 : s.g * 16 >= vectors ? 16 : 32;
    s.threads = s.g;
  }
  s.g_log2 = 0;
  while ((1 << s.g_log2) < s.g) ++s.g_log2;
  s.per = s.threads / s.g;
  return s;
}

template <bool X, bool R, int O>
Kernel forward_kernel(int vec, int nv) {
  if (vec == 8)
    return nv == 1 ? norm_forward_kernel<X, R, O, 8, 1>
                   : nv == 2 ? norm_forward_kernel<X, R, O, 8, 2> : norm_forward_kernel<X, R, O, 8, 4>;
  return nv == 2 ? norm_forward_kernel<X, R, O, 1, 2>
         : nv == 8 ? norm_forward_kernel<X, R, O, 1, 8>
         : nv == 16 ? norm_forward_kernel<X, R, O, 1, 16> : norm_forward_kernel<X, R, O, 1, 32>;
}
template <bool X, bool R>
Kernel forward_kernel(int out, int vec, int nv) {
  return out == LAPL_F32 ? forward_kernel<X, R, kF32>(vec, nv)
         : out == LAPL_BF16 ? forward_kernel<X, R, kBf16>(vec, nv) : forward_kernel<X, R, kF8>(vec, nv);
}
Kernel forward_kernel(bool x16, bool r16, int out, int vec, int nv) {
  return x16 ? (r16 ? forward_kernel<true, true>(out, vec, nv) : forward_kernel<true, false>(out, vec, nv))
             : (r16 ? forward_kernel<false, true>(out, vec, nv) : forward_kernel<false, false>(out, vec, nv));
}
template <bool R, bool G>
Kernel backward_kernel(int vec, int nv) {
  if (vec == 8)
    return nv == 1 ? norm_backward_kernel<R, G, 8, 1>
                   : nv == 2 ? norm_backward_kernel<R, G, 8, 2> : norm_backward_kernel<R, G, 8, 4>;
  return nv == 2 ? norm_backward_kernel<R, G, 1, 2>
         : nv == 8 ? norm_backward_kernel<R, G, 1, 8>
         : nv == 16 ? norm_backward_kernel<R, G, 1, 16> : norm_backward_kernel<R, G, 1, 32>;
}
Kernel backward_kernel(bool r16, bool g16, int vec, int nv) {
  return r16 ? (g16 ? backward_kernel<true, true>(vec, nv) : backward_kernel<true, false>(vec, nv))
             : (g16 ? backward_kernel<false, true>(vec, nv) : backward_kernel<false, false>(vec, nv));
}

// A kernel of a plan, with its launch shape.
struct Choice {
  Kernel kernel;
  Shape shape;
  int ctas;        // as many as the GPU holds, or as there are rows
  size_t smem;
};

lapl_status validate(const lapl_norm_config* c) {
  if (!c) return LAPL_ERR_INVALID_ARG;
  if (c->batch < 0 || c->heads < 1 || c->tokens < 1 || c->head_dim < 1) return LAPL_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || !isfinite(c->eps)) return LAPL_ERR_INVALID_ARG;
  if (!ops::is_float_dtype(c->x_dtype) || !ops::is_float_dtype(c->res_dtype) ||
      !ops::is_float_dtype(c->grad_dtype) ||
      !(ops::is_float_dtype(c->out_dtype) || c->out_dtype == LAPL_F8E4M3))
    return LAPL_ERR_INVALID_ARG;
  const int sg = c->scale_group;
  if (sg != 0 && (c->out_dtype != LAPL_F8E4M3 || (sg != 32 && sg != 64 && sg != 128)))
    return LAPL_ERR_INVALID_ARG;
  const long long width = (long long)c->heads * c->head_dim;
  if (sg != 0 && width % sg != 0) return LAPL_ERR_INVALID_ARG;
  if (width > kMaxWidth) return LAPL_ERR_UNSUPPORTED;
  // A CTA has at least one row.
  if ((long long)c->batch * c->tokens >= (1LL << 31)) return LAPL_ERR_UNSUPPORTED;
  return LAPL_OK;
}

}  // namespace norm
}  // namespace lapl

struct lapl_norm_plan {
  lapl_norm_config cfg;
  int device;
  long long rows;
  int width;
  lapl::norm::Divisor by_n, by_d;
  lapl::norm::Choice fwd[2], bwd[2];   // by single values, by vectors of 8
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

// The launch of `kernel` with shape s; smem beyond its own.
cudaError_t choose(const lapl_norm_plan& p, int sms, norm::Kernel kernel, const norm::Shape& s,
                   size_t smem, norm::Choice* out) {
  int per_sm = 0;
  const cudaError_t e =
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, s.threads, smem);
  if (e != cudaSuccess) return e;
  out->kernel = kernel;
  out->shape = s;
  out->smem = smem;
  out->ctas = (int)std::min<long long>((long long)sms * std::max(per_sm, 1),
                                       (p.rows + s.per - 1) / s.per);
  return cudaSuccess;
}

norm::Args base_args(const lapl_norm_plan& p, const norm::Shape& s) {
  norm::Args a = {};
  a.rows = (unsigned)p.rows;
  a.n = p.cfg.tokens;
  a.d = p.cfg.head_dim;
  a.heads = p.cfg.heads;
  a.width = p.width;
  a.by_n = p.by_n;
  a.by_d = p.by_d;
  a.g = s.g;
  a.g_log2 = s.g_log2;
  a.group_log2 = -1;
  for (int k = 5; k <= 7; ++k)
    if (p.cfg.scale_group == 1 << k) a.group_log2 = k;
  a.eps = p.cfg.eps;
  a.inv_width = 1.f / (float)p.width;
  return a;
}

}  // namespace

extern "C" {

lapl_status lapl_norm_create(const lapl_norm_config* cfg, lapl_norm_handle* out) {
  if (!out) return LAPL_ERR_INVALID_ARG;
  *out = nullptr;
  const lapl_status st = norm::validate(cfg);
  if (st != LAPL_OK) return st;
  lapl_norm_plan* p = new (std::nothrow) lapl_norm_plan();
  if (!p) return LAPL_ERR_INVALID_ARG;
  p->cfg = *cfg;
  p->rows = (long long)cfg->batch * cfg->tokens;
  p->width = cfg->heads * cfg->head_dim;
  p->by_n = norm::divisor((unsigned)cfg->tokens);
  p->by_d = norm::divisor((unsigned)cfg->head_dim);
  int sms = 0;
  cudaError_t e = cudaGetDevice(&p->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, p->device);
  const bool x16 = cfg->x_dtype == LAPL_BF16, r16 = cfg->res_dtype == LAPL_BF16;
  const bool g16 = cfg->grad_dtype == LAPL_BF16;
  for (int k = 0; k < 2 && e == cudaSuccess; ++k) {
    const int vec = k ? 8 : 1;
    const norm::Shape f = norm::shape_of(p->width, vec, false);
    const norm::Shape b = norm::shape_of(p->width, vec, true);
    e = choose(*p, sms, norm::forward_kernel(x16, r16, cfg->out_dtype, vec, f.nv), f, 0, &p->fwd[k]);
    if (e == cudaSuccess)
      e = choose(*p, sms, norm::backward_kernel(r16, g16, vec, b.nv), b,
                 b.per > 1 ? (size_t)b.per * p->width * sizeof(float) : 0, &p->bwd[k]);
  }
  if (e != cudaSuccess) {
    delete p;
    return LAPL_ERR_CUDA;
  }
  *out = p;
  return LAPL_OK;
}

lapl_status lapl_norm_forward(lapl_norm_handle p, const void* x, const void* residual,
                              const float* weight, void* sum, float* rstd, void* y,
                              float* scales, void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  if (p->rows == 0) return LAPL_OK;
  const lapl_norm_config& c = p->cfg;
  const bool f8 = c.out_dtype == LAPL_F8E4M3;
  if (!x || !y || f8 != (scales != nullptr)) return LAPL_ERR_INVALID_ARG;
  if (!ops::aligned(x, ops::dtype_bytes(c.x_dtype)) ||
      !ops::aligned(residual, ops::dtype_bytes(c.res_dtype)) || !ops::aligned(weight, 4) ||
      !ops::aligned(sum, ops::dtype_bytes(c.res_dtype)) || !ops::aligned(rstd, 4) ||
      !ops::aligned(y, ops::dtype_bytes(c.out_dtype)) || !ops::aligned(scales, 4))
    return LAPL_ERR_ALIGNMENT;
  const lapl_status st = ops::check_device(p->device, p->last_error, "norm_forward/device");
  if (st != LAPL_OK) return st;
  const bool wide = c.head_dim % 8 == 0 && ops::aligned(x, 16) && ops::aligned(residual, 16) &&
                    ops::aligned(sum, 16) && ops::aligned(y, 16);
  const norm::Choice& k = p->fwd[wide];
  norm::Args a = base_args(*p, k.shape);
  a.x = x;
  a.res = residual;
  a.weight = weight;
  a.sum = sum;
  a.rstd = rstd;
  a.y = y;
  a.scales = scales;
  k.kernel<<<k.ctas, k.shape.threads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "norm_forward");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

lapl_status lapl_norm_workspace_size(lapl_norm_handle p, size_t* bytes) {
  if (!p || !bytes) return LAPL_ERR_INVALID_ARG;
  *bytes = align_up((size_t)std::max(std::max(p->bwd[0].ctas, p->bwd[1].ctas), 1) * p->width *
                        sizeof(float), kAlign);
  return LAPL_OK;
}

lapl_status lapl_norm_backward(lapl_norm_handle p, const void* sum, const float* rstd,
                               const float* weight, const void* dy, const void* dsum, void* dx,
                               void* dres, float* dweight, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  const lapl_norm_config& c = p->cfg;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p->rows > 0) {
    if (!sum || !rstd || !dy || (!dx && !dres && !dweight)) return LAPL_ERR_INVALID_ARG;
    const int gb = ops::dtype_bytes(c.grad_dtype);
    if (!ops::aligned(sum, ops::dtype_bytes(c.res_dtype)) || !ops::aligned(rstd, 4) ||
        !ops::aligned(weight, 4) || !ops::aligned(dy, gb) || !ops::aligned(dsum, gb) ||
        !ops::aligned(dx, gb) || !ops::aligned(dres, gb))
      return LAPL_ERR_ALIGNMENT;
  }
  if (!ops::aligned(dweight, 4)) return LAPL_ERR_ALIGNMENT;
  if (dweight && p->rows > 0) {
    size_t need = 0;
    lapl_norm_workspace_size(p, &need);
    if (!workspace) return LAPL_ERR_INVALID_ARG;
    if (!ops::aligned(workspace, 16)) return LAPL_ERR_ALIGNMENT;
    if (workspace_bytes < need) return LAPL_ERR_WORKSPACE;
  }
  const lapl_status ok = ops::check_device(p->device, p->last_error, "norm_backward/device");
  if (ok != LAPL_OK) return ok;
  cudaError_t e = cudaSuccess;
  if (p->rows == 0) {
    if (dweight) e = cudaMemsetAsync(dweight, 0, p->width * sizeof(float), st);
  } else {
    const bool wide = c.head_dim % 8 == 0 && ops::aligned(sum, 16) && ops::aligned(dy, 16) &&
                      ops::aligned(dsum, 16) && ops::aligned(dx, 16) && ops::aligned(dres, 16);
    const norm::Choice& k = p->bwd[wide];
    norm::Args a = base_args(*p, k.shape);
    a.res = sum;
    a.rstd = const_cast<float*>(rstd);
    a.weight = weight;
    a.dy = dy;
    a.dsum = dsum;
    a.dx = dx;
    a.dres = dres;
    a.part = dweight ? static_cast<float*>(workspace) : nullptr;
    k.kernel<<<k.ctas, k.shape.threads, k.smem, st>>>(a);
    e = cudaGetLastError();
    if (e == cudaSuccess && dweight) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)((p->width + 31) / 32));
      cfg.blockDim = dim3(32, 32);
      cfg.stream = st;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, norm::norm_dweight_kernel, static_cast<const float*>(a.part),
                             dweight, k.ctas, p->width);
    }
  }
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "norm_backward");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

const char* lapl_norm_last_error(lapl_norm_handle p) { return p ? p->last_error : ""; }

lapl_status lapl_norm_destroy(lapl_norm_handle p) {
  delete p;
  return LAPL_OK;
}

}  // extern "C"
