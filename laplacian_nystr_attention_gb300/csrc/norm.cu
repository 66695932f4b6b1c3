// norm.cu -- residual addition + root-mean-square norm: lapl_norm_* of include/lapl_ops.h.
//
// Per row (token) of W = H d values, s = x + residual:
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
// and backward, with t = dy w and n = s rstd,
//   d = rstd (t - n mean(t n)) + dsum,  dw = sum over rows dy n.
//
// Every value is read once and held in registers between the row's sum and its use.  A row
// belongs to G threads (a power of two, 1 to 512), each with NV vectors of 8 values, vector j of
// thread t at columns (j G + t) 8: whole 16- or 32-byte pieces, neighbours side by side.  Rows of
// up to 32 threads are summed by shuffles alone, longer ones through shared memory.
// x comes head by head ([B,H,N,d]); a vector never straddles a head (d a multiple of 8), so
// merging the heads costs only where the pieces are read from.
// Where a row's pieces cannot be vectors (d not a multiple of 8, or a pointer off 16 bytes), the
// same kernels run with vectors of one value.
#include <algorithm>
#include <new>

#include "ops_common.cuh"

namespace lapl {
namespace norm {

constexpr int kMaxWidth = 16384;
constexpr int kThreads = 256;        // of a CTA whose rows have at most as many
constexpr int kMaxThreads = 512;
constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100
constexpr float kE4m3Max = 448.f;

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
  long long rows;
  int n, d, heads, width;
  int g, g_log2;        // threads of a row
  int group;            // values that share a scale
  float eps, inv_width;
};

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

enum Out { kF32, kBf16, kF8 };

template <bool kX16, bool kRes16, int kOut, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
norm_forward_kernel(const Args a) {
  __shared__ float scratch[2][kMaxThreads / 32];
  __shared__ float seg[VEC == 1 ? kMaxWidth / 32 : 1];   // largest |y| of each 32 columns
  const int t = threadIdx.x & (a.g - 1);
  const long long row = (long long)blockIdx.x * (blockDim.x >> a.g_log2) + (threadIdx.x >> a.g_log2);
  const bool live = row < a.rows;
  const long long b = live ? row / a.n : 0;
  const long long n = live ? row - b * a.n : 0;
  Raw<kX16, VEC> rx[NV];
  Raw<kRes16, VEC> rr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * a.g + t) * VEC;
    zero(rx[j]);
    zero(rr[j]);
    if (live && col < a.width) {
      const int h = col / a.d;
      load(rx[j], a.x, ((b * a.heads + h) * a.n + n) * a.d + (col - h * a.d));
      if (a.res) load(rr[j], a.res, row * a.width + col);
    }
  }
  float s[NV][VEC];
  float sq = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      s[j][i] = get(rx[j], i) + get(rr[j], i);
      sq = fmaf(s[j][i], s[j][i], sq);
    }
    const int col = (j * a.g + t) * VEC;
    if (a.sum && live && col < a.width) store<kRes16, VEC>(a.sum, row * a.width + col, s[j]);
  }
  sq = row_reduce<false>(sq, a.g, scratch[0]);
  const float rstd = rsqrtf(fmaf(sq, a.inv_width, a.eps));
  if (a.rstd && live && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * a.g + t) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      s[j][i] *= rstd;
      if (a.weight && col < a.width) s[j][i] *= __ldg(a.weight + col + i);
    }
  }
  if constexpr (kOut != kF8) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * a.g + t) * VEC;
      if (live && col < a.width) store<kOut == kBf16, VEC>(a.y, row * a.width + col, s[j]);
    }
  } else {
    float top[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      top[j] = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) top[j] = fmaxf(top[j], fabsf(s[j][i]));
    }
    if (a.group == a.width) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) m = fmaxf(m, top[j]);
      m = row_reduce<true>(m, a.g, scratch[1]);
#pragma unroll
      for (int j = 0; j < NV; ++j) top[j] = m;
    } else if constexpr (VEC == 8) {
      // 4, 8 or 16 neighbouring threads share a group.
#pragma unroll
      for (int j = 0; j < NV; ++j)
        for (int o = a.group >> 4; o > 0; o >>= 1)
          top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
    } else {
      // A warp has 32 columns side by side; a row has the CTA to itself.
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float m = top[j];
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int col = j * a.g + t;
        if ((t & 31) == 0 && col < a.width) seg[col >> 5] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = j * a.g + t;
        if (col < a.width) {
          const int first = col / a.group * (a.group >> 5);
          for (int k = 0; k < (a.group >> 5); ++k) top[j] = fmaxf(top[j], seg[first + k]);
        }
      }
    }
    const int groups = a.width / a.group;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * a.g + t) * VEC;
      if (!(live && col < a.width)) continue;
      const float m = fmaxf(top[j], kAmaxFloor);
      const float inv = kE4m3Max / m;
      if (col % a.group == 0) a.scales[row * groups + col / a.group] = m / kE4m3Max;
      unsigned char* p = reinterpret_cast<unsigned char*>(a.y) + row * a.width + col;
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

// Rows r, r + stride, ... of each group of G threads; a thread's columns stay its own, so it keeps
// their part of dweight in registers until the end.
template <bool kRes16, bool kGrad16, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
norm_backward_kernel(const Args a) {
  __shared__ float scratch[2][kMaxThreads / 32];
  extern __shared__ float sums[];   // [rows side by side, W]
  const int t = threadIdx.x & (a.g - 1);
  const int per = blockDim.x >> a.g_log2, mine = threadIdx.x >> a.g_log2;
  float dw[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[j][i] = 0.f;
  int parity = 0;
  for (long long first = (long long)blockIdx.x * per; first < a.rows;
       first += (long long)gridDim.x * per, parity ^= 1) {
    const long long row = first + mine;
    const bool live = row < a.rows;
    Raw<kRes16, VEC> rs[NV];
    Raw<kGrad16, VEC> ry[NV], rd[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * a.g + t) * VEC;
      zero(rs[j]);
      zero(ry[j]);
      zero(rd[j]);
      if (live && col < a.width) {
        load(rs[j], a.res, row * a.width + col);
        load(ry[j], a.dy, row * a.width + col);
        if (a.dsum) load(rd[j], a.dsum, row * a.width + col);
      }
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * a.g + t) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float w = a.weight && col < a.width ? __ldg(a.weight + col + i) : 1.f;
        const float dyn = get(ry[j], i) * (get(rs[j], i) * rstd);
        dw[j][i] += dyn;
        dot = fmaf(dyn, w, dot);
      }
    }
    dot = row_reduce<false>(dot, a.g, scratch[parity]);
    const float mean = dot * a.inv_width;
    const long long b = live ? row / a.n : 0;
    const long long n = live ? row - b * a.n : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * a.g + t) * VEC;
      if (!(live && col < a.width)) continue;
      float d[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float w = a.weight ? __ldg(a.weight + col + i) : 1.f;
        const float nrm = get(rs[j], i) * rstd;
        d[i] = fmaf(rstd, get(ry[j], i) * w - nrm * mean, get(rd[j], i));
      }
      if (a.dres) store<kGrad16, VEC>(a.dres, row * a.width + col, d);
      if (a.dx) {
        const int h = col / a.d;
        store<kGrad16, VEC>(a.dx, ((b * a.heads + h) * a.n + n) * a.d + (col - h * a.d), d);
      }
    }
  }
  if (!a.part) return;
  // The rows side by side in the CTA, one after the other.
  if (per > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * a.g + t) * VEC;
      if (col < a.width)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sums[(size_t)mine * a.width + col + i] = dw[j][i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
      float v = 0.f;
      for (int k = 0; k < per; ++k) v += sums[(size_t)k * a.width + c];
      a.part[(size_t)blockIdx.x * a.width + c] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * a.g + t) * VEC;
      if (col < a.width)
#pragma unroll
        for (int i = 0; i < VEC; ++i) a.part[(size_t)blockIdx.x * a.width + col + i] = dw[j][i];
    }
  }
}

// dweight[c] = sum over the CTAs' partials, in their order: 32 columns by 8 slices a CTA.
__global__ void __launch_bounds__(256)
norm_dweight_kernel(const float* __restrict__ part, float* __restrict__ dweight, int ctas, int width) {
  __shared__ float sm[8][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < width)
    for (int k = threadIdx.y; k < ctas; k += 8) v += part[(size_t)k * width + c];
  sm[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < width) {
    for (int k = 1; k < 8; ++k) v += sm[k][threadIdx.x];
    dweight[c] = v;
  }
}

// ---- host --------------------------------------------------------------------------------

using Kernel = void (*)(Args);

// Threads of a row and vectors of a thread.
struct Shape {
  int g, g_log2, nv, threads, per;
};
Shape shape_of(int width, int vec) {
  const int vectors = (width + vec - 1) / vec;
  Shape s;
  if (vec == 8) {
    s.g = 1;
    while (s.g < vectors && s.g < kMaxThreads) s.g *= 2;
    s.nv = 1;
    while (s.g * s.nv < vectors) s.nv *= 2;     // 1, 2 or 4
  } else {
    // A row has a CTA of whole warps to itself; 4, 16 or 32 values a thread.
    s.g = 32;
    while (s.g * 4 < vectors && s.g < kMaxThreads) s.g *= 2;
    s.nv = s.g * 4 >= vectors ? 4 : s.g * 16 >= vectors ? 16 : 32;
  }
  s.g_log2 = 0;
  while ((1 << s.g_log2) < s.g) ++s.g_log2;
  s.threads = vec == 8 ? std::max(s.g, kThreads) : s.g;
  s.per = s.threads / s.g;
  return s;
}

template <bool X, bool R, int O>
Kernel forward_kernel(int vec, int nv) {
  if (vec == 8)
    return nv == 1 ? norm_forward_kernel<X, R, O, 8, 1>
                   : nv == 2 ? norm_forward_kernel<X, R, O, 8, 2> : norm_forward_kernel<X, R, O, 8, 4>;
  return nv == 4 ? norm_forward_kernel<X, R, O, 1, 4>
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
  return nv == 4 ? norm_backward_kernel<R, G, 1, 4>
                 : nv == 16 ? norm_backward_kernel<R, G, 1, 16> : norm_backward_kernel<R, G, 1, 32>;
}
Kernel backward_kernel(bool r16, bool g16, int vec, int nv) {
  return r16 ? (g16 ? backward_kernel<true, true>(vec, nv) : backward_kernel<true, false>(vec, nv))
             : (g16 ? backward_kernel<false, true>(vec, nv) : backward_kernel<false, false>(vec, nv));
}

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
  int ctas;   // of the backward, at most: partials of dweight
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

norm::Args base_args(const lapl_norm_plan& p, const norm::Shape& s) {
  norm::Args a = {};
  a.rows = p.rows;
  a.n = p.cfg.tokens;
  a.d = p.cfg.head_dim;
  a.heads = p.cfg.heads;
  a.width = p.width;
  a.g = s.g;
  a.g_log2 = s.g_log2;
  a.group = p.cfg.scale_group ? p.cfg.scale_group : p.width;
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
  int sms = 0;
  cudaError_t e = cudaGetDevice(&p->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, p->device);
  if (e != cudaSuccess) {
    delete p;
    return LAPL_ERR_CUDA;
  }
  p->ctas = 4 * sms;
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
  const norm::Shape s = norm::shape_of(p->width, wide ? 8 : 1);
  norm::Args a = base_args(*p, s);
  a.x = x;
  a.res = residual;
  a.weight = weight;
  a.sum = sum;
  a.rstd = rstd;
  a.y = y;
  a.scales = scales;
  const norm::Kernel k = norm::forward_kernel(c.x_dtype == LAPL_BF16, c.res_dtype == LAPL_BF16,
                                              c.out_dtype, wide ? 8 : 1, s.nv);
  k<<<(unsigned)((p->rows + s.per - 1) / s.per), s.threads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "norm_forward");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

lapl_status lapl_norm_workspace_size(lapl_norm_handle p, size_t* bytes) {
  if (!p || !bytes) return LAPL_ERR_INVALID_ARG;
  *bytes = align_up((size_t)std::min<long long>(p->ctas, p->rows) * p->width * sizeof(float), kAlign);
  return LAPL_OK;
}

lapl_status lapl_norm_backward(lapl_norm_handle p, const void* sum, const float* rstd,
                               const float* weight, const void* dy, const void* dsum, void* dx,
                               void* dres, float* dweight, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  const lapl_norm_config& c = p->cfg;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  lapl_status ok;
  if (p->rows > 0) {
    if (!sum || !rstd || !dy || (!dx && !dres && !dweight)) return LAPL_ERR_INVALID_ARG;
    const int gb = ops::dtype_bytes(c.grad_dtype);
    if (!ops::aligned(sum, ops::dtype_bytes(c.res_dtype)) || !ops::aligned(rstd, 4) ||
        !ops::aligned(weight, 4) || !ops::aligned(dy, gb) || !ops::aligned(dsum, gb) ||
        !ops::aligned(dx, gb) || !ops::aligned(dres, gb))
      return LAPL_ERR_ALIGNMENT;
  }
  if (!ops::aligned(dweight, 4)) return LAPL_ERR_ALIGNMENT;
  size_t need = 0;
  lapl_norm_workspace_size(p, &need);
  if (dweight && p->rows > 0) {
    if (!workspace) return LAPL_ERR_INVALID_ARG;
    if (!ops::aligned(workspace, 16)) return LAPL_ERR_ALIGNMENT;
    if (workspace_bytes < need) return LAPL_ERR_WORKSPACE;
  }
  ok = ops::check_device(p->device, p->last_error, "norm_backward/device");
  if (ok != LAPL_OK) return ok;
  cudaError_t e = cudaSuccess;
  if (p->rows == 0) {
    if (dweight) e = cudaMemsetAsync(dweight, 0, p->width * sizeof(float), st);
  } else {
    const bool wide = c.head_dim % 8 == 0 && ops::aligned(sum, 16) && ops::aligned(dy, 16) &&
                      ops::aligned(dsum, 16) && ops::aligned(dx, 16) && ops::aligned(dres, 16);
    const norm::Shape s = norm::shape_of(p->width, wide ? 8 : 1);
    norm::Args a = base_args(*p, s);
    a.res = sum;
    a.rstd = const_cast<float*>(rstd);
    a.weight = weight;
    a.dy = dy;
    a.dsum = dsum;
    a.dx = dx;
    a.dres = dres;
    a.part = dweight ? static_cast<float*>(workspace) : nullptr;
    const norm::Kernel k = norm::backward_kernel(c.res_dtype == LAPL_BF16, c.grad_dtype == LAPL_BF16,
                                                 wide ? 8 : 1, s.nv);
    const int ctas = (int)std::min<long long>(p->ctas, (p->rows + s.per - 1) / s.per);
    const size_t smem = dweight && s.per > 1 ? (size_t)s.per * p->width * sizeof(float) : 0;
    k<<<ctas, s.threads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e == cudaSuccess && dweight) {
      norm::norm_dweight_kernel<<<(p->width + 31) / 32, dim3(32, 8), 0, st>>>(a.part, dweight, ctas,
                                                                             p->width);
      e = cudaGetLastError();
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
