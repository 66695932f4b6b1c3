// norm.cu -- residual addition + root-mean-square norm: the backward kernel, and lapl_norm_* of
// include/lapl_ops.h (norm_kernels.cuh has the formulas and the work split).
//
// HBM-bound: the backward at 32 x 784 rows of 256 fp32 values takes 20 us (the bytes: 19.0) and 23.9
// with the launch that sums dweight's partials; 8193 rows of 2049 bf16 values, whose vectors start
// anywhere, 36.3 us (68%: issue in 63% of the cycles, the rows' reductions, and 4 us for dweight).
#include <algorithm>
#include <new>

#include "norm_kernels.cuh"

namespace lapl {
namespace norm {

// Rows of bf16 that start at any value (kShifted), and the longest ones, reach a thread through shared
// memory, kStages - 1 rows ahead: 36 us instead of 40 with the next row in registers, at 8193 rows of
// 2049 values, 62 instead of 67 at 32768 of 1001; 63 instead of 81 with none ahead at 2046 of 8200.
// Shorter rows of whole vectors gain nothing by it (57 and 55 us at 32768 of 1000), and of fp32 they
// lose, a vector's two copies taking half of a sector each (28 us and 23 at 8192 of 512).
constexpr int stages_of(int nv) { return nv == 4 ? 2 : 4; }
constexpr int staged(int nv) { return nv == 4 ? 2 : 3; }   // tensors: all, or all but dsum
constexpr bool in_stages(bool res16, bool grad16, bool shift, int nv) {
  return res16 && grad16 && (shift || nv == 4);
}

// The sum over lanes `first` apart and more, in all of them.
__device__ __forceinline__ ops::Pair across(ops::Pair v, int first) {
  for (int o = first; o < 32; o *= 2) {
    const float hi = __shfl_xor_sync(0xffffffffu, v.hi, o);
    v.add(hi, __shfl_xor_sync(0xffffffffu, v.lo, o));
  }
  return v;
}

// dweight: a thread adds its rows' values in fp32, some tens of them; what follows, over its warp, its CTA
// and all CTAs, goes in pairs of floats.  Off by at most, in units of 2^-24 of the largest value: 1.1 at
// 25088 rows of 256 fp32 values, 1.4 at 8193 of 2049 bf16 ones, 3.5 at a million of 64, a hundred for
// each thread (all in fp32: 2.3, 2.1, 3.8; the terms' rounding alone: 0.6 to 1.1).
template <bool kRes16, bool kGrad16, int VEC, int NV, bool kShift>
__global__ void __launch_bounds__(kMaxThreads)
norm_backward_kernel(const Args a) {
  __shared__ float scratch[2][kMaxThreads / 32];
  extern __shared__ __align__(16) float dynamic[];
  constexpr bool kInStages = VEC == 8 && in_stages(kRes16, kGrad16, kShift, NV);
  constexpr int kStages = stages_of(NV), kStaged = staged(NV);
  constexpr bool kAhead =
      !kInStages && NV * ((kRes16 ? 4 : 8) + 2 * (kGrad16 ? 4 : 8)) * VEC / 8 <= 24;
  constexpr bool kLate = NV * VEC >= 32 && !kInStages;   // dsum is read after the row's sum: registers
  // The kernel that sums the partials may be placed now; it waits for this grid's end.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = place_in_row(a);
  const unsigned per = 1u << a.per_log2;
  Rows<kShift> rows(a);
  Columns<VEC, NV, kShift> cols;
  cols.init(a, t, rows.shift, dynamic);
  const long long end = (long long)a.rows * a.width;
  using X = Values<VEC>;
  X dw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < X::kN; ++i) dw[j].v[i] = ops::fill<X::kW>(0.f);
  Raw<kRes16, VEC> rs[NV];
  Raw<kGrad16, VEC> ry[NV], rd[NV];
  auto fetch = [&](unsigned r) {
    const long long at = (long long)r * a.width;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      zero(rs[j]);
      zero(ry[j]);
      zero(rd[j]);
      if (r < a.rows && cols.in(j)) {
        cols.template fetch<kRes16>(rs[j], a.res, j, at + cols.col(j), end);
        cols.template fetch<kGrad16>(ry[j], a.dy, j, at + cols.col(j), end);
        if (a.dsum && !kLate) cols.template fetch<kGrad16>(rd[j], a.dsum, j, at + cols.col(j), end);
      }
    }
  };
  // A stage: kStaged vectors of 16 bytes for each of a thread's, beside its neighbours'.  A thread
  // reads what it copied itself, so that nothing else waits.
  const unsigned apart = blockDim.x * 16, stage_bytes = NV * kStaged * apart;
  const unsigned stages =
      ops::smem_u32(dynamic) + threadIdx.x * 16 + blockDim.x * weight_bytes(VEC, NV);
  auto copy = [&](unsigned r, unsigned stage) {
    const long long at = (long long)r * a.width;
    unsigned to = stages + stage * stage_bytes;
#pragma unroll
    for (int j = 0; j < NV; ++j, to += kStaged * apart) {
      const bool on = r < a.rows && cols.in(j);
      cols.copy(to, a.res, on, at + cols.col(j), end);
      cols.copy(to + apart, a.dy, on, at + cols.col(j), end);
      if (kStaged == 3 && a.dsum) cols.copy(to + 2 * apart, a.dsum, on, at + cols.col(j), end);
    }
    ops::close_copies();
  };
  auto rstd_of = [&](unsigned r) { return r < a.rows ? a.rstd[r] : 0.f; };
  float next_rstd = rstd_of(rows.row);
  unsigned stage = 0;
  if constexpr (kInStages) {
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) copy(rows.row + k * rows.stride, k);
  } else if constexpr (kAhead) {
    fetch(rows.row);
  }
  int parity = 0;
  for (; rows.first < a.rows; rows.first += rows.stride, rows.row += rows.stride, parity ^= 1) {
    const unsigned row = rows.row;
    const bool live = row < a.rows;
    const long long row0 = (long long)row * a.width;
    const float rstd = next_rstd;
    next_rstd = rstd_of(row + rows.stride);
    if constexpr (kInStages) {
      copy(row + (kStages - 1) * rows.stride, (stage + kStages - 1) % kStages);
      ops::copies_left<kStages - 1>();
      unsigned from = stages + stage * stage_bytes;
      stage = (stage + 1) % kStages;
#pragma unroll
      for (int j = 0; j < NV; ++j, from += kStaged * apart) {
        read_copy(rs[j], from);
        read_copy(ry[j], from + apart);
        zero(rd[j]);
        if (!a.dsum) continue;
        if constexpr (kStaged == 3) read_copy(rd[j], from + 2 * apart);
        else if (live && cols.in(j))
          cols.template fetch<kGrad16>(rd[j], a.dsum, j, row0 + cols.col(j), end);
      }
    } else if constexpr (!kAhead) {
      fetch(row);
    }
    Raw<kRes16, VEC> cs[NV];
    Raw<kGrad16, VEC> cy[NV], cd[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      cs[j] = rs[j];
      cy[j] = ry[j];
      cd[j] = rd[j];
      cols.template trim<kRes16>(cs[j], j);
      cols.template trim<kGrad16>(cy[j], j);
    }
    if constexpr (kAhead) fetch(row + rows.stride);
    ops::Vec<X::kW> dots = ops::fill<X::kW>(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const X w = cols.weights(a, j);
#pragma unroll
      for (int i = 0; i < X::kN; ++i) {
        const auto dyn = ops::mul(get(cy[j], i), ops::mul(get(cs[j], i), ops::fill<X::kW>(rstd)));
        dw[j].v[i] = ops::add(dw[j].v[i], dyn);
        dots = ops::fma(dyn, w.v[i], dots);
      }
    }
    float dot = dots.f[0];
    if constexpr (X::kW == 2) dot += dots.f[X::kW - 1];
    dot = row_reduce<false>(dot, a.g, scratch[parity]);
    const float back = -rstd * rstd * dot * a.inv_width;   // of s
    const long long hr = a.dx ? head_row(a, row) : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!(live && cols.in(j))) continue;
      if (kLate && a.dsum) cols.template fetch<kGrad16>(cd[j], a.dsum, j, row0 + cols.col(j), end);
      const X w = cols.weights(a, j);
      X d;
#pragma unroll
      for (int i = 0; i < X::kN; ++i)
        d.v[i] = ops::fma(ops::fill<X::kW>(rstd), ops::mul(get(cy[j], i), w.v[i]),
                          ops::fma(ops::fill<X::kW>(back), get(cs[j], i), get(cd[j], i)));
      if (a.dres) cols.template put<kGrad16>(a.dres, j, row0 + cols.col(j), d);
      if (a.dx) cols.template scatter<kGrad16>(a.dx, a, j, hr, d);
    }
  }
  if constexpr (kInStages) ops::copies_left<0>();
  if (!a.part) return;
  // The CTA's part: its rows side by side, those of a warp first, then one warp after the other.
  float* part = a.part + (size_t)blockIdx.x * a.width;
  if (per > 1) {
    ops::Pair* sums = reinterpret_cast<ops::Pair*>(dynamic);   // [warps, W], where the stages were
    ops::Pair* mine = sums + (size_t)(threadIdx.x >> 5) * a.width;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const ops::Pair v = across({at(dw[j], i), 0.f}, a.g);
        if ((int)(threadIdx.x & 31) < a.g && cols.valid(j, i)) mine[cols.col(j) + i] = v;
      }
    __syncthreads();
    for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
      ops::Pair v = {};
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) {
        const ops::Pair w = sums[(size_t)k * a.width + c];
        v.add(w.hi, w.lo);
      }
      part[c] = v.value();
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (cols.valid(j, i)) part[cols.col(j) + i] = at(dw[j], i);
  }
}

// dweight[c] = sum over the CTAs' partials in a fixed order: kCols columns a CTA, kSlices threads of
// each: 8 by 128 for rows of a few thousand, 32 by 32 for longer ones, 32 by 8 for few partials.
template <int kCols, int kSlices>
__global__ void __launch_bounds__(kCols * kSlices)
norm_dweight_kernel(const float* part, float* dweight, int ctas, int width) {
  constexpr int kWarps = kCols * kSlices / 32;
  __shared__ ops::Pair sm[kWarps][kCols + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials are written
  const int c = blockIdx.x * kCols + threadIdx.x % kCols;
  ops::Pair v = {};
  if (c < width) {
#pragma unroll 4
    for (int k = threadIdx.x / kCols; k < ctas; k += kSlices) v.add(part[(size_t)k * width + c]);
  }
  v = across(v, kCols);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane < kCols) sm[warp][lane] = v;
  __syncthreads();
  if constexpr (kWarps == 32) {   // column `warp`, one of its sums a lane
    if (warp >= kCols) return;
    v = across(sm[lane][warp], 1);
    if (lane == 0 && blockIdx.x * kCols + warp < width) dweight[blockIdx.x * kCols + warp] = v.value();
  } else if (warp == 0 && c < width) {
    v = {};
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v.add(sm[k][lane].hi, sm[k][lane].lo);
    dweight[c] = v.value();
  }
}

// ---- host --------------------------------------------------------------------------------

Divisor divisor(unsigned long long n) {
  Divisor d = {0, 0};
  while ((1ull << d.shift) < n) ++d.shift;
  d.mul = (unsigned)((((1ull << d.shift) - n) << 32) / n + 1);
  return d;
}

// Threads of a row and vectors of a thread.
struct Shape {
  int g, nv, threads, per, per_log2;
};
// `two`: longer rows take two vectors a thread (the forward, and the backward where all is bf16: its
// part of dweight and of the next row fits the registers), else one, for as long as 512 threads do.
// `full`: one, too, where two leave more threads idle (768 values, 2^24 in all: bf16 backward 30.4
// against 32.6 us, fp32 and a bf16 residual forward 25.7 against 27.9; but bf16 forward at 1600 24 against
// 22, fp32 at 600 48 against 43).
Shape shape_of(int width, Cut cut, bool two, bool full) {
  Shape s;
  int vectors = width;
  s.nv = 1;
  if (cut != kValues) {
    // One warp where up to 2 vectors a thread do: no exchange between warps.
    vectors = (width + (cut == kShifted ? 14 : 7)) / 8;
    if (vectors <= 64) {
      while (32 * s.nv < vectors) s.nv *= 2;
    } else {
      auto idle = [&](int nv) { return ((vectors + nv - 1) / nv + 31) / 32 * 32 * nv - vectors; };
      s.nv = two && !(full && idle(2) > idle(1)) ? 2 : 1;
      while (kMaxThreads * s.nv < vectors && s.nv < 4) s.nv *= 2;
    }
  } else {
    // A row has a CTA to itself, 4 values a thread in rows up to 2048.
    s.nv = kMaxThreads * 4 >= width ? 4 : 32;
  }
  const int need = (vectors + s.nv - 1) / s.nv;
  s.g = 1;
  if (need > 32 || cut == kValues) {
    s.g = std::min((need + 31) / 32 * 32, kMaxThreads);
  } else {
    while (s.g < need) s.g *= 2;
  }
  s.per = cut != kValues && s.g <= 32 ? kThreads / s.g : 1;
  s.threads = s.g * s.per;
  s.per_log2 = 0;
  while ((1 << s.per_log2) < s.per) ++s.per_log2;
  return s;
}

template <bool R, bool G, bool kShift>
Kernel backward_vectors(int nv) {
  switch (nv) {
    case 1: return norm_backward_kernel<R, G, 8, 1, kShift>;
    case 2: return norm_backward_kernel<R, G, 8, 2, kShift>;
  }
  return norm_backward_kernel<R, G, 8, 4, kShift>;
}
template <bool R, bool G>
Kernel backward_kernel(Cut cut, int nv) {
  if (cut == kVectors) return backward_vectors<R, G, false>(nv);
  if (cut == kShifted) return backward_vectors<R, G, true>(nv);
  return nv == 4 ? norm_backward_kernel<R, G, 1, 4, false> : norm_backward_kernel<R, G, 1, 32, false>;
}
Kernel forward_kernel(int out, bool x16, bool r16, Cut cut, int nv) {
  return out == LAPL_F32 ? forward_f32(x16, r16, cut, nv)
         : out == LAPL_BF16 ? forward_bf16(x16, r16, cut, nv) : forward_f8(x16, r16, cut, nv);
}
Kernel backward_kernel(bool r16, bool g16, Cut cut, int nv) {
  return r16 ? (g16 ? backward_kernel<true, true>(cut, nv) : backward_kernel<true, false>(cut, nv))
             : (g16 ? backward_kernel<false, true>(cut, nv) : backward_kernel<false, false>(cut, nv));
}

// Dynamic shared memory of the backward: the stages of rows to come, then the side-by-side sums.
size_t backward_smem(const lapl_norm_config& c, const Shape& s, Cut cut) {
  const bool stages = in_stages(c.res_dtype == LAPL_BF16, c.grad_dtype == LAPL_BF16,
                                cut == kShifted, s.nv);
  const size_t sums = s.per > 1 ? (size_t)(kThreads / 32) * c.heads * c.head_dim * sizeof(ops::Pair) : 0;
  const size_t a_thread = (cut == kValues ? 0 : weight_bytes(8, s.nv)) +
                          (stages ? stages_of(s.nv) * s.nv * staged(s.nv) * 16 : 0);
  return std::max(a_thread * s.threads, sums);
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
  int period;   // of the rows' starts among vectors of 8
  int sms;
  lapl::norm::Choice fwd[lapl::norm::kCuts], bwd[lapl::norm::kCuts];
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

// The launch of `kernel` with shape s; smem beyond its own.
cudaError_t choose(const lapl_norm_plan& p, int sms, norm::Kernel kernel, const norm::Shape& s,
                   norm::Cut cut, size_t smem, norm::Choice* out) {
  int per_sm = 0;
  cudaError_t e = cudaSuccess;
  // The same for every plan: it is the kernel's, not the launch's.
  constexpr size_t kMost = 24 * 16 * norm::kMaxThreads;   // pieces of a thread
  if (smem > kMost) return cudaErrorInvalidValue;
  if (smem > 0)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
  if (e != cudaSuccess) return e;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, s.threads, smem);
  if (e != cudaSuccess) return e;
  out->kernel = kernel;
  out->shape = s;
  out->smem = smem;
  // kShifted: a multiple of the period, each of whose places has rows / period rows, rounded up.
  const long long parts = cut == norm::kShifted ? p.period : 1;
  const long long rows = (p.rows + parts - 1) / parts;
  out->ctas = (int)(parts * std::max<long long>(1, std::min<long long>(
                                (long long)sms * std::max(per_sm, 1) / parts,
                                (rows + s.per - 1) / s.per)));
  return cudaSuccess;
}

// aligned: every tensor starts at a multiple of 16 bytes; by_head: written head by head, too.
norm::Cut cut_of(const lapl_norm_plan& p, bool aligned, bool by_head) {
  if (!aligned) return norm::kValues;
  if (p.cfg.head_dim % 8 == 0) return norm::kVectors;
  // Values written one by one of a thread's 8 in a row cost more than the vectors read give, where a
  // value a thread keeps a CTA's threads busy and 4 do for a row (backward, 8000 x 8 x 150 fp32: 39
  // against 61 us; 60000 x 4 x 3: 21 against 9; 186 x 2 x 1718: 40 against 12).
  if (by_head && p.cfg.heads > 1 && p.width >= 64 && p.width <= 4 * norm::kMaxThreads)
    return norm::kValues;
  // A row of W values touches up to (W + 14) / 8 vectors; 512 threads have 4 each.
  return p.width + 14 < 8 * (4 * norm::kMaxThreads + 1) ? norm::kShifted : norm::kValues;
}

norm::Args base_args(const lapl_norm_plan& p, const norm::Shape& s) {
  norm::Args a = {};
  a.rows = (unsigned)p.rows;
  a.n = p.cfg.tokens;
  a.d = p.cfg.head_dim;
  a.heads = p.cfg.heads;
  a.width = p.width;
  a.period = p.period;
  a.by_n = p.by_n;
  a.by_d = p.by_d;
  a.g = s.g;
  a.per_log2 = s.per_log2;
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
  p->sms = sms;
  const bool x16 = cfg->x_dtype == LAPL_BF16, r16 = cfg->res_dtype == LAPL_BF16;
  const bool g16 = cfg->grad_dtype == LAPL_BF16;
  p->period = 8;
  while (p->period > 1 && (long long)p->period / 2 * p->width % 8 == 0) p->period /= 2;
  for (int k = 0; k < norm::kCuts && e == cudaSuccess; ++k) {
    const norm::Cut cut = (norm::Cut)k;
    const norm::Shape f = norm::shape_of(p->width, cut, true, !x16 && r16);
    const norm::Shape b = norm::shape_of(p->width, cut, r16 && g16, true);
    e = choose(*p, sms, norm::forward_kernel(cfg->out_dtype, x16, r16, cut, f.nv), f, cut,
               cut == norm::kValues ? 0 : (size_t)norm::weight_bytes(8, f.nv) * f.threads, &p->fwd[k]);
    if (e == cudaSuccess)
      e = choose(*p, sms, norm::backward_kernel(r16, g16, cut, b.nv), b, cut,
                 norm::backward_smem(*cfg, b, cut), &p->bwd[k]);
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
  const norm::Choice& k = p->fwd[cut_of(
      *p, ops::aligned(x, 16) && ops::aligned(residual, 16) && ops::aligned(sum, 16) &&
              ops::aligned(y, 16), false)];
  norm::Args a = base_args(*p, k.shape);
  a.x = x;
  a.res = residual;
  a.weight = weight;
  a.sum = sum;
  a.rstd = rstd;
  a.y = y;
  a.scales = scales;
  k.kernel<<<k.ctas, k.shape.threads, k.smem, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "norm_forward");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

lapl_status lapl_norm_workspace_size(lapl_norm_handle p, size_t* bytes) {
  if (!p || !bytes) return LAPL_ERR_INVALID_ARG;
  *bytes = align_up((size_t)std::max({p->bwd[0].ctas, p->bwd[1].ctas, p->bwd[2].ctas}) *
                        p->width * sizeof(float), kAlign);
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
    const norm::Choice& k = p->bwd[cut_of(
        *p, ops::aligned(sum, 16) && ops::aligned(dy, 16) && ops::aligned(dsum, 16) &&
                ops::aligned(dx, 16) && ops::aligned(dres, 16), dx != nullptr)];
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
      // One wave, of 1024 threads two CTAs an SM (6000 columns of 152 partials: 2 us less than by 8).
      const int wave = 2 * p->sms;
      const bool few = k.ctas <= 64 || p->width > 32 * wave, wide = p->width > 8 * wave;
      const int cols = few || wide ? 32 : 8;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)((p->width + cols - 1) / cols));
      cfg.blockDim = dim3(few ? 256 : 1024);
      cfg.stream = st;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, few ? norm::norm_dweight_kernel<32, 8>
                                 : wide ? norm::norm_dweight_kernel<32, 32>
                                        : norm::norm_dweight_kernel<8, 128>,
                             static_cast<const float*>(a.part), dweight, k.ctas, p->width);
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
