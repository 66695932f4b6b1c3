// decay_rows.cu -- a pass of the linear attention with decays token by token (decay.cuh has the
// formulas): any sizes, types and alignment, and single tokens.
//
// A warp holds kCols columns of a sequence's state for each lane, all rows of them, in registers; a
// token costs it a fused multiply-add for y_i z_j and one for x_i S_ij for each value, two rows at a
// time in packed fp32 instructions.  The decay costs nothing: within a stage of kTok tokens the state
// is held times g^-i (z times that instead, and outputs times g^i), and put right at the stage's end.
// Where g^-kTok is large (over 2^4; a larger one could overflow what the sums do not) the state is
// multiplied at every token.  The warps of a CTA take the same sequence's next columns, so that x and
// y are read and widened to fp32 once; tokens are copied a stage ahead.
//
// Bound by fp32 arithmetic for long sequences (2 a b multiply-adds a token, 3 with segments), by the
// bytes of the states for single tokens.
#include <algorithm>

#include "decay.cuh"

namespace lapl {
namespace decay {
namespace {

using ops::Vec;

constexpr int kTok = 16;          // tokens of a stage
constexpr float kMostUp = 4.f;    // log2 of the largest g^-kTok that the state is held times

// Copies `bytes` (a run of whole elements) to shared memory, in the widest pieces that both sides
// start on; `there`: dst is as far into 16 bytes as src.
__device__ __forceinline__ void copy_run(unsigned char* dst, const unsigned char* src, int bytes,
                                         int thread, int threads) {
  const unsigned to = ops::smem_u32(dst);
  if (((uintptr_t)src & 15) == 0) {
    for (int i = thread * 16; i < bytes; i += threads * 16) {
      // The last piece may be short: none are read past the run, zeros are written.
      const int n = min(16, bytes - i);
      if ((n & 3) == 0) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to + i), "l"(src + i),
                     "r"(n)
                     : "memory");
      } else {
        for (int e = 0; e < n; e += 2)
          *reinterpret_cast<uint16_t*>(dst + i + e) = *reinterpret_cast<const uint16_t*>(src + i + e);
      }
    }
  } else if (((uintptr_t)src & 3) == 0) {
    for (int i = thread * 4; i < bytes; i += threads * 4) {
      if (bytes - i >= 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + i), "l"(src + i) : "memory");
      } else {
        *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
      }
    }
  } else {
    for (int i = thread * 2; i < bytes; i += threads * 2)
      *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
  }
}

// Where the tokens [i0, i0 + n) of the processing order start in memory.
__device__ __forceinline__ long long first_token(const Pass& p, int len, int i0, int n) {
  return p.reverse ? len - i0 - n : i0;
}

template <int KD, int kCols, bool kOut>
__global__ void __launch_bounds__(128, 2)
decay_rows_kernel(const __grid_constant__ Args a, int pass0) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Pass& p = a.pass[pass0 + blockIdx.z];
  const int bh = blockIdx.x / a.segments, segment = blockIdx.x % a.segments;
  const Range range(a, bh, segment);
  const int live = range.live(a, p);
  if (!kOut && segment == a.segments - 1) return;   // no segment comes after it
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
  const int rows = p.a, cols = p.b;
  int col[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) col[c] = (warp * 32 + lane) * kCols + c;
  // Shared memory: two raw stages (x, y, z as they are), then one stage in fp32.
  const int xb = p.x_half ? 2 : 4, yb = p.y_half ? 2 : 4, zb = p.z_half ? 2 : 4;
  const unsigned raw_x = kOut ? (unsigned)((kTok * rows * xb + 15) & ~15) : 0u;
  const unsigned raw_y = (unsigned)((kTok * rows * yb + 15) & ~15);
  const unsigned raw_z = (unsigned)((kTok * cols * zb + 15) & ~15);
  const unsigned raw = raw_x + raw_y + raw_z;
  float* fx = reinterpret_cast<float*>(smem + 2 * raw);       // [kTok][KD]
  float* fy = fx + (kOut ? kTok * KD : 0);                    // [kTok][KD]
  float* fz = fy + kTok * KD;                                 // [kTok][cols]

  const float l = log_decay(a, bh), l2 = l * kLog2e;
  const bool held = -l2 * kTok <= kMostUp;

  Vec<2> S[kCols][KD / 2];
#pragma unroll
  for (int c = 0; c < kCols; ++c)
#pragma unroll
    for (int i = 0; i < KD / 2; ++i) S[c][i] = ops::fill<2>(0.f);
  if (kOut) {
    const float* from = nullptr;
    long long row_step = cols, col_step = 1;
    if (p.states) {
      from = p.states + ((long long)bh * a.segments + segment) * rows * cols;
    } else if (p.first) {
      from = p.first + (long long)bh * rows * cols;
      if (p.first_across) row_step = 1, col_step = rows;
    }
    if (from) {
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < KD; ++i)
          if (i < rows && col[c] < cols) S[c][i / 2].f[i & 1] = from[i * row_step + col[c] * col_step];
    }
  }

  auto copy = [&](int i0, int stage) {
    const int n = min(kTok, range.begin + live - i0);
    if (n > 0) {
      const long long token = (long long)bh * a.tokens + first_token(p, range.len, i0, n);
      unsigned char* to = smem + stage * raw;
      if (kOut)
        copy_run(to, static_cast<const unsigned char*>(p.x) + token * rows * xb, n * rows * xb,
                 threadIdx.x, threads);
      copy_run(to + raw_x, static_cast<const unsigned char*>(p.y) + token * rows * yb, n * rows * yb,
               threadIdx.x, threads);
      copy_run(to + raw_x + raw_y, static_cast<const unsigned char*>(p.z) + token * cols * zb,
               n * cols * zb, threadIdx.x, threads);
    }
    ops::close_copies();
  };
  // One stage's rows in fp32, in processing order; `pad`: to KD with zeros.
  auto widen = [&](float* to, const unsigned char* from, int half, int n, int width, int pad) {
    for (int i = threadIdx.x; i < n * pad; i += threads) {
      const int t = i / pad, e = i - t * pad;
      const int src = (p.reverse ? n - 1 - t : t) * width + e;
      float v = 0.f;
      if (e < width)
        v = half ? ops::bf16_bits(reinterpret_cast<const uint16_t*>(from)[src])
                 : reinterpret_cast<const float*>(from)[src];
      to[i] = v;
    }
  };

  copy(range.begin, 0);
  int stage = 0;
  bool first = kOut && p.undecayed && segment == 0;
  for (int i0 = range.begin; i0 < range.begin + live; i0 += kTok, stage ^= 1) {
    const int n = min(kTok, range.begin + live - i0);
    copy(i0 + kTok, stage ^ 1);
    ops::copies_left<1>();
    __syncthreads();   // this stage's copies are there; the last one's fp32 values are used up
    const unsigned char* from = smem + stage * raw;
    if (kOut) widen(fx, from, p.x_half, n, rows, KD);
    widen(fy, from + raw_x, p.y_half, n, rows, KD);
    widen(fz, from + raw_x + raw_y, p.z_half, n, cols, cols);
    __syncthreads();
    // The state's factor: it is S times `up` (held), which a token multiplies by 1 / g.
    if (held && first) {
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < KD / 2; ++i) S[c][i] = ops::mul(S[c][i], ops::fill<2>(exp2f(-l2)));
      first = false;
    }
    const float g = exp2f(l2);
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      const float up = held ? exp2f(-l2 * (float)(t + 1)) : 1.f;
      const float down = held ? exp2f(l2 * (float)(t + 1)) : 1.f;
      if (!held && !first) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
          for (int i = 0; i < KD / 2; ++i) S[c][i] = ops::mul(S[c][i], ops::fill<2>(g));
      }
      first = false;
      Vec<2> z[kCols], o[kCols][2];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        z[c] = ops::fill<2>(col[c] < cols ? fz[t * cols + col[c]] * p.zs * up : 0.f);
        o[c][0] = o[c][1] = ops::fill<2>(0.f);
      }
      const float4* y4 = reinterpret_cast<const float4*>(fy + t * KD);
      const float4* x4 = reinterpret_cast<const float4*>(fx + t * KD);
#pragma unroll
      for (int i = 0; i < KD / 4; ++i) {
        const float4 y = y4[i];
        const Vec<2> y0 = {{y.x, y.y}}, y1 = {{y.z, y.w}};
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          S[c][2 * i] = ops::fma(y0, z[c], S[c][2 * i]);
          S[c][2 * i + 1] = ops::fma(y1, z[c], S[c][2 * i + 1]);
        }
        if (kOut) {
          const float4 x = x4[i];
          const Vec<2> x0 = {{x.x, x.y}}, x1 = {{x.z, x.w}};
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            o[c][0] = ops::fma(x0, S[c][2 * i], o[c][0]);
            o[c][1] = ops::fma(x1, S[c][2 * i + 1], o[c][1]);
          }
        }
      }
      if (kOut) {
        const int i = i0 + t;
        const long long row =
            ((long long)bh * a.tokens + (p.reverse ? range.len - 1 - i : i)) * cols;
        const float f = p.os * down;
        float v[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          v[c] = f * ((o[c][0].f[0] + o[c][0].f[1]) + (o[c][1].f[0] + o[c][1].f[1]));
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (col[c] < cols) {
            if (p.out_half) static_cast<__nv_bfloat16*>(p.out)[row + col[c]] = __float2bfloat16_rn(v[c]);
            else static_cast<float*>(p.out)[row + col[c]] = v[c];
          }
      }
    }
    if (held) {
      const Fade fade(l, n);
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < KD / 2; ++i) S[c][i] = fade(S[c][i]);
    }
  }
  // Where the state goes: this segment's own, or after the last segment the sequence's.
  float* to = nullptr;
  float f = 1.f;
  if (!kOut) {
    to = p.states + ((long long)bh * a.segments + segment) * rows * cols;
  } else if (p.last && segment == a.segments - 1) {
    to = p.last + (long long)bh * rows * cols;
    if (p.undecayed && range.len > 0) f = exp2f(l2);
  }
  if (to) {
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int i = 0; i < KD; ++i)
        if (i < rows && col[c] < cols) to[(long long)i * cols + col[c]] = S[c][i / 2].f[i & 1] * f;
  }
  // Zeros for the segment's padding.
  if (kOut) {
    const long long row0 = (long long)bh * a.tokens;
    const long long from = (row0 + max(range.begin, range.len)) * cols;
    const long long to_end = (row0 + range.end) * cols;
    for (long long i = from + threadIdx.x; i < to_end; i += threads) {
      if (p.out_half) static_cast<uint16_t*>(p.out)[i] = 0;
      else static_cast<float*>(p.out)[i] = 0.f;
    }
  }
}

// The state before each segment, from every segment's own (in place): a thread for each value.
__global__ void __launch_bounds__(256)
decay_carry_kernel(const __grid_constant__ Args a, int tiles) {
  const Pass& p = a.pass[blockIdx.z];
  const int size = p.a * p.b, bh = blockIdx.x / tiles;
  const int i = (blockIdx.x - bh * tiles) * 256 + threadIdx.x;
  if (i >= size) return;
  const float l = log_decay(a, bh);
  float s = 0.f;
  if (p.first) {
    const int row = i / p.b, col = i - row * p.b;
    s = p.first[(long long)bh * size + (p.first_across ? col * p.a + row : i)];
  }
  float* at = p.states + (long long)bh * a.segments * size + i;
  bool undecayed = p.undecayed;
  constexpr int kAhead = 8;   // loads in flight
  for (int g0 = 0; g0 < a.segments; g0 += kAhead) {
    float own[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      own[u] = g0 + u < a.segments - 1 ? at[(long long)(g0 + u) * size] : 0.f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (g0 + u >= a.segments) break;
      const int live = Range(a, bh, g0 + u).live(a, p);
      at[(long long)(g0 + u) * size] = s;
      if (live > 0) s = Fade(l, live - undecayed)(s) + own[u];
      if (live > 0) undecayed = false;
    }
  }
}

template <int KD, int kCols>
cudaError_t launch_pass(const Args& a, int pass0, int passes, int bh, bool out, int warps, size_t smem,
                        cudaStream_t st) {
  auto kernel = out ? decay_rows_kernel<KD, kCols, true> : decay_rows_kernel<KD, kCols, false>;
  if (smem > 48 * 1024) {
    // As large as any call needs: calls at once do not set it lower for each other.
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kTok * (KD + KD + 128) * 4 * 3);
    if (e != cudaSuccess) return e;
  }
  kernel<<<dim3((unsigned)(bh * a.segments), 1, (unsigned)passes), 32 * warps, smem, st>>>(a, pass0);
  return cudaGetLastError();
}

// Rows of a pass as the kernels pad them.
int padded(int rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

}  // namespace

cudaError_t launch_carry(const Args& a, int passes, int bh, cudaStream_t st) {
  int most = 0;
  for (int i = 0; i < passes; ++i) most = std::max(most, a.pass[i].a * a.pass[i].b);
  const int tiles = (most + 255) / 256;
  decay_carry_kernel<<<dim3((unsigned)(bh * tiles), 1, (unsigned)passes), 256, 0, st>>>(a, tiles);
  return cudaGetLastError();
}

cudaError_t launch_rows(const Args& a, int passes, int bh, cudaStream_t st) {
  for (int stage = a.segments > 1 ? 0 : a.pass[0].states ? 1 : 2; stage < 3; ++stage) {
    if (stage == 1) {
      const cudaError_t e = launch_carry(a, passes, bh, st);
      if (e != cudaSuccess) return e;
      continue;
    }
    // Passes of the same padded rows in one launch.
    for (int i = 0; i < passes;) {
      const int kd = padded(a.pass[i].a);
      int n = 1;
      while (i + n < passes && padded(a.pass[i + n].a) == kd) ++n;
      int cols = 0;
      size_t smem = 0;
      for (int j = i; j < i + n; ++j) {
        const Pass& p = a.pass[j];
        cols = std::max(cols, p.b);
        const size_t x = stage == 2 ? align_up((size_t)kTok * p.a * (p.x_half ? 2 : 4), 16) : 0;
        const size_t y = align_up((size_t)kTok * p.a * (p.y_half ? 2 : 4), 16);
        const size_t z = align_up((size_t)kTok * p.b * (p.z_half ? 2 : 4), 16);
        smem = std::max(smem, 2 * (x + y + z) +
                                  sizeof(float) * kTok * ((stage == 2 ? 2 : 1) * kd + p.b));
      }
      cudaError_t e;
      const bool out = stage == 2;
      if (kd == 128) {
        e = launch_pass<128, 1>(a, i, n, bh, out, (cols + 31) / 32, smem, st);
      } else if (kd == 64) {
        e = cols > 32 ? launch_pass<64, 2>(a, i, n, bh, out, (cols + 63) / 64, smem, st)
                      : launch_pass<64, 1>(a, i, n, bh, out, 1, smem, st);
      } else {
        e = cols > 32 ? launch_pass<32, 2>(a, i, n, bh, out, (cols + 63) / 64, smem, st)
                      : launch_pass<32, 1>(a, i, n, bh, out, 1, smem, st);
      }
      if (e != cudaSuccess) return e;
      i += n;
    }
  }
  return cudaSuccess;
}

}  // namespace decay
}  // namespace lapl
