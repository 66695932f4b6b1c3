// decay_rows.cu -- a pass of the linear attention with decays token by token (decay.cuh has the
// formulas): any sizes, types and alignment, and single tokens.
//
// A warp holds 8 kCols columns of a sequence's state, all rows of them, in registers: a lane kCols columns of
// a quarter of the rows.  A token costs it a fused multiply-add for y_i z_j and one for x_i S_ij for each value,
// two rows at a time in packed fp32 instructions; the quarters' outputs meet in six shuffles.  (With whole
// columns in a lane every lane read all of x and y: 32 reads of 16 bytes a token at 64 x 64 instead of 10, and
// shared memory, 4 clocks for each, took three times as long as the arithmetic.)  The decay costs
// nothing: within a stage of kTok tokens the state is held times g^-i (z times that instead, and outputs
// times g^i), and put right at the stage's end.  Where g^-16 is large (over 2^4; a larger one could
// overflow what the sums do not) the state is multiplied at every token.  The warps of a CTA take the
// same sequence's next columns, so that x and y are read and widened to fp32 once (rows in fp32 that need no
// padding stay as they are: 416 us instead of 490); tokens are copied a stage ahead.
//
// Bound by fp32 instructions for long sequences (2 a b multiply-adds a token, 3 with segments), by the
// bytes of the states for single tokens.  4 x 8 sequences of 16384 tokens of 64 x 64 in fp32: 425 us, 30
// tera-operations a second (of 537 MB, 1.3 TB/s); 8 x 2 of 3136 tokens of 32 x 32: 32 us; one token of 512
// sequences of 64 x 64 in bf16: 6.4 us (2.7 TB/s of 17 MB).
#include <algorithm>

#include "decay.cuh"

namespace lapl {
namespace decay {
namespace {

using ops::Vec;

// Tokens of a stage: as many as leave room in shared memory for the warps that registers do (64 x 64 in fp32
// with 16: 472 us for what took 416).
constexpr int kMostTok = 16;
constexpr int tokens_of(int kd) { return kd <= 48 ? 16 : 12; }
constexpr float kMostUp = 4.f;    // log2 of the largest g^-kMostTok that the state is held times

// Two floats in a register pair as the packed instructions take them.  (As two floats that happen to be
// neighbours, half of a token's instructions were moves.)
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Vec<2> apart(Two v) {
  Vec<2> r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.f[0]), "=f"(r.f[1]) : "l"(v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

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

// Sums over the four quarters of the warp, kCols / 4 of each lane's kCols: those from column
// (lane / 16) kCols / 2 + (lane / 8 % 2) kCols / 4 on.
template <int kCols>
__device__ __forceinline__ void across_quarters(float (&v)[kCols], int lane) {
  const bool upper = lane & 16, odd = lane & 8;
#pragma unroll
  for (int c = 0; c < kCols / 2; ++c) {
    const float other = __shfl_xor_sync(0xffffffffu, upper ? v[c] : v[c + kCols / 2], 16);
    v[c] = (upper ? v[c + kCols / 2] : v[c]) + other;
  }
#pragma unroll
  for (int c = 0; c < kCols / 4; ++c) {
    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + kCols / 4], 8);
    v[c] = (odd ? v[c + kCols / 4] : v[c]) + other;
  }
}

// Registers for as many warps as a lane's part of the state allows: a warp issues every 4 to 5 clocks.
template <int KD, int kCols, bool kOut>
__global__ void __launch_bounds__(128, rows_ctas(KD, kCols))
decay_rows_kernel(const __grid_constant__ Args a, int pass0) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kTok = tokens_of(KD);
  constexpr int kRows = KD / 4, kPairs = kRows / 2;   // of a lane
  constexpr int kWide = 8 * kCols;                    // columns of a warp
  const Pass& p = a.pass[pass0 + blockIdx.z];
  const int bh = blockIdx.x / a.segments, segment = blockIdx.x % a.segments;
  const Range range(a, bh, segment);
  const int live = range.live(a, p);
  if (!kOut) release_next();
  if (!kOut && segment == a.segments - 1) return;   // no segment comes after it
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x, warps = threads / 32;
  const int rows = p.a, cols = p.b;
  const int row0 = (lane >> 3) * kRows, col0 = warp * kWide + (lane & 7) * kCols;
  // First of the columns whose outputs are left to the lane.
  const int out_col = col0 + ((lane >> 4) & 1) * (kCols / 2) + ((lane >> 3) & 1) * (kCols / 4);
  // Shared memory: two raw stages (x, y, z as they are), then one stage in fp32, padded.
  const int xb = p.x_half ? 2 : 4, yb = p.y_half ? 2 : 4, zb = p.z_half ? 2 : 4;
  const unsigned raw_x = kOut ? (unsigned)((kTok * rows * xb + 15) & ~15) : 0u;
  const unsigned raw_y = (unsigned)((kTok * rows * yb + 15) & ~15);
  const unsigned raw_z = (unsigned)((kTok * cols * zb + 15) & ~15);
  const unsigned raw = raw_x + raw_y + raw_z;
  // Rows of fp32 that need no padding are read as they were copied.
  const int wide = warps * kWide;
  const bool x_as_is = !p.x_half && rows == KD, y_as_is = !p.y_half && rows == KD;
  const bool z_as_is = !p.z_half && cols == wide;
  float* fx = reinterpret_cast<float*>(smem + 2 * raw);       // [kTok][KD]
  float* fy = fx + (kOut && !x_as_is ? kTok * KD : 0);        // [kTok][KD]
  float* fz = fy + (y_as_is ? 0 : kTok * KD);                 // [kTok][wide]
  float* up = fz + (z_as_is ? 0 : kTok * wide);               // [kTok] what z is multiplied by,
  float* down = up + kTok;                                    // [kTok] and what outputs are

  const float l = log_decay(a, bh), l2 = l * kLog2e;
  const bool held = -l2 * kMostTok <= kMostUp;
  if (threadIdx.x < kTok) {
    const float n = (float)(threadIdx.x + 1);
    up[threadIdx.x] = held ? p.zs * exp2f(-l2 * n) : p.zs;
    down[threadIdx.x] = held ? p.os * exp2f(l2 * n) : p.os;
  }
  const Fade whole(l, kTok);

  Two S[kPairs][kCols];
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
#pragma unroll
    for (int c = 0; c < kCols; ++c) S[i][c] = 0;
  // Calls use(value, row, column) for every value of the lane's that is there.
  auto each_value = [&](auto use) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        Vec<2> v = apart(S[i][c]);
        if (col0 + c < cols) {
          if (row0 + 2 * i < rows) use(v.f[0], row0 + 2 * i, col0 + c);
          if (row0 + 2 * i + 1 < rows) use(v.f[1], row0 + 2 * i + 1, col0 + c);
        }
        S[i][c] = two(v.f[0], v.f[1]);
      }
  };
  // The same for four columns, where rows are whole vectors.
  auto each_four = [&](auto use) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        Vec<2> v[4] = {apart(S[i][c]), apart(S[i][c + 1]), apart(S[i][c + 2]), apart(S[i][c + 3])};
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (row0 + 2 * i + e < rows && col0 + c < cols)
            use(v[0].f[e], v[1].f[e], v[2].f[e], v[3].f[e], (row0 + 2 * i + e) * cols + col0 + c);
#pragma unroll
        for (int k = 0; k < 4; ++k) S[i][c + k] = two(v[k].f[0], v[k].f[1]);
      }
  };
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
  // Value e of row t of a raw stage.
  auto value = [&](const unsigned char* from, int half, int width, int t, int e) {
    return half ? ops::bf16_bits(reinterpret_cast<const uint16_t*>(from)[t * width + e])
                : reinterpret_cast<const float*>(from)[t * width + e];
  };
  // One stage's rows in fp32, padded to KD with zeros; a warp takes a row.
  auto widen = [&](float* to, const unsigned char* from, int half, int n) {
#pragma unroll 4
    for (int t = warp; t < n; t += warps) {
#pragma unroll
      for (int j = 0; j < (KD + 31) / 32; ++j) {
        const int e = lane + 32 * j;
        if (KD % 32 && e >= KD) break;
        to[t * KD + e] = e < rows ? value(from, half, rows, t, e) : 0.f;
      }
    }
  };

  copy(range.begin, 0);
  if (kOut) {
    if (p.states) await_last();   // the states before each segment are there
    const long long at = (long long)bh * rows * cols;
    const float* from = p.states ? p.states + ((long long)bh * a.segments + segment) * rows * cols
                        : p.first ? p.first + at : nullptr;
    if (from && !p.states && p.first_across) {
      each_value([&](float& v, int row, int col) { v = from[col * rows + row]; });
    } else if (from && cols % 4 == 0 && ((uintptr_t)from & 15) == 0) {
      each_four([&](float& v0, float& v1, float& v2, float& v3, int i) {
        const float4 f = *reinterpret_cast<const float4*>(from + i);
        v0 = f.x, v1 = f.y, v2 = f.z, v3 = f.w;
      });
    } else if (from) {
      each_value([&](float& v, int row, int col) { v = from[row * cols + col]; });
    }
  }
  int stage = 0;
  bool first = kOut && p.undecayed && segment == 0;
  for (int i0 = range.begin; i0 < range.begin + live; i0 += kTok, stage ^= 1) {
    const int n = min(kTok, range.begin + live - i0);
    ops::copies_left<0>();
    __syncthreads();   // this stage's copies are there; the last one's values are used up
    copy(i0 + kTok, stage ^ 1);
    const unsigned char* from = smem + stage * raw;
    if (kOut && !x_as_is) widen(fx, from, p.x_half, n);
    if (!y_as_is) widen(fy, from + raw_x, p.y_half, n);
    if (!z_as_is) {
#pragma unroll 4
      for (int t = warp; t < n; t += warps)
        for (int e = lane; e < wide; e += 32)
          fz[t * wide + e] = e < cols ? value(from + raw_x + raw_y, p.z_half, cols, t, e) : 0.f;
    }
    __syncthreads();
    // Rows go up or down in memory.
    const int at0 = p.reverse ? n - 1 : 0, step = p.reverse ? -1 : 1;
    const float* sx = (x_as_is ? reinterpret_cast<const float*>(from) : fx) + row0 + at0 * KD;
    const float* sy = (y_as_is ? reinterpret_cast<const float*>(from + raw_x) : fy) + row0 + at0 * KD;
    const float* sz =
        (z_as_is ? reinterpret_cast<const float*>(from + raw_x + raw_y) : fz) + col0 + at0 * wide;
    long long to = 0;
    if (kOut)
      to = ((long long)bh * a.tokens + (p.reverse ? range.len - 1 - i0 : i0)) * cols + out_col;
    if (held && first) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
#pragma unroll
        for (int c = 0; c < kCols; ++c) S[i][c] = mul(S[i][c], two(exp2f(-l2), exp2f(-l2)));
      first = false;
    }
    const float g = exp2f(l2);
#pragma unroll 1
    for (int t = 0; t < n; ++t, sx += step * KD, sy += step * KD, sz += step * wide, to += step * cols) {
      if (!held) {
        if (!first) {
#pragma unroll
          for (int i = 0; i < kPairs; ++i)
#pragma unroll
            for (int c = 0; c < kCols; ++c) S[i][c] = mul(S[i][c], two(g, g));
        }
        first = false;
      }
      Two z[kCols], o[kCols];
      const float w = up[t];
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        const float4 f = *reinterpret_cast<const float4*>(sz + c);
        const float z0 = f.x * w, z1 = f.y * w, z2 = f.z * w, z3 = f.w * w;
        z[c] = two(z0, z0), z[c + 1] = two(z1, z1);
        z[c + 2] = two(z2, z2), z[c + 3] = two(z3, z3);
      }
      const ulonglong2* y2 = reinterpret_cast<const ulonglong2*>(sy);
      const ulonglong2* x2 = reinterpret_cast<const ulonglong2*>(sx);
#pragma unroll
      for (int i = 0; i < kPairs; i += 2) {
        const ulonglong2 y = y2[i / 2];
#pragma unroll
        for (int c = 0; c < kCols; ++c) S[i][c] = fma(y.x, z[c], S[i][c]);
#pragma unroll
        for (int c = 0; c < kCols; ++c) S[i + 1][c] = fma(y.y, z[c], S[i + 1][c]);
        if (kOut) {
          const ulonglong2 x = x2[i / 2];
#pragma unroll
          for (int c = 0; c < kCols; ++c) o[c] = i == 0 ? mul(x.x, S[i][c]) : fma(x.x, S[i][c], o[c]);
#pragma unroll
          for (int c = 0; c < kCols; ++c) o[c] = fma(x.y, S[i + 1][c], o[c]);
        }
      }
      if (kOut) {
        float v[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const Vec<2> both = apart(o[c]);
          v[c] = both.f[0] + both.f[1];
        }
        across_quarters(v, lane);
        const float f = down[t];
        if (out_col < cols) {
          if (p.out_half) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + to;
#pragma unroll
            for (int c = 0; c < kCols / 4; ++c)
              if (c == 0 || out_col + c < cols) out[c] = __float2bfloat16_rn(f * v[c]);
          } else {
            float* out = static_cast<float*>(p.out) + to;
#pragma unroll
            for (int c = 0; c < kCols / 4; ++c)
              if (c == 0 || out_col + c < cols) out[c] = f * v[c];
          }
        }
      }
    }
    if (held) {
      const Fade fade = n == kTok ? whole : Fade(l, n);
      const Two less = two(fade.less, fade.less), factor = two(fade.factor, fade.factor);
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
#pragma unroll
        for (int c = 0; c < kCols; ++c) S[i][c] = fma(S[i][c], less, mul(S[i][c], factor));
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
  if (to && cols % 4 == 0 && ((uintptr_t)to & 15) == 0)
    each_four([&](float v0, float v1, float v2, float v3, int i) {
      *reinterpret_cast<float4*>(to + i) = make_float4(v0 * f, v1 * f, v2 * f, v3 * f);
    });
  else if (to)
    each_value([&](float v, int row, int col) { to[row * cols + col] = v * f; });
  // Zeros for the segment's padding.
  if (kOut) {
    const long long start = (long long)bh * a.tokens;
    const long long from = (start + max(range.begin, range.len)) * cols;
    const long long to_end = (start + range.end) * cols;
    for (long long i = from + threadIdx.x; i < to_end; i += threads) {
      if (p.out_half) static_cast<uint16_t*>(p.out)[i] = 0;
      else static_cast<float*>(p.out)[i] = 0.f;
    }
  }
}

// The state before each segment, from every segment's own (in place): a thread for each value.
__global__ void __launch_bounds__(256)
decay_carry_kernel(const __grid_constant__ Args a, int tiles) {
  __shared__ Fade fades[kMostSegments];
  const Pass& p = a.pass[blockIdx.z];
  const int size = p.a * p.b, bh = blockIdx.x / tiles;
  const int i = (blockIdx.x - bh * tiles) * 256 + threadIdx.x;
  release_next();
  // The segments with tokens come first.
  if (threadIdx.x < a.segments) {
    const int live = Range(a, bh, threadIdx.x).live(a, p);
    fades[threadIdx.x] = Fade(log_decay(a, bh), live - (p.undecayed && threadIdx.x == 0 && live > 0));
  }
  __syncthreads();
  await_last();   // the segments' own states are there
  if (i >= size) return;
  float s = 0.f;
  if (p.first) {
    const int row = i / p.b, col = i - row * p.b;
    s = p.first[(long long)bh * size + (p.first_across ? col * p.a + row : i)];
  }
  float* at = p.states + (long long)bh * a.segments * size + i;
  constexpr int kAhead = 32;   // loads in flight (8: 11 us instead of 6 for 32 x 19 states of 64 x 64)
  for (int g0 = 0; g0 < a.segments; g0 += kAhead) {
    float own[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      own[u] = g0 + u < a.segments - 1 ? at[(long long)(g0 + u) * size] : 0.f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (g0 + u >= a.segments) break;
      at[(long long)(g0 + u) * size] = s;
      s = fades[g0 + u](s) + own[u];   // (a segment without tokens: s, and its own state is zeros)
    }
  }
}

// The most shared memory of any pass: two stages of fp32 rows of 128, one of them padded.
constexpr int kMostSmem = tokens_of(128) * 4 * (2 * 3 * 128 + 3 * 128 + 2);

template <int KD, int kCols>
cudaError_t launch_pass(const Args& a, int pass0, int passes, int bh, bool out, int warps, size_t smem,
                        bool early, cudaStream_t st) {
  auto kernel = out ? decay_rows_kernel<KD, kCols, true> : decay_rows_kernel<KD, kCols, false>;
  if (smem > 48 * 1024) {
    // As large as any call needs: calls at once do not set it lower for each other.
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMostSmem);
    if (e != cudaSuccess) return e;
  }
  return launch(kernel, dim3((unsigned)(bh * a.segments), 1, (unsigned)passes), 32 * warps, smem, early, st,
                a, pass0);
}

}  // namespace

cudaError_t launch_carry(const Args& a, int passes, int bh, cudaStream_t st) {
  int most = 0;
  for (int i = 0; i < passes; ++i) most = std::max(most, a.pass[i].a * a.pass[i].b);
  const int tiles = (most + 255) / 256;
  return launch(decay_carry_kernel, dim3((unsigned)(bh * tiles), 1, (unsigned)passes), 256, 0, true, st, a,
                tiles);
}

cudaError_t launch_rows(const Args& a, int passes, int bh, cudaStream_t st) {
  for (int stage = a.segments > 1 ? 0 : 2; stage < 3; ++stage) {
    if (stage == 1) {
      const cudaError_t e = launch_carry(a, passes, bh, st);
      if (e != cudaSuccess) return e;
      continue;
    }
    // Passes of the same padded rows in one launch.
    for (int i = 0; i < passes;) {
      const int n = rows_together(i, passes, [&](int k) { return a.pass[k].a; });
      int cols = 0;
      for (int j = i; j < i + n; ++j) cols = std::max(cols, a.pass[j].b);
      const RowsShape shape = rows_shape(a.pass[i].a, cols);
      const int kd = shape.rows, tok = tokens_of(kd), warps = shape.warps;
      size_t smem = 0;
      const bool out = stage == 2, early = out && i == 0 && a.segments > 1;   // right after the carry
      for (int j = i; j < i + n; ++j) {
        const Pass& p = a.pass[j];
        const size_t x = stage == 2 ? align_up((size_t)tok * p.a * (p.x_half ? 2 : 4), 16) : 0;
        const size_t y = align_up((size_t)tok * p.a * (p.y_half ? 2 : 4), 16);
        const size_t z = align_up((size_t)tok * p.b * (p.z_half ? 2 : 4), 16);
        const size_t padded_x = out && (p.x_half || p.a != kd) ? kd : 0;
        const size_t padded_y = p.y_half || p.a != kd ? kd : 0;
        smem = std::max(smem, 2 * (x + y + z) + sizeof(float) * tok * (padded_x + padded_y));
      }
      cudaError_t e;
      smem += sizeof(float) * tok * (warps * shape.cols + 2);
      switch (kd * 2 + (shape.cols == 64)) {
        case 32: e = launch_pass<16, 4>(a, i, n, bh, out, warps, smem, early, st); break;
        case 33: e = launch_pass<16, 8>(a, i, n, bh, out, warps, smem, early, st); break;
        case 64: e = launch_pass<32, 4>(a, i, n, bh, out, warps, smem, early, st); break;
        case 65: e = launch_pass<32, 8>(a, i, n, bh, out, warps, smem, early, st); break;
        case 96: e = launch_pass<48, 4>(a, i, n, bh, out, warps, smem, early, st); break;
        case 128: e = launch_pass<64, 4>(a, i, n, bh, out, warps, smem, early, st); break;
        case 160: e = launch_pass<80, 4>(a, i, n, bh, out, warps, smem, early, st); break;
        case 192: e = launch_pass<96, 4>(a, i, n, bh, out, warps, smem, early, st); break;
        default: e = launch_pass<128, 4>(a, i, n, bh, out, warps, smem, early, st); break;
      }
      if (e != cudaSuccess) return e;
      i += n;
    }
  }
  return cudaSuccess;
}

}  // namespace decay
}  // namespace lapl
