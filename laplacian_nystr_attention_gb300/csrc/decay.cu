// decay.cu -- lapl_decay_* of include/lapl_ops.h: linear attention with a decay for each head.  The
// kernels are in decay_tc.cu (chunks on the tensor cores) and decay_rows.cu (token by token);
// decay.cuh has the formulas.
#include <algorithm>
#include <cmath>
#include <new>

#include "decay.cuh"

struct lapl_decay_plan {
  lapl_decay_config cfg;
  lapl_decay_plan_info info;
  int row_segments, backward_row_segments;   // where the tensor-core kernels cannot run
  int bh;
  int sms, device;
  unsigned* dev_err;
  unsigned long long wait_ns;
  int skip_last;
  char last_error[lapl::ops::kErrorText];
};

using namespace lapl;

namespace {

constexpr unsigned long long kWaitNs = 1000000000ull;

lapl_status validate(const lapl_decay_config* c) {
  if (!c || c->batch < 0 || c->heads < 1 || c->tokens < 1 || c->key_dim < 1 || c->value_dim < 1 ||
      c->reverse < 0 || c->reverse > 1 || !std::isfinite(c->scale))
    return LAPL_ERR_INVALID_ARG;
  if (!ops::is_float_dtype(c->in_dtype) || !ops::is_float_dtype(c->out_dtype) ||
      !ops::is_float_dtype(c->grad_dtype))
    return LAPL_ERR_INVALID_ARG;
  if (c->key_dim > LAPL_DECAY_MAX_DIM || c->value_dim > LAPL_DECAY_MAX_DIM ||
      c->tokens > (1 << 30) || (long long)c->batch * c->heads > (1 << 22))
    return LAPL_ERR_UNSUPPORTED;
  return LAPL_OK;
}

// Segments of a sequence token by token.  A segment's warps walk its tokens alone; by registers 16, 12 or
// 8 warps of an SM are resident.  Times in us, about as measured: a token of the outputs 0.35, of the
// segments' sums 0.2, a launch 3, its CTAs 2, and 0.05 for each segment.  (16 sequences of 3136 tokens of
// 32 x 32 in fp32: 33 us in 98 segments, 45 in 64, 68 in 32, 120 in 16.)
int row_segments(int tokens, long long bh, int rows, int cols, int sms, double* us) {
  const int per_warp = rows <= 32 && cols > 32 ? 64 : 32;
  const long long warps = bh * ((cols + per_warp - 1) / per_warp);
  const long long room = (rows <= 64 ? 16LL : 48LL) * sms;
  int best = 1;
  double least = 0;
  for (int g = 1; g <= decay::kMostSegments && (g == 1 || tokens / g >= 16); ++g) {
    const double waves = (double)((warps * g + room - 1) / room);
    const int per = (tokens + g - 1) / g;
    const double token = std::max(rows, 16) / 32.0;
    double time = waves * (2.0 + 0.35 * token * per);
    if (g > 1) time += waves * (2.0 + 0.2 * token * per) + 6.0 + 0.05 * g;
    if (g == 1 || time < least) least = time, best = g;
  }
  *us = least;
  return best;
}

// Segments of a sequence in chunks: a CTA of an SM walks its chunks, of 64 columns of the state.  Times in
// us, as measured, for rows of up to 64 values and for longer ones, and the same for fp32 outputs: a chunk of
// the outputs and what a CTA has besides, the same of the segments' sums; the launch between 4, and 0.4 for each
// segment.  (4 x 8 sequences of 128 chunks of 64 x 64: 110 us in 4 segments, 249 in 1, 121 in 9.)
int chunk_segments(int tokens, long long bh, int rows, int cols, bool exact, int sms, double* us) {
  static const double kTimes[2][2][4] = {{{2.05, 4.5, 1.25, 3.0}, {3.6, 6.0, 1.9, 4.0}},
                                         {{3.4, 5.5, 1.25, 3.0}, {4.0, 6.0, 1.9, 4.0}}};
  const double* t = kTimes[exact][rows > 64];
  const int chunks = (tokens + decay::kTcChunk - 1) / decay::kTcChunk;
  bh *= (cols + 63) / 64;
  int best = 1;
  double least = 0;
  for (int g = 1; g <= 64 && g <= chunks; ++g) {
    const int per = (chunks + g - 1) / g, n = (chunks + per - 1) / per;
    double time = (double)((bh * n + sms - 1) / sms) * (t[1] + t[0] * per);
    if (n > 1) time += (double)((bh * (n - 1) + sms - 1) / sms) * (t[3] + t[2] * per) + 4.0 + 0.4 * n;
    if (g == 1 || time < least) least = time, best = n;
  }
  *us = least;
  return best;
}

// Tokens of a segment: whole stages or chunks.
int per_segment(int tokens, int segments, int step) {
  return ((tokens + segments - 1) / segments + step - 1) / step * step;   // (step: of a stage or chunk)
}

bool tc_sizes(const lapl_decay_config& c) {
  return c.in_dtype == LAPL_BF16 && c.key_dim % 8 == 0 && c.value_dim % 8 == 0;
}

// Segments of sequences by both kernels, and whether the tensor cores are faster where they can run: for
// short sequences, up to one chunk, a CTA's own time against that of the tokens one by one.  (64 x 64 bf16:
// 8 sequences of 16 tokens 8.3 us and 11.0, 512 of them 26 and 12.7, of 48 30 and 30.)
void choose(const lapl_decay_config& c, long long bh, int rows, int cols, bool exact, int sms, bool tc_can,
            int* row, int* segments, int* tc) {
  double row_us = 0, tc_us = 0;
  *row = row_segments(c.tokens, bh, rows, cols, sms, &row_us);
  const int chunked = chunk_segments(c.tokens, bh, rows, cols, exact, sms, &tc_us);
  *tc = tc_can && tc_us < row_us;
  *segments = *tc ? chunked : *row;
}

size_t states_bytes(const lapl_decay_plan& p, int segments) {
  return sizeof(float) * p.bh * (size_t)segments * p.cfg.key_dim * p.cfg.value_dim;
}

lapl_status check_pointers(std::initializer_list<std::pair<const void*, int>> list) {
  for (const auto& x : list)
    if (!ops::aligned(x.first, x.second)) return LAPL_ERR_ALIGNMENT;
  return LAPL_OK;
}

lapl_status check_workspace(lapl_decay_plan* p, bool backward, const void* workspace, size_t bytes) {
  size_t need[2];
  lapl_decay_workspace_size(p, &need[0], &need[1]);
  if (need[backward] == 0) return LAPL_OK;
  if (!workspace) return LAPL_ERR_INVALID_ARG;
  if (!ops::aligned(workspace, 16)) return LAPL_ERR_ALIGNMENT;
  return bytes < need[backward] ? LAPL_ERR_WORKSPACE : LAPL_OK;
}

decay::Args common(const lapl_decay_plan& p, const float* log_decay, const int* lengths) {
  decay::Args a = {};
  a.log_decay = log_decay;
  a.lengths = lengths;
  a.heads = p.cfg.heads;
  a.tokens = p.cfg.tokens;
  return a;
}
void cut(decay::Args* a, int segments, int step, int chunks) {
  a->segments = segments;
  a->per_segment = per_segment(a->tokens, segments, step);
  a->chunks = chunks;
}

}  // namespace

extern "C" {

lapl_status lapl_decay_create(const lapl_decay_config* cfg, lapl_decay_handle* out) {
  if (!out) return LAPL_ERR_INVALID_ARG;
  *out = nullptr;
  const lapl_status st = validate(cfg);
  if (st != LAPL_OK) return st;
  int sms = 0, device = 0;
  unsigned* dev_err = nullptr;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) e = device_error_word(&dev_err);
  if (e != cudaSuccess) return LAPL_ERR_CUDA;
  lapl_decay_plan* p = new (std::nothrow) lapl_decay_plan();
  if (!p) return LAPL_ERR_INVALID_ARG;
  p->cfg = *cfg;
  p->bh = cfg->batch * cfg->heads;
  p->sms = sms;
  p->device = device;
  p->dev_err = dev_err;
  p->wait_ns = kWaitNs;
  choose(*cfg, p->bh, cfg->key_dim, cfg->value_dim, cfg->out_dtype == LAPL_F32, sms, tc_sizes(*cfg),
         &p->row_segments, &p->info.segments, &p->info.tensor_cores);
  // The backward's three passes go side by side.
  const int most = std::max(cfg->key_dim, cfg->value_dim);
  choose(*cfg, 3LL * p->bh, most, most, false, sms, tc_sizes(*cfg) && cfg->grad_dtype == LAPL_BF16,
         &p->backward_row_segments, &p->info.backward_segments, &p->info.backward_tensor_cores);
  *out = p;
  return LAPL_OK;
}

lapl_status lapl_decay_workspace_size(lapl_decay_handle p, size_t* forward_bytes,
                                      size_t* backward_bytes) {
  if (!p || !forward_bytes || !backward_bytes) return LAPL_ERR_INVALID_ARG;
  const int f = std::max(p->info.segments, p->row_segments);
  const int b = std::max(p->info.backward_segments, p->backward_row_segments);
  *forward_bytes = f > 1 ? align_up(states_bytes(*p, f), kAlign) : 0;
  *backward_bytes = decay::kMaxPasses * align_up(states_bytes(*p, b), kAlign);
  return LAPL_OK;
}

lapl_status lapl_decay_forward(lapl_decay_handle p, const void* q, const void* k, const void* v,
                               const float* log_decay, const float* state, const int* lengths,
                               void* out, float* final_state, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  const lapl_decay_config& c = p->cfg;
  if (c.batch > 0 && (!q || !k || !v || !log_decay || !out)) return LAPL_ERR_INVALID_ARG;
  const int i = ops::dtype_bytes(c.in_dtype), o = ops::dtype_bytes(c.out_dtype);
  lapl_status st = check_pointers({{q, i}, {k, i}, {v, i}, {out, o}, {log_decay, 4}, {state, 4},
                                   {lengths, 4}, {final_state, 4}});
  if (st == LAPL_OK && c.batch > 0) st = check_workspace(p, false, workspace, workspace_bytes);
  if (st == LAPL_OK) st = ops::check_device(p->device, p->last_error, "decay_forward/device");
  if (st != LAPL_OK || c.batch == 0) return st;
  decay::Args a = common(*p, log_decay, lengths);
  decay::Pass& f = a.pass[0];
  f.x = q, f.y = k, f.z = v, f.out = out;
  f.first = state, f.last = final_state;
  f.a = c.key_dim, f.b = c.value_dim;
  f.x_half = f.y_half = f.z_half = c.in_dtype == LAPL_BF16;
  f.out_half = c.out_dtype == LAPL_BF16;
  f.reverse = c.reverse;
  f.zs = 1.f, f.os = c.scale;
  const bool tc = p->info.tensor_cores && decay::tc_fits(a, 1);
  if (tc) cut(&a, p->info.segments, decay::kTcChunk, 1);
  else cut(&a, p->row_segments, 16, 0);
  f.states = a.segments > 1 ? static_cast<float*>(workspace) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = tc ? decay::launch_tc(a, 1, p->bh, p->dev_err, p->wait_ns, p->skip_last, s)
                           : decay::launch_rows(a, 1, p->bh, s);
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "decay_forward");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

lapl_status lapl_decay_backward(lapl_decay_handle p, const void* q, const void* k, const void* v,
                                const float* log_decay, const float* state, const int* lengths,
                                const void* dout, const float* dfinal, void* dq, void* dk, void* dv,
                                float* dstate, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!p) return LAPL_ERR_INVALID_ARG;
  const lapl_decay_config& c = p->cfg;
  if (c.batch > 0 && (!q || !k || !v || !log_decay || !dout || !dq || !dk || !dv))
    return LAPL_ERR_INVALID_ARG;
  const int i = ops::dtype_bytes(c.in_dtype), g = ops::dtype_bytes(c.grad_dtype);
  lapl_status st = check_pointers({{q, i}, {k, i}, {v, i}, {dout, g}, {dq, g}, {dk, g}, {dv, g},
                                   {log_decay, 4}, {state, 4}, {lengths, 4}, {dfinal, 4}, {dstate, 4}});
  if (st == LAPL_OK && c.batch > 0) st = check_workspace(p, true, workspace, workspace_bytes);
  if (st == LAPL_OK) st = ops::check_device(p->device, p->last_error, "decay_backward/device");
  if (st != LAPL_OK || c.batch == 0) return st;
  decay::Args a = common(*p, log_decay, lengths);
  const int in = c.in_dtype == LAPL_BF16, gr = c.grad_dtype == LAPL_BF16;
  const int fwd = c.reverse, back = !c.reverse;
  a.pass[0] = {dout, v, k, dq, state, nullptr, nullptr, c.value_dim, c.key_dim, gr, in, in, gr,
               fwd, 1, 0, 1.f, c.scale};
  a.pass[1] = {v, dout, q, dk, dfinal, nullptr, nullptr, c.value_dim, c.key_dim, in, gr, in, gr,
               back, 1, 1, c.scale, 1.f};
  a.pass[2] = {k, q, dout, dv, dfinal, dstate, nullptr, c.key_dim, c.value_dim, in, in, gr, gr,
               back, 0, 1, c.scale, 1.f};
  const bool tc = p->info.backward_tensor_cores && decay::tc_fits(a, 3);
  if (tc) cut(&a, p->info.backward_segments, decay::kTcChunk, 1);
  else cut(&a, p->backward_row_segments, 16, 0);
  // dstate may be dfinal: the passes that read dfinal go by a copy of it then.
  const size_t step = align_up(states_bytes(*p, a.segments), kAlign);
  if (a.segments > 1 || (dfinal && dstate == dfinal))
    for (int n = 0; n < 3; ++n)
      a.pass[n].states = reinterpret_cast<float*>(static_cast<char*>(workspace) + n * step);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = tc ? decay::launch_tc(a, 3, p->bh, p->dev_err, p->wait_ns, p->skip_last, s)
                           : decay::launch_rows(a, 3, p->bh, s);
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "decay_backward");
    return LAPL_ERR_CUDA;
  }
  return LAPL_OK;
}

lapl_status lapl_decay_plan_info_get(lapl_decay_handle p, lapl_decay_plan_info* info) {
  if (!p || !info) return LAPL_ERR_INVALID_ARG;
  *info = p->info;
  return LAPL_OK;
}

lapl_status lapl_decay_device_errors(lapl_decay_handle p, void* stream, unsigned* flags) {
  if (!p || !flags) return LAPL_ERR_INVALID_ARG;
  const lapl_status ok = ops::check_device(p->device, p->last_error, "device_errors/device");
  if (ok != LAPL_OK) return ok;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, p->dev_err, sizeof(word), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(p->dev_err, 0, sizeof(word), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    ops::set_error(p->last_error, e, "device_errors");
    return LAPL_ERR_CUDA;
  }
  *flags = word;
  if (!word) return LAPL_OK;
  snprintf(p->last_error, sizeof(p->last_error),
           "device error flags 0x%x: a bounded wait gave up in:%s%s%s", word,
           (word & kErrBitDecay) ? " the linear attention's tensor-core kernels;" : "",
           (word & kErrBitScan) ? " the recurrence's exchange between CTAs;" : "",
           (word & ~(kErrBitDecay | kErrBitScan)) ? " a kernel of the attention;" : "");
  return LAPL_ERR_DEVICE_TIMEOUT;
}

lapl_status lapl_decay_set_fault_injection(lapl_decay_handle p, unsigned long long wait_ns,
                                           int skip_last) {
  if (!p || skip_last < 0 || skip_last > 1) return LAPL_ERR_INVALID_ARG;
  p->wait_ns = wait_ns ? wait_ns : kWaitNs;
  p->skip_last = skip_last;
  return LAPL_OK;
}

const char* lapl_decay_last_error(lapl_decay_handle p) { return p ? p->last_error : ""; }

lapl_status lapl_decay_destroy(lapl_decay_handle p) {
  delete p;
  return LAPL_OK;
}

}  // extern "C"
