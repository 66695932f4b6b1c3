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
  int device;
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

// Rows and columns of a pass's states.
struct Size {
  int rows, cols;
};

// Tokens of a segment: whole stages or chunks (step), and the segments that are left.
int per_segment(int tokens, int segments, int step) {
  return ((tokens + segments - 1) / segments + step - 1) / step * step;
}
int segments_of(int tokens, int segments, int step) {
  const int per = per_segment(tokens, segments, step);
  return (tokens + per - 1) / per;
}

// Time in us of the passes token by token, in segments.  A token takes a warp as long as its chain of
// instructions does, or an SM as long as it takes to issue those of all its warps, whichever is longer; the
// segments' sums their chain; a launch 3.2; the states of segments, written and read twice, their bytes; and a last
// round of warps that does not fill the SMs a tenth of what it leaves empty.  Fitted to 2532 times: rows of 16 to
// 128 values, one sequence to 4096 and 16 to 16384 tokens in 1 to 128 segments, forward and backward, fp32 and bf16:
// 14% off (root mean square), 3 in 100 by a third and none by over half.  Of 130 calls that were measured in several
// numbers of segments the one it takes is 1% slower than the best, 17% at most.  (8 x 2 sequences of 3136 tokens of
// 32 x 32 in fp32: 32 us in 98 segments, 160 in 8, 816 in 1.)
double rows_time(const Size* size, int passes, bool half, int tokens, long long bh, int segments, int sms) {
  const int per = std::min(per_segment(tokens, segments, decay::kRowsStep), tokens);
  double us = 0, bytes = 0, empty = 0;
  for (int i = 0; i < passes;) {
    const int n = decay::rows_together(i, passes, [&](int k) { return size[k].rows; });
    int cols = 0;
    for (int k = i; k < i + n; ++k) cols = std::max(cols, size[k].cols);
    const decay::RowsShape s = decay::rows_shape(size[i].rows, cols);
    // Rows that have to be widened to fp32 or padded, or some of them.
    bool padded = false;
    for (int k = i; k < i + n; ++k) {
      padded = padded || size[k].rows != s.rows || size[k].cols != s.warps * s.cols;
      bytes += 16.0 * size[k].rows * size[k].cols * (double)(bh * segments);
    }
    const double widened = half ? 1.0 : padded ? 0.6 : 0.0;
    const double warps = (double)(bh * n * segments * s.warps) / sms;
    const double chain = 0.22 + 0.0016 * s.rows + 0.2 * widened;
    const double issue = (0.019 + 0.0005 * s.rows) * (s.cols == 64 ? 1.8 : 1.0) * (1.0 + 0.22 * widened);
    const double rounds = warps / s.room;
    if (rounds > 1.0) empty = std::max(empty, std::ceil(rounds) / rounds - 1.0);
    us += 3.2 + per * std::max(chain, issue * warps);
    if (segments > 1) us += per * (0.105 + 0.0025 * s.rows + 0.13 * widened);
    i += n;
  }
  if (segments > 1) us += 4.0 + bytes / 3.2e6;
  return us * (1.0 + 0.1 * empty);
}

// Time in us of the passes in chunks, in segments: a CTA of an SM walks its chunks, of 64 columns of the state.
// For rows of up to 64 values and for longer ones, and the same for fp32 outputs: a chunk of the outputs and what
// a CTA has besides, the same of the segments' sums; the launch between 2, and 0.4 for each segment.  Fitted to 378
// times, 10 to 14% off and none by over 1.7.  (4 x 8 sequences of 128 chunks of 64 x 64 in bf16: 104 us in 4
// segments, 249 in 1, 121 in 9.)
double chunks_time(const Size* size, int passes, bool exact, int tokens, long long bh, int segments, int sms) {
  static const double kTimes[2][2][4] = {{{2.1, 4.1, 0.8, 4.0}, {3.75, 3.9, 1.2, 8.0}},
                                         {{3.7, 3.3, 0.85, 2.6}, {4.3, 3.7, 1.3, 8.0}}};
  int rows = 0;
  long long ctas = 0;   // of each segment
  for (int i = 0; i < passes; ++i) {
    rows = std::max(rows, size[i].rows);
    ctas += bh * ((size[i].cols + 63) / 64);
  }
  const double* t = kTimes[exact][rows > 64];
  const int per = per_segment(tokens, segments, decay::kTcChunk) / decay::kTcChunk;
  const double us = (double)((ctas * segments + sms - 1) / sms) * (t[1] + t[0] * per);
  if (segments == 1) return us;
  return us + (double)((ctas * (segments - 1) + sms - 1) / sms) * (t[3] + t[2] * per) + 2.0 + 0.4 * segments;
}

// The segments, up to `most`, that take the least time, or the fewest that take no more than `slack` of it.
template <class Time>
int best_segments(int tokens, int most, int step, double slack, Time time, double* us) {
  int best = 1;
  double least = 0;
  for (const bool choosing : {false, true}) {
    for (int i = 1, last = 0; i <= most && i <= (tokens + step - 1) / step; ++i) {
      const int g = segments_of(tokens, i, step);
      if (g == last) continue;
      last = g;
      const double t = time(g);
      if (choosing && t <= slack * least) {
        *us = t;
        return g;
      }
      if (!choosing && (g == 1 || t < least)) least = t, best = g;
    }
  }
  return best;
}

bool tc_sizes(const lapl_decay_config& c) {
  return c.in_dtype == LAPL_BF16 && c.key_dim % 8 == 0 && c.value_dim % 8 == 0;
}

// Segments of sequences by both kernels, and whether the tensor cores are faster where they can run.  (bf16,
// 8 x 16 tokens of 64 x 64: 6.9 us in chunks and 11.6 token by token; 512 x 16: 24 and 13; 512 x 128: 25 and 76;
// 512 x 16 of 128 x 128: 48 and 30; 512 x 64: 48 and 100; the backward of 512 x 128 of 128 x 128: 159 and 517.  Of
// 368 calls by both, the one taken was over a tenth slower in 3, by a fifth at most.)
// Where they are taken, the rows' kernel is left for pointers off 16 bytes, and its states have no more room than
// the other's or than `room`, the bytes of a tensor of the call.
void choose(const Size* size, int passes, int tokens, long long bh, bool half, bool exact, int sms, bool tc_can,
            size_t room, int* row, int* segments, int* tc) {
  double row_us = 0, tc_us = 0;
  *row = best_segments(tokens, decay::kMostSegments, decay::kRowsStep, 1.0, [&](int g) {
    return rows_time(size, passes, half, tokens, bh, g, sms);
  }, &row_us);
  // (The chunks' model is no finer: the backward of 32 x 16384 tokens of 64 x 64 258 us in 1 segment, 270 in 3.)
  const int chunked = best_segments(tokens, 64, decay::kTcChunk, 1.05, [&](int g) {
    return chunks_time(size, passes, exact, tokens, bh, g, sms);
  }, &tc_us);
  *tc = tc_can && tc_us < row_us;
  *segments = *tc ? chunked : *row;
  if (!*tc) return;
  const size_t states = sizeof(float) * (size_t)bh * size[0].rows * size[0].cols * passes;
  const size_t most = std::max((size_t)chunked, room / std::max<size_t>(states, 1));
  if ((size_t)*row > most) *row = segments_of(tokens, (int)most, decay::kRowsStep);
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
  a->per_segment = per_segment(a->tokens, segments, step);
  a->segments = segments;   // (as segments_of gave them: none is empty)
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
  p->device = device;
  p->dev_err = dev_err;
  p->wait_ns = kWaitNs;
  const bool half = cfg->in_dtype == LAPL_BF16, grad_half = cfg->grad_dtype == LAPL_BF16;
  const Size across = {cfg->value_dim, cfg->key_dim}, along = {cfg->key_dim, cfg->value_dim};
  const size_t room = (size_t)p->bh * cfg->tokens * std::max(cfg->key_dim, cfg->value_dim) *
                      ops::dtype_bytes(cfg->in_dtype);
  choose(&along, 1, cfg->tokens, p->bh, half, cfg->out_dtype == LAPL_F32, sms, tc_sizes(*cfg), room,
         &p->row_segments, &p->info.segments, &p->info.tensor_cores);
  // The backward's three passes go side by side.
  const Size back[3] = {across, across, along};
  choose(back, 3, cfg->tokens, p->bh, half || grad_half, false, sms, tc_sizes(*cfg) && grad_half, room,
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
  *backward_bytes = (b > 1 ? decay::kMaxPasses : 1) * align_up(states_bytes(*p, b), kAlign);
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
  else cut(&a, p->row_segments, decay::kRowsStep, 0);
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
  else cut(&a, p->backward_row_segments, decay::kRowsStep, 0);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const size_t step = align_up(states_bytes(*p, a.segments), kAlign);
  if (a.segments > 1) {
    for (int n = 0; n < 3; ++n)
      a.pass[n].states = reinterpret_cast<float*>(static_cast<char*>(workspace) + n * step);
  } else if (dfinal && dstate == dfinal) {
    // The passes that read dfinal go by a copy of it, as one of them writes dstate.
    e = cudaMemcpyAsync(workspace, dfinal, states_bytes(*p, 1), cudaMemcpyDeviceToDevice, s);
    a.pass[1].first = a.pass[2].first = static_cast<const float*>(workspace);
  }
  if (e == cudaSuccess)
    e = tc ? decay::launch_tc(a, 3, p->bh, p->dev_err, p->wait_ns, p->skip_last, s)
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
