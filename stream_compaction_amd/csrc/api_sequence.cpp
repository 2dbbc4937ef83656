// C ABI of the sequence operators (declared in include/scan.h): host-side
// validation, then one launcher call.  Nothing here allocates, frees,
// synchronizes or throws.
#include "../../include/scan.h"

#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "launch.hpp"

namespace {

using sca::api::aligned;
using sca::api::hip_status;

constexpr int64_t kMaxN = 2147483647;        // INT32_MAX
constexpr int64_t kMaxChannels = 1ll << 22;
constexpr uint64_t kMaxBytes = 1ull << 47;   // a device address

bool activation_fmt(scan_dtype d, sca::Fmt* f, size_t* bytes) {
  switch (d) {
    case SCAN_F32: *f = sca::Fmt::F32; *bytes = 4; return true;
    case SCAN_F16: *f = sca::Fmt::F16; *bytes = 2; return true;
    case SCAN_BF16: *f = sca::Fmt::BF16; *bytes = 2; return true;
    default: return false;
  }
}

// The arrays of one call, checked as they are added: null (when required),
// alignment, size; then outputs against everything.
class Ranges {
 public:
  // A contiguous array of count elements.
  void add(const void* p, uint64_t count, size_t eb, bool output, bool required) {
    add_bytes(p, (unsigned __int128)count * eb, eb, output, required);
  }
  // dims[i] entries strides[i] elements apart, then `inner` contiguous ones.
  void add_strided(const void* p, const int64_t* dims, const int64_t* strides, int nd,
                   int64_t inner, size_t eb, bool required) {
    unsigned __int128 count = (unsigned __int128)inner;
    for (int i = 0; i < nd; ++i) {
      if (strides[i] < 0) {
        status_ = SCAN_EINVAL;
        return;
      }
      if (dims[i] == 0) count = 0;
    }
    if (count != 0)
      for (int i = 0; i < nd; ++i)
        count += (unsigned __int128)(dims[i] - 1) * (unsigned __int128)strides[i];
    add_bytes(p, count * eb, eb, false, required);
  }
  scan_status status() const {
    if (status_ != SCAN_OK) return status_;
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < n_; ++j)
        if (i != j && r_[i].output && r_[i].a < r_[j].e && r_[j].a < r_[i].e) return SCAN_EALIAS;
    return SCAN_OK;
  }

 private:
  struct Range {
    uintptr_t a, e;
    bool output;
  };
  void add_bytes(const void* p, unsigned __int128 bytes, size_t eb, bool output, bool required) {
    if (bytes >= kMaxBytes) {
      status_ = SCAN_EINVAL;
      return;
    }
    if (bytes == 0) return;
    if (p == nullptr) {
      if (required) status_ = SCAN_EINVAL;
      return;
    }
    if (!aligned(p, eb)) {
      status_ = SCAN_EINVAL;
      return;
    }
    r_[n_++] = Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, output};
  }
  Range r_[24];
  int n_ = 0;
  scan_status status_ = SCAN_OK;
};

// Whether [batch, length, channels] has a size below kMaxBytes.  (Its factors'
// product can pass 64 bits; below kMaxBytes, no product of sizes in this file
// does: a scan's rows of B and C and its kept states are at most 2^6 times as much,
// its state is at most 2^31 2^22 2^6 elements.)
bool activations_fit(int64_t batch, int64_t length, int64_t channels, size_t eb) {
  return (unsigned __int128)batch * (unsigned __int128)length * (unsigned __int128)channels * eb <
         kMaxBytes;
}

// Sizes and types of a convolution; with `step`, of one token.
scan_status conv_problem(const causal_conv_args* a, bool step, sca::ConvProblem* p, sca::Fmt* fmt,
                         size_t* eb) {
  if (a == nullptr) return SCAN_EINVAL;
  if (!activation_fmt(a->dtype, fmt, eb)) return SCAN_ENOTSUP;
  if (a->width < 1 || a->width > 8) return SCAN_ENOTSUP;
  if (a->silu != 0 && a->silu != 1) return SCAN_EINVAL;
  const int64_t length = step ? 1 : a->length;
  if (a->batch < 0 || a->batch > kMaxN || length < 0 || length > kMaxN) return SCAN_EINVAL;
  if (a->channels < 1 || a->channels > kMaxChannels) return SCAN_EINVAL;
  if (!activations_fit(a->batch, length, a->channels, *eb)) return SCAN_EINVAL;
  p->x = a->x;
  p->weight = a->weight;
  p->bias = a->bias;
  p->initial_state = step ? nullptr : a->initial_state;
  p->lengths = step ? nullptr : a->lengths;
  p->batch = a->batch;
  p->length = length;
  p->channels = a->channels;
  p->width = a->width;
  // the stride of an axis with one entry means nothing: it must not decide alignment
  p->x_batch = a->batch > 1 ? a->x_stride[0] : 0;
  p->x_token = length > 1 ? a->x_stride[1] : 0;
  p->silu = a->silu == 1;
  return SCAN_OK;
}

void conv_inputs(const sca::ConvProblem& p, size_t eb, Ranges* r) {
  const int64_t dims[2] = {p.batch, p.length}, xs[2] = {p.x_batch, p.x_token};
  r->add_strided(p.x, dims, xs, 2, p.channels, eb, true);
  r->add(p.weight, (uint64_t)(p.channels * p.width), 4, false, true);
  r->add(p.bias, (uint64_t)p.channels, 4, false, false);
  r->add(p.initial_state, (uint64_t)p.batch * (uint64_t)((p.width - 1) * p.channels), eb, false,
         false);
  r->add(p.lengths, (uint64_t)p.batch, 4, false, false);
}

scan_status scan_problem(const selective_scan_args* a, bool step, sca::ScanProblem* p,
                         sca::Fmt* fmt, size_t* eb) {
  if (a == nullptr) return SCAN_EINVAL;
  if (!activation_fmt(a->dtype, fmt, eb)) return SCAN_ENOTSUP;
  if (a->states < 1 || a->states > 64) return SCAN_ENOTSUP;
  if (a->softplus != 0 && a->softplus != 1) return SCAN_EINVAL;
  const int64_t length = step ? 1 : a->length;
  if (a->batch < 0 || a->batch > kMaxN || length < 0 || length > kMaxN) return SCAN_EINVAL;
  if (a->channels < 1 || a->channels > kMaxChannels) return SCAN_EINVAL;
  if (a->groups < 1 || a->channels % a->groups != 0) return SCAN_EINVAL;
  if (!activations_fit(a->batch, length, a->channels, *eb)) return SCAN_EINVAL;
  *p = sca::ScanProblem{
      a->x, a->dt, a->B, a->C, a->z, a->A, a->D, a->dt_bias,
      step ? nullptr : a->initial_state, step ? nullptr : a->lengths,
      a->batch, length, a->channels, a->states, a->groups,
      a->x_stride[0], a->x_stride[1], a->dt_stride[0], a->dt_stride[1], a->z_stride[0],
      a->z_stride[1], a->B_stride[0], a->B_stride[1], a->B_stride[2], a->C_stride[0],
      a->C_stride[1], a->C_stride[2], a->softplus == 1};
  // the stride of an axis with one entry means nothing: it must not decide alignment
  if (length <= 1) p->x_token = p->dt_token = p->z_token = p->B_token = p->C_token = 0;
  if (a->batch <= 1) p->x_batch = p->dt_batch = p->z_batch = p->B_batch = p->C_batch = 0;
  if (a->groups == 1) p->B_group = p->C_group = 0;
  return SCAN_OK;
}

void scan_inputs(const sca::ScanProblem& p, size_t eb, Ranges* r) {
  const int64_t dims[3] = {p.batch, p.length, p.groups};
  const int64_t xs[2] = {p.x_batch, p.x_token}, ds[2] = {p.dt_batch, p.dt_token};
  const int64_t zs[2] = {p.z_batch, p.z_token};
  const int64_t Bs[3] = {p.B_batch, p.B_token, p.B_group}, Cs[3] = {p.C_batch, p.C_token, p.C_group};
  r->add_strided(p.x, dims, xs, 2, p.channels, eb, true);
  r->add_strided(p.dt, dims, ds, 2, p.channels, eb, true);
  if (p.z != nullptr) r->add_strided(p.z, dims, zs, 2, p.channels, eb, true);
  r->add_strided(p.B, dims, Bs, 3, p.states, eb, true);
  r->add_strided(p.C, dims, Cs, 3, p.states, eb, true);
  r->add(p.A, (uint64_t)(p.channels * p.states), 4, false, true);
  r->add(p.D, (uint64_t)p.channels, 4, false, false);
  r->add(p.dt_bias, (uint64_t)p.channels, 4, false, false);
  r->add(p.initial_state, (uint64_t)p.batch * (uint64_t)(p.channels * p.states), 4, false, false);
  r->add(p.lengths, (uint64_t)p.batch, 4, false, false);
}

// Float32 values of the states that a scan keeps for its gradient.
uint64_t starts_count(const sca::ScanProblem& p) {
  const int64_t blocks = (p.length + sca::kScanKeepTokens - 1) / sca::kScanKeepTokens;
  return (uint64_t)(p.batch * blocks) * (uint64_t)(p.channels * p.states);
}

}  // namespace

extern "C" {

scan_status causal_conv(const causal_conv_args* args, void* y, void* final_state, void* stream) {
  sca::ConvProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = conv_problem(args, false, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (p.batch == 0) return SCAN_OK;
  Ranges r;
  conv_inputs(p, eb, &r);
  r.add(y, (uint64_t)p.batch * (uint64_t)p.length * (uint64_t)p.channels, eb, true, true);
  r.add(final_state, (uint64_t)p.batch * (uint64_t)((p.width - 1) * p.channels), eb, true, false);
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(sca::launch_conv(p, fmt, y, final_state, (hipStream_t)stream));
}

size_t causal_conv_grad_scratch_bytes(const causal_conv_args* args) {
  sca::ConvProblem p;
  sca::Fmt fmt;
  size_t eb;
  if (conv_problem(args, false, &p, &fmt, &eb) != SCAN_OK) return 0;
  return sca::conv_grad_scratch(p);
}

scan_status causal_conv_grad(const causal_conv_args* args, const void* dy,
                             const int64_t* dy_stride, const void* dfinal, void* dx,
                             float* dweight, float* dbias, void* dinitial, void* scratch,
                             size_t scratch_bytes, void* stream) {
  sca::ConvProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = conv_problem(args, false, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (dy_stride == nullptr) return SCAN_EINVAL;
  const size_t need = sca::conv_grad_scratch(p);
  const uint64_t state = (uint64_t)p.batch * (uint64_t)((p.width - 1) * p.channels);
  const int64_t dims[2] = {p.batch, p.length};
  Ranges r;
  conv_inputs(p, eb, &r);
  r.add_strided(dy, dims, dy_stride, 2, p.channels, eb, true);
  r.add(dfinal, state, eb, false, false);
  r.add(dx, (uint64_t)p.batch * (uint64_t)p.length * (uint64_t)p.channels, eb, true, true);
  r.add(dweight, (uint64_t)(p.channels * p.width), 4, true, true);
  r.add(dbias, (uint64_t)p.channels, 4, true, false);
  r.add(dinitial, state, eb, true, false);
  r.add(scratch, need, 1, true, true);
  if (!aligned(scratch, 16)) return SCAN_EINVAL;
  if (scratch_bytes < need) return SCAN_ESCRATCH;
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(sca::launch_conv_grad(p, fmt, dy, dy_stride[0], dy_stride[1], dfinal, dx,
                                          dweight, dbias, dinitial, scratch, (hipStream_t)stream));
}

scan_status causal_conv_step(const causal_conv_args* args, const void* state, void* new_state,
                             void* y, void* stream) {
  sca::ConvProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = conv_problem(args, true, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (p.batch * p.channels > kMaxN) return SCAN_EINVAL;
  if (p.batch == 0) return SCAN_OK;
  const uint64_t count = (uint64_t)p.batch * (uint64_t)((p.width - 1) * p.channels);
  Ranges r;
  conv_inputs(p, eb, &r);
  if (state != new_state) r.add(state, count, eb, false, true);
  r.add(new_state, count, eb, true, true);
  r.add(y, (uint64_t)p.batch * (uint64_t)p.channels, eb, true, true);
  if (count > 0 && state == nullptr) return SCAN_EINVAL;
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(sca::launch_conv_step(p, fmt, state, new_state, y, (hipStream_t)stream));
}

size_t selective_scan_starts_bytes(const selective_scan_args* args) {
  sca::ScanProblem p;
  sca::Fmt fmt;
  size_t eb;
  if (scan_problem(args, false, &p, &fmt, &eb) != SCAN_OK) return 0;
  const uint64_t bytes = starts_count(p) * 4;
  return bytes < kMaxBytes ? bytes : 0;
}

static scan_status scan_call(const selective_scan_args* args, void* y, float* final_state,
                             float* starts, bool split, void* scratch, size_t scratch_bytes,
                             void* stream) {
  sca::ScanProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = scan_problem(args, false, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (p.batch == 0) return SCAN_OK;
  const size_t need = split ? sca::selective_scan_scratch(p) : 0;
  Ranges r;
  scan_inputs(p, eb, &r);
  r.add(y, (uint64_t)p.batch * (uint64_t)p.length * (uint64_t)p.channels, eb, true, true);
  r.add(final_state, (uint64_t)p.batch * (uint64_t)(p.channels * p.states), 4, true, false);
  if (starts != nullptr) r.add(starts, starts_count(p), 4, true, false);
  r.add(scratch, need, 1, true, true);
  if (need > 0 && !aligned(scratch, 16)) return SCAN_EINVAL;
  if (scratch_bytes < need) return SCAN_ESCRATCH;
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(sca::launch_selective_scan(p, fmt, y, final_state, starts,
                                               need > 0 ? scratch : nullptr, (hipStream_t)stream));
}

scan_status selective_scan(const selective_scan_args* args, void* y, float* final_state,
                           float* starts, void* stream) {
  return scan_call(args, y, final_state, starts, false, nullptr, 0, stream);
}

size_t selective_scan_split_scratch_bytes(const selective_scan_args* args) {
  sca::ScanProblem p;
  sca::Fmt fmt;
  size_t eb;
  if (scan_problem(args, false, &p, &fmt, &eb) != SCAN_OK) return 0;
  return sca::selective_scan_scratch(p);
}

scan_status selective_scan_split(const selective_scan_args* args, void* y, float* final_state,
                                 float* starts, void* scratch, size_t scratch_bytes, void* stream) {
  return scan_call(args, y, final_state, starts, true, scratch, scratch_bytes, stream);
}

size_t selective_scan_grad_scratch_bytes(const selective_scan_args* args) {
  sca::ScanProblem p;
  sca::Fmt fmt;
  size_t eb;
  if (scan_problem(args, false, &p, &fmt, &eb) != SCAN_OK) return 0;
  return sca::selective_scan_grad_scratch(p);
}

scan_status selective_scan_grad(const selective_scan_args* args, const selective_scan_grads* grads,
                                void* scratch, size_t scratch_bytes, void* stream) {
  sca::ScanProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = scan_problem(args, false, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (grads == nullptr) return SCAN_EINVAL;
  if ((p.z != nullptr) != (grads->dz != nullptr) && p.batch > 0 && p.length > 0) return SCAN_EINVAL;
  const size_t need = sca::selective_scan_grad_scratch(p);
  const uint64_t tokens = (uint64_t)p.batch * (uint64_t)p.length;
  const uint64_t state = (uint64_t)p.batch * (uint64_t)(p.channels * p.states);
  const int64_t dims[2] = {p.batch, p.length};
  Ranges r;
  scan_inputs(p, eb, &r);
  r.add_strided(grads->dy, dims, grads->dy_stride, 2, p.channels, eb, true);
  r.add(grads->dfinal, state, 4, false, false);
  r.add(grads->starts, starts_count(p), 4, false, true);
  r.add(grads->dx, tokens * (uint64_t)p.channels, eb, true, true);
  r.add(grads->ddt, tokens * (uint64_t)p.channels, eb, true, true);
  r.add(grads->dz, tokens * (uint64_t)p.channels, eb, true, false);
  r.add(grads->dB, tokens * (uint64_t)(p.groups * p.states), eb, true, true);
  r.add(grads->dC, tokens * (uint64_t)(p.groups * p.states), eb, true, true);
  r.add(grads->dA, (uint64_t)(p.channels * p.states), 4, true, true);
  r.add(grads->dD, (uint64_t)p.channels, 4, true, false);
  r.add(grads->ddt_bias, (uint64_t)p.channels, 4, true, false);
  r.add(grads->dinitial, state, 4, true, false);
  r.add(scratch, need, 1, true, true);
  if (!aligned(scratch, 16)) return SCAN_EINVAL;
  if (scratch_bytes < need) return SCAN_ESCRATCH;
  if (r.status() != SCAN_OK) return r.status();
  const sca::ScanGrads g{grads->dy, grads->dy_stride[0], grads->dy_stride[1], grads->dfinal,
                         grads->starts, grads->dx, grads->ddt, grads->dB, grads->dC, grads->dz,
                         grads->dA, grads->dD, grads->ddt_bias, grads->dinitial};
  return hip_status(sca::launch_selective_scan_grad(p, fmt, g, scratch, (hipStream_t)stream));
}

scan_status selective_scan_step(const selective_scan_args* args, const float* state,
                                float* new_state, void* y, void* stream) {
  sca::ScanProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = scan_problem(args, true, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (p.batch * p.channels > kMaxN / 16) return SCAN_EINVAL;
  if (p.batch == 0) return SCAN_OK;
  const uint64_t count = (uint64_t)p.batch * (uint64_t)(p.channels * p.states);
  Ranges r;
  scan_inputs(p, eb, &r);
  if (state != new_state) r.add(state, count, 4, false, true);
  r.add(new_state, count, 4, true, true);
  r.add(y, (uint64_t)p.batch * (uint64_t)p.channels, eb, true, true);
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(
      sca::launch_selective_scan_step(p, fmt, state, new_state, y, (hipStream_t)stream));
}

static scan_status embedding_sizes(int64_t tokens, int64_t rows, int64_t channels,
                                   int64_t row_stride, scan_dtype id_dtype) {
  if (id_dtype != SCAN_I32 && id_dtype != SCAN_I64) return SCAN_ENOTSUP;
  if (tokens < 0 || tokens > kMaxN || rows < 1 || rows > kMaxN) return SCAN_EINVAL;
  if (channels < 1 || channels > kMaxChannels || row_stride < 0) return SCAN_EINVAL;
  return SCAN_OK;
}

scan_status embedding(const void* weight, const void* ids, void* out, int64_t tokens, int64_t rows,
                      int64_t channels, int64_t row_stride, scan_dtype dtype, scan_dtype id_dtype,
                      float scale, void* stream) {
  sca::Fmt fmt;
  size_t eb;
  if (!activation_fmt(dtype, &fmt, &eb)) return SCAN_ENOTSUP;
  const scan_status st =
      embedding_sizes(tokens, rows, channels, row_stride, id_dtype);
  if (st != SCAN_OK) return st;
  if (tokens == 0) return SCAN_OK;
  const bool wide = id_dtype == SCAN_I64;
  Ranges r;
  r.add_strided(weight, &rows, &row_stride, 1, channels, eb, true);
  r.add(ids, (uint64_t)tokens, wide ? 8 : 4, false, true);
  r.add(out, (uint64_t)tokens * (uint64_t)channels, eb, true, true);
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(sca::launch_embedding(weight, ids, wide, out, tokens, rows, channels,
                                          row_stride, fmt, scale, (hipStream_t)stream));
}

size_t embedding_grad_scratch_bytes(int64_t tokens, int64_t rows, int64_t channels) {
  if (tokens < 0 || tokens > kMaxN || rows < 1 || rows > kMaxN || channels < 1 ||
      channels > kMaxChannels)
    return 0;
  return sca::embedding_grad_scratch(tokens, rows, channels);
}

scan_status embedding_grad(const void* dout, const void* ids, void* dweight, int64_t tokens,
                           int64_t rows, int64_t channels, int64_t row_stride, scan_dtype dtype,
                           scan_dtype id_dtype, scan_dtype out_dtype, float scale, void* scratch,
                           size_t scratch_bytes, void* stream) {
  sca::Fmt fmt, out_fmt;
  size_t eb, ob;
  if (!activation_fmt(dtype, &fmt, &eb) || !activation_fmt(out_dtype, &out_fmt, &ob))
    return SCAN_ENOTSUP;
  if (out_dtype != dtype && out_dtype != SCAN_F32) return SCAN_ENOTSUP;
  const scan_status st =
      embedding_sizes(tokens, rows, channels, row_stride, id_dtype);
  if (st != SCAN_OK) return st;
  const bool wide = id_dtype == SCAN_I64;
  const size_t need = sca::embedding_grad_scratch(tokens, rows, channels);
  Ranges r;
  r.add_strided(dout, &tokens, &row_stride, 1, channels, eb, true);
  r.add(ids, (uint64_t)tokens, wide ? 8 : 4, false, true);
  r.add(dweight, (uint64_t)rows * (uint64_t)channels, ob, true, true);
  r.add(scratch, need, 1, true, true);
  if (!aligned(scratch, 16)) return SCAN_EINVAL;
  if (scratch_bytes < need) return SCAN_ESCRATCH;
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(sca::launch_embedding_grad(dout, ids, wide, dweight, tokens, rows, channels,
                                               row_stride, fmt, out_fmt, scale, scratch,
                                               (hipStream_t)stream));
}

}  // extern "C"
