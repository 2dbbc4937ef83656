// C ABI of the gated scan (declared in include/scan.h): host-side validation,
// then one launcher call.  Nothing here allocates, frees, synchronizes or throws.
#include "../../include/scan.h"

#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "launch.hpp"

namespace {

using namespace sca::api;

// Sizes and types; with `step`, of one token.
scan_status gated_problem(const gated_scan_args* a, bool step, sca::GatedProblem* p, sca::Fmt* fmt,
                          size_t* eb) {
  if (a == nullptr) return SCAN_EINVAL;
  if (!activation_fmt(a->dtype, fmt, eb)) return SCAN_ENOTSUP;
  const int64_t length = step ? 1 : a->length;
  if (a->batch < 0 || a->batch > kMaxN || length < 0 || length > kMaxN) return SCAN_EINVAL;
  if (a->channels < 1 || a->channels > kMaxChannels) return SCAN_EINVAL;
  if (!activations_fit(a->batch, length, a->channels, *eb)) return SCAN_EINVAL;
  *p = sca::GatedProblem{
      a->x, a->forget, a->input_gate, a->z, a->rate, step ? nullptr : a->initial_state,
      step ? nullptr : a->lengths, a->batch, length, a->channels,
      a->x_stride[0], a->x_stride[1], a->forget_stride[0], a->forget_stride[1],
      a->input_gate_stride[0], a->input_gate_stride[1], a->z_stride[0], a->z_stride[1]};
  // the stride of an axis with one entry means nothing: it must not decide alignment
  if (length <= 1) p->x_token = p->forget_token = p->input_token = p->z_token = 0;
  if (a->batch <= 1) p->x_batch = p->forget_batch = p->input_batch = p->z_batch = 0;
  return SCAN_OK;
}

void gated_inputs(const sca::GatedProblem& p, size_t eb, Ranges* r) {
  const int64_t dims[2] = {p.batch, p.length};
  const int64_t xs[2] = {p.x_batch, p.x_token}, fs[2] = {p.forget_batch, p.forget_token};
  const int64_t is[2] = {p.input_batch, p.input_token}, zs[2] = {p.z_batch, p.z_token};
  r->add_strided(p.x, dims, xs, 2, p.channels, eb, true);
  r->add_strided(p.forget, dims, fs, 2, p.channels, eb, true);
  if (p.input_gate != nullptr) r->add_strided(p.input_gate, dims, is, 2, p.channels, eb, true);
  if (p.z != nullptr) r->add_strided(p.z, dims, zs, 2, p.channels, eb, true);
  r->add(p.rate, (uint64_t)p.channels, 4, false, false);
  r->add(p.initial_state, (uint64_t)p.batch * (uint64_t)p.channels, 4, false, false);
  r->add(p.lengths, (uint64_t)p.batch, 4, false, false);
}

// Float32 values of the states that a scan keeps for its gradient.
uint64_t starts_count(const sca::GatedProblem& p) {
  const int64_t blocks = (p.length + sca::kGatedKeepTokens - 1) / sca::kGatedKeepTokens;
  return (uint64_t)(p.batch * blocks) * (uint64_t)p.channels;
}

}  // namespace

extern "C" {

size_t gated_scan_starts_bytes(const gated_scan_args* args) {
  sca::GatedProblem p;
  sca::Fmt fmt;
  size_t eb;
  if (gated_problem(args, false, &p, &fmt, &eb) != SCAN_OK) return 0;
  const uint64_t bytes = starts_count(p) * 4;
  return bytes < kMaxBytes ? bytes : 0;
}

size_t gated_scan_scratch_bytes(const gated_scan_args* args) {
  sca::GatedProblem p;
  sca::Fmt fmt;
  size_t eb;
  if (gated_problem(args, false, &p, &fmt, &eb) != SCAN_OK) return 0;
  return sca::gated_scan_scratch(p);
}

scan_status gated_scan(const gated_scan_args* args, void* y, float* final_state, float* starts,
                       void* scratch, size_t scratch_bytes, void* stream) {
  sca::GatedProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = gated_problem(args, false, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (p.batch == 0) return SCAN_OK;
  const size_t need = sca::gated_scan_scratch(p);
  Ranges r;
  gated_inputs(p, eb, &r);
  r.add(y, (uint64_t)p.batch * (uint64_t)p.length * (uint64_t)p.channels, eb, true, true);
  r.add(final_state, (uint64_t)p.batch * (uint64_t)p.channels, 4, true, false);
  if (starts != nullptr) r.add(starts, starts_count(p), 4, true, false);
  r.add(scratch, need, 1, true, true);
  if (need > 0 && !aligned(scratch, 16)) return SCAN_EINVAL;
  if (scratch_bytes < need) return SCAN_ESCRATCH;
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(sca::launch_gated_scan(p, fmt, y, final_state, starts,
                                           need > 0 ? scratch : nullptr, (hipStream_t)stream));
}

size_t gated_scan_grad_scratch_bytes(const gated_scan_args* args) {
  sca::GatedProblem p;
  sca::Fmt fmt;
  size_t eb;
  if (gated_problem(args, false, &p, &fmt, &eb) != SCAN_OK) return 0;
  return sca::gated_scan_grad_scratch(p);
}

scan_status gated_scan_grad(const gated_scan_args* args, const gated_scan_grads* grads,
                            void* scratch, size_t scratch_bytes, void* stream) {
  sca::GatedProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = gated_problem(args, false, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (grads == nullptr) return SCAN_EINVAL;
  if (p.batch > 0 && p.length > 0) {
    if ((p.z != nullptr) != (grads->dz != nullptr)) return SCAN_EINVAL;
    if ((p.input_gate != nullptr) != (grads->dinput_gate != nullptr)) return SCAN_EINVAL;
  }
  if ((p.rate != nullptr) != (grads->drate != nullptr)) return SCAN_EINVAL;
  const size_t need = sca::gated_scan_grad_scratch(p);
  const uint64_t values = (uint64_t)p.batch * (uint64_t)p.length * (uint64_t)p.channels;
  const uint64_t state = (uint64_t)p.batch * (uint64_t)p.channels;
  const int64_t dims[2] = {p.batch, p.length};
  Ranges r;
  gated_inputs(p, eb, &r);
  r.add_strided(grads->dy, dims, grads->dy_stride, 2, p.channels, eb, true);
  r.add(grads->dfinal, state, 4, false, false);
  r.add(grads->starts, starts_count(p), 4, false, true);
  r.add(grads->dx, values, eb, true, true);
  r.add(grads->dforget, values, eb, true, true);
  r.add(grads->dinput_gate, values, eb, true, false);
  r.add(grads->dz, values, eb, true, false);
  r.add(grads->drate, (uint64_t)p.channels, 4, true, false);
  r.add(grads->dinitial, state, 4, true, false);
  r.add(scratch, need, 1, true, true);
  if (need > 0 && !aligned(scratch, 16)) return SCAN_EINVAL;
  if (scratch_bytes < need) return SCAN_ESCRATCH;
  if (r.status() != SCAN_OK) return r.status();
  const sca::GatedGrads g{grads->dy,
                          p.batch > 1 ? grads->dy_stride[0] : 0,
                          p.length > 1 ? grads->dy_stride[1] : 0,
                          grads->dfinal, grads->starts, grads->dx, grads->dforget,
                          grads->dinput_gate, grads->dz, grads->drate, grads->dinitial};
  return hip_status(sca::launch_gated_scan_grad(p, fmt, g, need > 0 ? scratch : nullptr,
                                                (hipStream_t)stream));
}

scan_status gated_scan_step(const gated_scan_args* args, const float* state, float* new_state,
                            void* y, void* stream) {
  sca::GatedProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = gated_problem(args, true, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (p.batch * p.channels > kMaxN) return SCAN_EINVAL;
  if (p.batch == 0) return SCAN_OK;
  const uint64_t count = (uint64_t)p.batch * (uint64_t)p.channels;
  Ranges r;
  gated_inputs(p, eb, &r);
  if (state != new_state) r.add(state, count, 4, false, true);
  r.add(new_state, count, 4, true, true);
  r.add(y, count, eb, true, true);
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(
      sca::launch_gated_scan_step(p, fmt, state, new_state, y, (hipStream_t)stream));
}

}  // extern "C"
