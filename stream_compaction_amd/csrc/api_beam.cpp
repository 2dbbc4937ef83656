// C ABI of beam search (declared in include/scan.h): host-side validation, then one
// launcher call.  Nothing here allocates, frees, synchronizes or throws.
#include "../../include/scan.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.hpp"
#include "launch.hpp"

namespace {

using namespace sca::api;

constexpr int64_t kMostBeams = 64, kMostCount = 64, kMostTensors = 1024;
constexpr int64_t kMostRowBytes = 1ll << 43;   // its columns' workgroups are counted in 32 bits

scan_status beam_problem(const beam_select_args* a, sca::BeamProblem* p, sca::Fmt* fmt, size_t* eb) {
  if (a == nullptr) return SCAN_EINVAL;
  if (!activation_fmt(a->dtype, fmt, eb)) return SCAN_ENOTSUP;
  if (a->beams < 1 || a->count < 1 || a->vocab < 1 || a->vocab > kMaxN) return SCAN_EINVAL;
  if (a->beams > kMostBeams || a->count > kMostCount) return SCAN_ENOTSUP;
  if (a->count > a->beams * a->vocab) return SCAN_EINVAL;
  if (a->batch < 0 || a->batch > kMaxN) return SCAN_EINVAL;
  if (a->finished != nullptr && (a->end_token < 0 || a->end_token >= a->vocab)) return SCAN_EINVAL;
  // (the logits' size counts whatever their strides, so that no product below passes 64 bits)
  if ((unsigned __int128)a->batch * (uint64_t)a->beams * (uint64_t)a->vocab * *eb >= kMaxBytes) return SCAN_EINVAL;
  *p = sca::BeamProblem{a->logits, a->scores, a->finished, a->batch, a->beams, a->vocab, a->count,
                        a->end_token, a->batch > 1 ? a->logits_stride[0] : 0,
                        a->beams > 1 ? a->logits_stride[1] : 0};
  return SCAN_OK;
}

struct Span {
  uintptr_t a, e;
  bool output;
};

}  // namespace

extern "C" {

size_t beam_select_scratch_bytes(const beam_select_args* args) {
  sca::BeamProblem p;
  sca::Fmt fmt;
  size_t eb;
  if (beam_problem(args, &p, &fmt, &eb) != SCAN_OK) return 0;
  return sca::beam_select_scratch(p, fmt);
}

scan_status beam_select(const beam_select_args* args, float* out_scores, int32_t* parents,
                        int32_t* tokens, void* scratch, size_t scratch_bytes, void* stream) {
  sca::BeamProblem p;
  sca::Fmt fmt;
  size_t eb;
  const scan_status st = beam_problem(args, &p, &fmt, &eb);
  if (st != SCAN_OK) return st;
  if (p.batch == 0) return SCAN_OK;
  const size_t need = sca::beam_select_scratch(p, fmt);
  const int64_t dims[2] = {p.batch, p.beams}, strides[2] = {p.logits_batch, p.logits_beam};
  const uint64_t rows = (uint64_t)p.batch * (uint64_t)p.beams;
  const uint64_t chosen = (uint64_t)p.batch * (uint64_t)p.count;
  Ranges r;
  r.add_strided(p.logits, dims, strides, 2, p.vocab, eb, true);
  r.add(p.scores, rows, 4, false, true);
  r.add(p.finished, rows, 1, false, false);
  r.add(out_scores, chosen, 4, true, true);
  r.add(parents, chosen, 4, true, true);
  r.add(tokens, chosen, 4, true, true);
  r.add(scratch, need, 1, true, true);
  if (!aligned(scratch, 16)) return SCAN_EINVAL;
  if (scratch_bytes < need) return SCAN_ESCRATCH;
  if (r.status() != SCAN_OK) return r.status();
  return hip_status(sca::launch_beam_select(p, fmt, out_scores, parents, tokens, scratch,
                                            (hipStream_t)stream));
}

scan_status beam_reorder(const void* const* states, void* const* new_states,
                         const int64_t* row_bytes, int64_t tensors, const int32_t* parents,
                         int64_t batch, int64_t beams, void* stream) {
  if (beams < 1 || tensors < 0 || tensors > kMostTensors) return SCAN_EINVAL;
  if (beams > kMostBeams) return SCAN_ENOTSUP;
  if (batch < 0 || batch > kMaxN) return SCAN_EINVAL;
  if (tensors == 0 || batch == 0) return SCAN_OK;
  if (states == nullptr || new_states == nullptr || row_bytes == nullptr) return SCAN_EINVAL;
  if (parents == nullptr || !aligned(parents, 4)) return SCAN_EINVAL;
  const uint64_t rows = (uint64_t)batch * (uint64_t)beams;
  Span spans[2 * kMostTensors + 1];
  int n = 0;
  spans[n++] = Span{(uintptr_t)parents, (uintptr_t)parents + 4 * rows, false};
  for (int64_t i = 0; i < tensors; ++i) {
    if (row_bytes[i] < 0 || row_bytes[i] >= kMostRowBytes) return SCAN_EINVAL;
    const unsigned __int128 bytes = (unsigned __int128)row_bytes[i] * rows;
    if (bytes >= kMaxBytes) return SCAN_EINVAL;
    if (bytes == 0) continue;
    if (states[i] == nullptr || new_states[i] == nullptr) return SCAN_EINVAL;
    const uintptr_t from = (uintptr_t)states[i], to = (uintptr_t)new_states[i];
    if (from != to) spans[n++] = Span{from, from + (uintptr_t)bytes, false};
    spans[n++] = Span{to, to + (uintptr_t)bytes, true};
  }
  // in the order of their starts: an output begins behind all before it, an input
  // behind all outputs
  std::sort(spans, spans + n, [](const Span& x, const Span& y) { return x.a < y.a; });
  uintptr_t any = 0, out = 0;
  for (int i = 0; i < n; ++i) {
    if (spans[i].a < (spans[i].output ? any : out)) return SCAN_EALIAS;
    any = std::max(any, spans[i].e);
    if (spans[i].output) out = std::max(out, spans[i].e);
  }
  return hip_status(sca::launch_beam_reorder(states, new_states, row_bytes, tensors, parents, batch,
                                             beams, (hipStream_t)stream));
}

}  // extern "C"
