// Internal host-side interface between the C ABI (api.cpp) and the kernel
// translation units.  Arguments reaching these launchers are already
// validated; each returns the hipError_t of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sca {

enum class Fmt : int { F32, F16, BF16, F64, I32, U32, I64, U64 };

// Workgroup size of every kernel (four wave64s).
constexpr int kBlock = 256;

// Row-wise scan; op: 0 add, 1 min, 2 max, 3 mul (floating formats).
hipError_t launch_scan_rows(const void* in, void* out, int64_t rows, int64_t n, Fmt fmt, int op,
                            bool exclusive, hipStream_t stream);

// Device-wide exclusive (or inclusive) scan; op: 0 add, 1 min, 2 max.
size_t scan_device_tiles(int64_t n, Fmt fmt);       // descriptors needed
// n_dev (all launchers below): when not null, the live count is read from it
// on the device and clamped to [0, n]; n is then the capacity that grids and
// scratch are sized for.
// descs_clear: the caller has already zeroed the first scan_device_tiles(n,
// fmt) descriptors of `scratch` earlier on `stream`, so no fill kernel runs.
hipError_t launch_scan_device(const void* in, void* out, int64_t n, Fmt fmt, int op,
                              bool inclusive, void* scratch, hipStream_t stream,
                              const int32_t* n_dev = nullptr, bool descs_clear = false);

// Device-wide reduction into out[0]; op: 0 add, 1 min, 2 max.  n == 0 writes
// the identity.  Scratch holds one partial per workgroup of the first launch.
size_t reduce_partials(int64_t n, Fmt fmt);         // partials (8-byte slots) needed
hipError_t launch_reduce(const void* in, void* out, int64_t n, Fmt fmt, int op, void* scratch,
                         hipStream_t stream, const int32_t* n_dev = nullptr);

// Reduce-by-key (32-bit keys and values): one descriptor (four 64-bit words)
// per tile.
size_t reduce_by_key_tiles(int64_t n);
hipError_t launch_reduce_by_key(const void* keys, const void* values, void* keys_out,
                                void* values_out, int32_t* num_runs, int64_t n, Fmt kfmt,
                                Fmt vfmt, void* scratch, hipStream_t stream,
                                const int32_t* n_dev = nullptr);

// Radix sort (0 <= n <= INT32_MAX); value_bytes 0 (keys only), 4 or 8.
size_t radix_sort_scratch(int64_t n, size_t key_bytes);
hipError_t launch_radix_sort(void* keys, void* tmp_keys, void* values, void* tmp_values, int64_t n,
                             Fmt kfmt, int value_bytes, int end_bit, void* scratch,
                             hipStream_t stream, const int32_t* n_dev = nullptr);

// Stream compaction.
size_t select_tiles(int64_t n, size_t elem_bytes);
hipError_t launch_select(const void* in, const uint8_t* flags, void* out, int32_t* num_out,
                         int64_t n, size_t elem_bytes, void* scratch, hipStream_t stream,
                         const int32_t* n_dev = nullptr);

// ---- sequence operators (f32 / f16 / bf16 activations; see scan.h) ----
// Strides count elements; the last axis of every array is contiguous and the
// arrays a call writes are contiguous throughout.
struct ConvProblem {
  const void* x;
  const float* weight;              // [channels, width]
  const float* bias;                // [channels] or null
  const void* initial_state;        // [batch, width - 1, channels] or null (zeros)
  const int32_t* lengths;           // [batch] or null (all tokens exist)
  int64_t batch, length, channels, width;
  int64_t x_batch, x_token;
  bool silu;
};
hipError_t launch_conv(const ConvProblem& p, Fmt fmt, void* y, void* final_state,
                       hipStream_t stream);
size_t conv_grad_scratch(const ConvProblem& p);
hipError_t launch_conv_grad(const ConvProblem& p, Fmt fmt, const void* dy, int64_t dy_batch,
                            int64_t dy_token, const void* dfinal, void* dx, float* dweight,
                            float* dbias, void* dinitial, void* scratch, hipStream_t stream);
hipError_t launch_conv_step(const ConvProblem& p, Fmt fmt, const void* state, void* new_state,
                            void* y, hipStream_t stream);

struct ScanProblem {
  const void *x, *dt, *B, *C, *z;   // z may be null
  const float *A, *D, *dt_bias;     // [channels, states], [channels] or null (both)
  const float* initial_state;       // [batch, channels, states] or null (zeros)
  const int32_t* lengths;           // [batch] or null
  int64_t batch, length, channels, states, groups;
  int64_t x_batch, x_token, dt_batch, dt_token, z_batch, z_token;
  int64_t B_batch, B_token, B_group, C_batch, C_token, C_group;
  bool softplus;
};
// The forward keeps the state before every so many tokens for the gradient.
constexpr int kScanKeepTokens = 16;
// Chunks that a scan of few channels is split into when it is given scratch.
int64_t scan_chunks(const ScanProblem& p, int64_t* tokens);
size_t selective_scan_scratch(const ScanProblem& p);     // 0: not split
hipError_t launch_selective_scan(const ScanProblem& p, Fmt fmt, void* y, float* final_state,
                                 float* starts, void* scratch, hipStream_t stream);
struct ScanGrads {
  const void* dy;
  int64_t dy_batch, dy_token;
  const float* dfinal;              // [batch, channels, states] or null
  const float* starts;
  void *dx, *ddt, *dB, *dC, *dz;    // dz null without z
  float *dA, *dD, *ddt_bias, *dinitial;   // any of the last three may be null
};
size_t selective_scan_grad_scratch(const ScanProblem& p);
hipError_t launch_selective_scan_grad(const ScanProblem& p, Fmt fmt, const ScanGrads& g,
                                      void* scratch, hipStream_t stream);
hipError_t launch_selective_scan_step(const ScanProblem& p, Fmt fmt, const float* state,
                                      float* new_state, void* y, hipStream_t stream);

hipError_t launch_embedding(const void* weight, const void* ids, bool wide_ids, void* out,
                            int64_t tokens, int64_t rows, int64_t channels, int64_t row_stride,
                            Fmt fmt, float scale, hipStream_t stream);
size_t embedding_grad_scratch(int64_t tokens, int64_t rows, int64_t channels);
hipError_t launch_embedding_grad(const void* dout, const void* ids, bool wide_ids, void* dweight,
                                 int64_t tokens, int64_t rows, int64_t channels,
                                 int64_t row_stride, Fmt fmt, Fmt out_fmt, float scale,
                                 void* scratch, hipStream_t stream);

// The gated scan.
struct GatedProblem {
  const void *x, *forget, *input_gate, *z;   // the last two may be null
  const float* rate;                // [channels] or null (a convex average)
  const float* initial_state;       // [batch, channels] or null (zeros)
  const int32_t* lengths;           // [batch] or null
  int64_t batch, length, channels;
  int64_t x_batch, x_token, forget_batch, forget_token, input_batch, input_token, z_batch, z_token;
};
// The forward keeps the state before every so many tokens for the gradient.
constexpr int kGatedKeepTokens = 64;
size_t gated_scan_scratch(const GatedProblem& p);        // 0: none needed
hipError_t launch_gated_scan(const GatedProblem& p, Fmt fmt, void* y, float* final_state,
                             float* starts, void* scratch, hipStream_t stream);
struct GatedGrads {
  const void* dy;
  int64_t dy_batch, dy_token;
  const float* dfinal;              // [batch, channels] or null
  const float* starts;
  void *dx, *dforget, *dinput_gate, *dz;   // the last two null without their input
  float *drate, *dinitial;          // drate null without rates; dinitial may be null
};
size_t gated_scan_grad_scratch(const GatedProblem& p);
hipError_t launch_gated_scan_grad(const GatedProblem& p, Fmt fmt, const GatedGrads& g,
                                  void* scratch, hipStream_t stream);
hipError_t launch_gated_scan_step(const GatedProblem& p, Fmt fmt, const float* state,
                                  float* new_state, void* y, hipStream_t stream);

// Beam search: the `count` best of batch x [beams, vocab] continuations, and the
// states' rows moved to their new beams.
struct BeamProblem {
  const void* logits;
  const float* scores;              // [batch, beams]
  const uint8_t* finished;          // [batch, beams] or null
  int64_t batch, beams, vocab, count, end_token;
  int64_t logits_batch, logits_beam;
};
size_t beam_select_scratch(const BeamProblem& p, Fmt fmt);
hipError_t launch_beam_select(const BeamProblem& p, Fmt fmt, float* scores, int32_t* parents,
                              int32_t* tokens, void* scratch, hipStream_t stream);
hipError_t launch_beam_reorder(const void* const* states, void* const* new_states,
                               const int64_t* row_bytes, int64_t tensors, const int32_t* parents,
                               int64_t batch, int64_t beams, hipStream_t stream);

// Scratch of the look-back kernels holds only the tile descriptors, one per
// 128-byte line (kDescBytes), whose used words are zeroed at the start of
// every call by a small fill kernel (no hipMemsetAsync, so the call can sit
// in a captured graph).
// The descriptors start at the first 128-byte boundary of the caller's
// (16-byte aligned) scratch, so scratch sizes carry one line of slack.
constexpr size_t kDescBytes = 128;
inline size_t desc_scratch_bytes(size_t ntiles) {
  return ntiles == 0 ? 0 : ntiles * kDescBytes + kDescBytes;
}
inline uint64_t* desc_base(void* scratch) {
  return (uint64_t*)(((uintptr_t)scratch + kDescBytes - 1) & ~(uintptr_t)(kDescBytes - 1));
}
hipError_t launch_fill_desc(uint64_t* desc, int64_t ntiles, int words, hipStream_t stream);

// The allocation-free device scan keeps its descriptors in a static device
// array of this many bytes per GPU; noalloc_scratch() returns the current
// device's copy (hipGetSymbolAddress, once per device).
constexpr size_t kNoAllocScratchBytes = (size_t)8 << 20;
hipError_t noalloc_scratch(void** ptr);

}  // namespace sca
