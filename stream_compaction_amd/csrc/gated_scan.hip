// Gated scan: forward and single-token step.
//
//   h[t] = a[t] h[t-1] + w[t] v[t] x[t],  y = h silu(z)      (gates: gated.hpp)
//
// A thread per channel walks its sequence's tokens in order.
#include "gated.hpp"

namespace sca {

constexpr int64_t kMaxGroups = 1ll << 21;    // workgroups per launch

template <class F, bool RATE>
__device__ __forceinline__ float gated_token(float h, typename F::S x, typename F::S f,
                                             const typename F::S* ig, float nr) {
  const Gate g = gate<RATE>(widen<F>(f), nr);
  float u = g.w * widen<F>(x);
  if (ig != nullptr) u *= sigmoid(widen<F>(*ig));
  return __builtin_fmaf(g.a, h, u);
}

template <class F, bool RATE>
__global__ __launch_bounds__(64) void gated_scan_kernel(GatedProblem p, void* yv,
                                                        float* final_state, float* starts,
                                                        int64_t b0) {
  using S = typename F::S;
  int64_t part;
  const int64_t parts = (p.channels + 63) / 64;
  const int64_t b = b0 + divide((int64_t)blockIdx.x, parts, &part), c = part * 64 + threadIdx.x;
  if (c >= p.channels) return;
  const float nr = RATE ? rate_log2(p.rate[c]) : 0.0f;
  const int64_t n = p.lengths == nullptr ? p.length : live_count(p.length, p.lengths + b);
  float h = p.initial_state == nullptr ? 0.0f : p.initial_state[b * p.channels + c];
  const int64_t blocks = (p.length + kGatedKeepTokens - 1) / kGatedKeepTokens;
  S* y = (S*)yv + b * p.length * p.channels + c;
  for (int64_t t = 0; t < p.length; ++t) {
    if (starts != nullptr && t % kGatedKeepTokens == 0)
      starts[(b * blocks + t / kGatedKeepTokens) * p.channels + c] = h;
    float out = 0.0f;
    if (t < n) {
      const S* ig = p.input_gate == nullptr
                        ? nullptr
                        : (const S*)p.input_gate + b * p.input_batch + t * p.input_token + c;
      h = gated_token<F, RATE>(h, ((const S*)p.x)[b * p.x_batch + t * p.x_token + c],
                               ((const S*)p.forget)[b * p.forget_batch + t * p.forget_token + c],
                               ig, nr);
      out = p.z == nullptr ? h
                           : h * silu(widen<F>(((const S*)p.z)[b * p.z_batch + t * p.z_token + c]));
    }
    y[t * p.channels] = narrow<F>(out);
  }
  if (final_state != nullptr) final_state[b * p.channels + c] = h;
}

size_t gated_scan_scratch(const GatedProblem&) { return 0; }

template <class F>
static hipError_t launch_gated_f(const GatedProblem& p, void* y, float* final_state, float* starts,
                                 hipStream_t stream) {
  const int64_t parts = (p.channels + 63) / 64;
  const int64_t step = kMaxGroups / parts;
  for (int64_t b0 = 0; b0 < p.batch; b0 += step) {
    const int64_t nb = p.batch - b0 < step ? p.batch - b0 : step;
    const dim3 grid((unsigned)(nb * parts));
    if (p.rate != nullptr)
      gated_scan_kernel<F, true><<<grid, dim3(64), 0, stream>>>(p, y, final_state, starts, b0);
    else
      gated_scan_kernel<F, false><<<grid, dim3(64), 0, stream>>>(p, y, final_state, starts, b0);
  }
  return hipGetLastError();
}

hipError_t launch_gated_scan(const GatedProblem& p, Fmt fmt, void* y, float* final_state,
                             float* starts, void*, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_gated_f<FmtF32>(p, y, final_state, starts, stream);
    case Fmt::F16: return launch_gated_f<FmtF16>(p, y, final_state, starts, stream);
    case Fmt::BF16: return launch_gated_f<FmtBF16>(p, y, final_state, starts, stream);
    default: return hipErrorInvalidValue;
  }
}

// One token: a thread per channel.
template <class F, bool RATE>
__global__ __launch_bounds__(256) void gated_scan_step_kernel(GatedProblem p, const float* state,
                                                              float* new_state, void* yv) {
  using S = typename F::S;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.batch * p.channels) return;
  int64_t c;
  const int64_t b = divide(i, p.channels, &c);
  const float nr = RATE ? rate_log2(p.rate[c]) : 0.0f;
  const S* ig =
      p.input_gate == nullptr ? nullptr : (const S*)p.input_gate + b * p.input_batch + c;
  const float h = gated_token<F, RATE>(state[i], ((const S*)p.x)[b * p.x_batch + c],
                                       ((const S*)p.forget)[b * p.forget_batch + c], ig, nr);
  new_state[i] = h;
  ((S*)yv)[i] = narrow<F>(
      p.z == nullptr ? h : h * silu(widen<F>(((const S*)p.z)[b * p.z_batch + c])));
}

template <class F>
static hipError_t launch_step_f(const GatedProblem& p, const float* state, float* new_state,
                                void* y, hipStream_t stream) {
  const dim3 grid((unsigned)((p.batch * p.channels + 255) / 256));
  if (p.rate != nullptr)
    gated_scan_step_kernel<F, true><<<grid, dim3(256), 0, stream>>>(p, state, new_state, y);
  else
    gated_scan_step_kernel<F, false><<<grid, dim3(256), 0, stream>>>(p, state, new_state, y);
  return hipGetLastError();
}

hipError_t launch_gated_scan_step(const GatedProblem& p, Fmt fmt, const float* state,
                                  float* new_state, void* y, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_step_f<FmtF32>(p, state, new_state, y, stream);
    case Fmt::F16: return launch_step_f<FmtF16>(p, state, new_state, y, stream);
    case Fmt::BF16: return launch_step_f<FmtBF16>(p, state, new_state, y, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sca
