// Gradient of the gated scan.
//
// With q = dy silu(z) the gradient of h[t] is g[t] = q[t] + a[t+1] g[t+1], and with
// s, v the two sigmoids:
//   dx = g w v,   dinput_gate = g w x v (1 - v),   dz = dy h silu'(z),
//   without rates  dforget = g (h[t-1] - v x) s (1 - s),
//   with a rate    E = p dL/dp = g (v x a^2 p / w - p a h[t-1]),
//                  dforget = E (1 - s),   drate = (sum of E over tokens) / rate,
// as p = rate s enters through log p alone.  p / w tends to 0 with p.
//
// A thread per channel goes through the blocks of 64 tokens from the last one on:
// each block's states are found again from its start, which the forward kept.
#include "gated.hpp"

namespace sca {

template <class F, bool RATE>
__global__ __launch_bounds__(64) void gated_scan_grad_kernel(GatedProblem p, GatedGrads g,
                                                             float* partial, int64_t b0) {
  using S = typename F::S;
  constexpr int K = kGatedKeepTokens;
  int64_t part;
  const int64_t parts = (p.channels + 63) / 64;
  const int64_t b = b0 + divide((int64_t)blockIdx.x, parts, &part), c = part * 64 + threadIdx.x;
  if (c >= p.channels) return;
  const float nr = RATE ? rate_log2(p.rate[c]) : 0.0f;
  const int64_t n = p.lengths == nullptr ? p.length : live_count(p.length, p.lengths + b);
  const int64_t blocks = (p.length + K - 1) / K;
  const S* x = (const S*)p.x + b * p.x_batch + c;
  const S* f = (const S*)p.forget + b * p.forget_batch + c;
  const S* ig = (const S*)p.input_gate + b * p.input_batch + c;
  const S* z = (const S*)p.z + b * p.z_batch + c;
  const S* dy = (const S*)g.dy + b * g.dy_batch + c;
  const int64_t row = b * p.length * p.channels + c;
  float carry = g.dfinal == nullptr ? 0.0f : g.dfinal[b * p.channels + c], total = 0.0f;
  for (int64_t t = n; t < p.length; ++t) {
    ((S*)g.dx)[row + t * p.channels] = ((S*)g.dforget)[row + t * p.channels] = narrow<F>(0.0f);
    if (p.input_gate != nullptr) ((S*)g.dinput_gate)[row + t * p.channels] = narrow<F>(0.0f);
    if (p.z != nullptr) ((S*)g.dz)[row + t * p.channels] = narrow<F>(0.0f);
  }
  for (int64_t blk = (n + K - 1) / K - 1; blk >= 0; --blk) {
    const int64_t t0 = blk * K;
    const int count = (int)(n - t0 < K ? n - t0 : K);
    float hs[K];
    float h = g.starts[(b * blocks + blk) * p.channels + c];
    for (int k = 0; k < count; ++k) {
      const int64_t t = t0 + k;
      hs[k] = h;
      const Gate gt = gate<RATE>(widen<F>(f[t * p.forget_token]), nr);
      const float v = p.input_gate == nullptr ? 1.0f : sigmoid(widen<F>(ig[t * p.input_token]));
      h = __builtin_fmaf(gt.a, h, gt.w * v * widen<F>(x[t * p.x_token]));
    }
    for (int k = count - 1; k >= 0; --k) {
      const int64_t t = t0 + k, at = row + t * p.channels;
      const float fv = widen<F>(f[t * p.forget_token]), xv = widen<F>(x[t * p.x_token]);
      const Gate gt = gate<RATE>(fv, nr);
      const Sides s = sides(fv);
      const float d = widen<F>(dy[t * g.dy_token]);
      float q = d;
      if (p.z != nullptr) {
        const float zv = widen<F>(z[t * p.z_token]);
        q = d * silu(zv);
        ((S*)g.dz)[at] = narrow<F>(d * h * silu_slope(zv));
      }
      Sides v = {1.0f, 0.0f};
      if (p.input_gate != nullptr) v = sides(widen<F>(ig[t * p.input_token]));
      const float grad = q + carry, dx = grad * gt.w * v.up;
      ((S*)g.dx)[at] = narrow<F>(dx);
      if (p.input_gate != nullptr) ((S*)g.dinput_gate)[at] = narrow<F>(dx * xv * v.down);
      if constexpr (RATE) {
        const float P = at_most(gt.log_a * -kLn2, 128.0f);   // exp(-128) is 0 in float32
        const float pw = gt.w > 0.0f ? P / gt.w : 0.0f;
        const float E = grad * (v.up * xv * gt.a * gt.a * pw - P * gt.a * hs[k]);
        ((S*)g.dforget)[at] = narrow<F>(E * s.down);
        total += E;
      } else {
        ((S*)g.dforget)[at] = narrow<F>(grad * (hs[k] - v.up * xv) * s.up * s.down);
      }
      carry = gt.a * grad;
      h = hs[k];
    }
  }
  if (g.dinitial != nullptr) g.dinitial[b * p.channels + c] = carry;
  if constexpr (RATE) partial[b * p.channels + c] = total;
}

__global__ __launch_bounds__(64) void gated_rate_kernel(const float* partial, const float* rate,
                                                        float* drate, int64_t rows,
                                                        int64_t channels) {
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (c >= channels) return;
  float sum = 0.0f;
  for (int64_t i = 0; i < rows; ++i) sum += partial[i * channels + c];
  drate[c] = rate[c] <= 0.0f ? 0.0f : sum / rate[c];
}

size_t gated_scan_grad_scratch(const GatedProblem& p) {
  return p.rate == nullptr ? 0 : (size_t)(p.batch * p.channels) * 4;
}

template <class F>
static hipError_t launch_grad_f(const GatedProblem& p, const GatedGrads& g, float* partial,
                                hipStream_t stream) {
  const int64_t parts = (p.channels + 63) / 64, step = (1ll << 21) / parts;
  for (int64_t b0 = 0; b0 < p.batch; b0 += step) {
    const int64_t nb = p.batch - b0 < step ? p.batch - b0 : step;
    const dim3 grid((unsigned)(nb * parts));
    if (p.rate != nullptr)
      gated_scan_grad_kernel<F, true><<<grid, dim3(64), 0, stream>>>(p, g, partial, b0);
    else
      gated_scan_grad_kernel<F, false><<<grid, dim3(64), 0, stream>>>(p, g, partial, b0);
  }
  if (p.rate != nullptr)
    gated_rate_kernel<<<dim3((unsigned)parts), dim3(64), 0, stream>>>(partial, p.rate, g.drate,
                                                                      p.batch, p.channels);
  return hipGetLastError();
}

hipError_t launch_gated_scan_grad(const GatedProblem& p, Fmt fmt, const GatedGrads& g,
                                  void* scratch, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_grad_f<FmtF32>(p, g, (float*)scratch, stream);
    case Fmt::F16: return launch_grad_f<FmtF16>(p, g, (float*)scratch, stream);
    case Fmt::BF16: return launch_grad_f<FmtBF16>(p, g, (float*)scratch, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sca
