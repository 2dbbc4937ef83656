// Short causal convolution along time, one filter per channel:
//   pre[t] = bias + sum_{k < W} w[k] x[t - W + 1 + k],   y = silu(pre) or pre,
// its gradient, and its step for one token.  Tokens before the first come from
// an initial state of W - 1 tokens (or are zero); tokens at and past a
// sequence's length do not exist (their outputs are zero).
//
// Forward and step are bound by memory: 2 W operations and a silu per element
// against 4 bytes.  A lane owns E neighbouring channels (one load of up to 16
// bytes per token) and walks a run of tokens with the last W inputs in
// registers, so each input is read once but for the W - 1 tokens before a run.
// Measured, bf16, W = 4: forward 4 x 4096 x 4096 with half of it padding (202 MB)
// 47.5 us, 4.2 TB/s, with inputs that no cache holds and 34 us with inputs in the
// last-level cache; step 128 x 4096 (8.5 MB) 4.6 us, most of it latency.  Rows off
// alignment go one channel per lane: 4 x 4096 x 2047 40 us against 29 for 2048.
#include "sequence.hpp"

namespace sca {

namespace {

__device__ __forceinline__ int64_t conv_length(const ConvProblem& p, int64_t b) {
  if (p.lengths == nullptr) return p.length;
  const int64_t v = p.lengths[b];
  return v < 0 ? 0 : (v > p.length ? p.length : v);
}

// The filters of E channels, channel c's tap k in w[k][c].  E W consecutive
// floats, 16 bytes at a time where the arrays are aligned and the lane's channels
// all exist: one by one they cost more than a run's input.
template <int E, int W>
__device__ __forceinline__ void load_filters(const ConvProblem& p, int64_t ch, float (&w)[W][E],
                                             float (&bias)[E]) {
  const int64_t n = p.channels - ch;
  const bool wide = E > 1 && p.channels % E == 0 &&
                    (((uintptr_t)p.weight | (uintptr_t)p.bias) % 16 == 0);
  typedef float vec4 __attribute__((ext_vector_type(4)));
  if (wide) {
#pragma unroll
    for (int j = 0; j < E * W; j += 4) {
      const vec4 v = *gptr<const vec4>((uintptr_t)(p.weight + ch * W + j));
#pragma unroll
      for (int i = 0; i < 4; ++i) w[(j + i) % W][(j + i) / W] = v[i];
    }
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      vec4 v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (p.bias != nullptr) v = *gptr<const vec4>((uintptr_t)(p.bias + ch + j));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < E) bias[j + i] = v[i];
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < E; ++c) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][c] = c < n ? p.weight[(ch + c) * W + k] : 0.0f;
    bias[c] = c < n && p.bias != nullptr ? p.bias[ch + c] : 0.0f;
  }
}

// Input token t of sequence b: the initial state before 0, zero past `len`.
template <class F, int E, int W, bool ALIGNED = true>
__device__ __forceinline__ typename RowIO<F, E>::Raw conv_input(const ConvProblem& p, int64_t b,
                                                               int64_t t, int64_t len, int64_t ch) {
  using S = typename F::S;
  const S* src = nullptr;
  if (t >= 0) {
    if (t < len) src = (const S*)p.x + b * p.x_batch + t * p.x_token + ch;
  } else if (p.initial_state != nullptr) {
    src = (const S*)p.initial_state + (b * (W - 1) + t + W - 1) * p.channels + ch;
  }
  if (src == nullptr) return typename RowIO<F, E>::Raw{};
  return RowIO<F, E>::template get<ALIGNED>(src, p.channels - ch);
}

}  // namespace

constexpr int kConvAhead = 4;     // token rows loaded together

template <class F, int E, int W, bool PAST>
__global__ __launch_bounds__(256) void causal_conv_kernel(ConvProblem p, void* yv,
                                                         void* final_state, int run_tokens) {
  using S = typename F::S;
  using IO = RowIO<F, E>;
  const int64_t vecs = (p.channels + E - 1) / E;
  const int64_t runs = p.length > 0 ? (p.length + run_tokens - 1) / run_tokens : 1;
  const int64_t total = p.batch * runs * vecs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    int64_t ch, run;
    const int64_t b = divide(divide(i, vecs, &ch), runs, &run);
    ch *= E;
    const int64_t len = conv_length(p, b);
    const int64_t t0 = run * run_tokens;
    const int64_t end = t0 + run_tokens < p.length ? t0 + run_tokens : p.length;
    const int64_t last = end < len ? end : len;        // tokens of the run that exist
    const S* x = (const S*)p.x + b * p.x_batch + ch;
    S* y = (S*)yv + b * p.length * p.channels + ch;
    int64_t t = t0;
    if (t < last) {
      auto row = [&](int64_t at) {
        return at < last ? IO::load(x + at * p.x_token) : typename IO::Raw{};
      };
      typename IO::Raw next[kConvAhead];
#pragma unroll
      for (int j = 0; j < kConvAhead; ++j) next[j] = row(t + j);
      float w[W][E], bias[E], win[W][E];
      load_filters<E, W>(p, ch, w, bias);
#pragma unroll
      for (int k = 0; k + 1 < W; ++k)
        IO::unpack(conv_input<F, E, W>(p, b, t0 - W + 1 + k, len, ch), win[k + 1]);
      for (; t < last; t += kConvAhead) {
        typename IO::Raw raw[kConvAhead];
#pragma unroll
        for (int j = 0; j < kConvAhead; ++j) raw[j] = next[j];
#pragma unroll
        for (int j = 0; j < kConvAhead; ++j) next[j] = row(t + kConvAhead + j);
#pragma unroll
        for (int j = 0; j < kConvAhead; ++j) {
#pragma unroll
          for (int k = 0; k + 1 < W; ++k)
#pragma unroll
            for (int c = 0; c < E; ++c) win[k][c] = win[k + 1][c];
          IO::unpack(raw[j], win[W - 1]);
          float out[E];
#pragma unroll
          for (int c = 0; c < E; ++c) {
            float a = bias[c];
#pragma unroll
            for (int k = 0; k < W; ++k) a = __builtin_fmaf(w[k][c], win[k][c], a);
            out[c] = p.silu ? silu(a) : a;
          }
          if (t + j < last)
            IO::template store_past<PAST>(y + (t + j) * p.channels, IO::pack(out));
        }
      }
      t = last;
    }
    for (; t < end; ++t)
      IO::template store_past<PAST>(y + t * p.channels, typename IO::Raw{});
    if (run == 0 && final_state != nullptr) {
      S* fs = (S*)final_state + b * (W - 1) * p.channels + ch;
#pragma unroll
      for (int k = 0; k + 1 < W; ++k)
        IO::store(fs + k * p.channels,
                  conv_input<F, E, W>(p, b, len - W + 1 + k, len, ch));
    }
  }
}

// Gradient.  With g = dy * slope(pre), dx[t] = sum_k w[k] g[t + W - 1 - k]: a
// lane recomputes g for its run and the W - 1 tokens after it.  Filter sums
// over a run stay in registers; the four waves of a workgroup (four runs of
// the same channels) add theirs in LDS, and a second kernel adds the
// workgroups' sums in a fixed order, so results are the same every time.  Some
// 40 instructions per element keep the vector units 73% busy beside 101 MB: 4 x
// 2048 x 2048 takes 32 us and 4 us for the filter sums.  Four channels per lane:
// eight hold too many values in registers for four waves a SIMD, two read rows in
// 4-byte pieces (37 us against 35).
constexpr int kConvGradWaves = 4;

// Gradients with respect to the final state reach line token t (x for t >= 0,
// the initial state for t < 0) when t is among the last W - 1 before len.
template <class F, int E, int W, bool ALIGNED>
__device__ __forceinline__ void add_final(const ConvProblem& p, const void* dfinal, int64_t b,
                                          int64_t t, int64_t len, int64_t ch, float (&d)[E]) {
  using S = typename F::S;
  const int64_t j = t - len + W - 1;
  if (dfinal == nullptr || j < 0 || j >= W - 1) return;
  float v[E];
  RowIO<F, E>::unpack(
      RowIO<F, E>::template get<ALIGNED>((const S*)dfinal + (b * (W - 1) + j) * p.channels + ch,
                                         p.channels - ch),
      v);
#pragma unroll
  for (int c = 0; c < E; ++c) d[c] += v[c];
}

template <class F, int E, int W, bool ALIGNED>
__global__ __launch_bounds__(64 * kConvGradWaves) void causal_conv_grad_kernel(
    ConvProblem p, const void* dyv, int64_t dy_batch, int64_t dy_token, const void* dfinal,
    void* dxv, void* dinitial, float* part, int run_tokens) {
  using S = typename F::S;
  using IO = RowIO<F, E>;
  constexpr int M = W + 1;                          // sums per channel
  __shared__ float s_sum[kConvGradWaves][E * M][64];
  const int lane = lane_id(), wave = wave_id();
  const int64_t vecs = (p.channels + E - 1) / E, cols = (vecs + 63) / 64;
  const int64_t runs = p.length > 0 ? (p.length + run_tokens - 1) / run_tokens : 1;
  const int64_t total = p.batch * runs;             // runs of all sequences
  const int64_t col = blockIdx.x % cols, set = blockIdx.x / cols;
  const int64_t sets = gridDim.x / cols;
  const int64_t ch = (col * 64 + lane) * E;
  const int64_t n = p.channels - ch;
  const bool live = n > 0;
  float w[W][E], bias[E], dw[W][E] = {}, db[E] = {};
  if (live) load_filters<E, W>(p, ch, w, bias);
  for (int64_t r = set * kConvGradWaves + wave; r < total; r += sets * kConvGradWaves) {
    if (!live) break;
    int64_t t0;
    const int64_t b = divide(r, runs, &t0);
    t0 *= run_tokens;
    const int64_t len = conv_length(p, b);
    const int64_t end = t0 + run_tokens < p.length ? t0 + run_tokens : p.length;
    const S* dy = (const S*)dyv + b * dy_batch + ch;
    S* dx = (S*)dxv + b * p.length * p.channels + ch;
    float win[W][E], g[W][E] = {};                  // inputs and gradients, newest last
#pragma unroll
    for (int k = 0; k + 1 < W; ++k)
      IO::unpack(conv_input<F, E, W, ALIGNED>(p, b, t0 - W + 1 + k, len, ch), win[k + 1]);
    const int steps = run_tokens + W - 1;
    for (int s0 = 0; s0 < steps; s0 += kConvAhead) {
      typename IO::Raw rx[kConvAhead], rdy[kConvAhead];
#pragma unroll
      for (int j = 0; j < kConvAhead; ++j) {
        const int64_t t = t0 + s0 + j;
        rx[j] = conv_input<F, E, W, ALIGNED>(p, b, t, len, ch);
        rdy[j] = t < len ? IO::template get<ALIGNED>(dy + t * dy_token, n) : typename IO::Raw{};
      }
#pragma unroll
      for (int j = 0; j < kConvAhead; ++j) {
        const int64_t t = t0 + s0 + j;
#pragma unroll
        for (int k = 0; k + 1 < W; ++k)
#pragma unroll
          for (int c = 0; c < E; ++c) {
            win[k][c] = win[k + 1][c];
            g[k][c] = g[k + 1][c];
          }
        IO::unpack(rx[j], win[W - 1]);
        IO::unpack(rdy[j], g[W - 1]);
        if (p.silu) {
#pragma unroll
          for (int c = 0; c < E; ++c) {
            float a = bias[c];
#pragma unroll
            for (int k = 0; k < W; ++k) a = __builtin_fmaf(w[k][c], win[k][c], a);
            g[W - 1][c] = t < len ? g[W - 1][c] * silu_slope(a) : 0.0f;
          }
        }
        if (s0 + j < run_tokens) {                 // the run's own tokens
#pragma unroll
          for (int c = 0; c < E; ++c) {
            db[c] += g[W - 1][c];
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][c] = __builtin_fmaf(g[W - 1][c], win[k][c], dw[k][c]);
          }
        }
        // line token t - W + 1 now has all its gradients
        const int64_t u = t - W + 1;
        if (u < end && (u >= t0 || (t0 == 0 && dinitial != nullptr))) {
          float d[E];
#pragma unroll
          for (int c = 0; c < E; ++c) {
            d[c] = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) d[c] = __builtin_fmaf(w[k][c], g[W - 1 - k][c], d[c]);
          }
          add_final<F, E, W, ALIGNED>(p, dfinal, b, u, len, ch, d);
          S* to = u >= 0 ? dx + u * p.channels
                         : (S*)dinitial + (b * (W - 1) + u + W - 1) * p.channels + ch;
          if (u < len) {
            IO::template put<ALIGNED>(to, IO::pack(d), n);
          } else {
            IO::template put<ALIGNED>(to, typename IO::Raw{}, n);
          }
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < E; ++c) {
#pragma unroll
    for (int k = 0; k < W; ++k) s_sum[wave][c * M + k][lane] = dw[k][c];
    s_sum[wave][c * M + W][lane] = db[c];
  }
  __syncthreads();
  // channel-major sums of this workgroup: [set][channel][M]
  for (int i = threadIdx.x; i < 64 * E * M; i += 64 * kConvGradWaves) {
    const int l = i / (E * M), m = i % (E * M);
    const int64_t c = (col * 64 + l) * E + m / M;
    if (c >= p.channels) continue;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kConvGradWaves; ++q) v += s_sum[q][m][l];
    part[set * p.channels * M + c * M + m % M] = v;
  }
}

// dweight and dbias from the workgroups' sums, in a fixed order: 64 values per
// workgroup, 16 strided partial sums each, whose loads travel four at a time.
constexpr int kSumStrands = 16;
__global__ __launch_bounds__(64 * kSumStrands) void conv_filter_sum_kernel(
    const float* part, int64_t sets, int64_t count, int M, float* dweight, float* dbias) {
  __shared__ float s[kSumStrands][64];
  const int l = threadIdx.x % 64, q = threadIdx.x / 64;
  const int64_t i = (int64_t)blockIdx.x * 64 + l;
  float v = 0.0f;
  if (i < count) {
#pragma unroll 4
    for (int64_t k = q; k < sets; k += kSumStrands) v += part[k * count + i];
  }
  s[q][l] = v;
  __syncthreads();
  if (q != 0 || i >= count) return;
#pragma unroll
  for (int k = 1; k < kSumStrands; ++k) v += s[k][l];
  const int64_t c = i / M;
  const int m = (int)(i % M);
  if (m + 1 < M) {
    dweight[c * (M - 1) + m] = v;
  } else if (dbias != nullptr) {
    dbias[c] = v;
  }
}

// One token: the state's W - 1 rows and the new input, each read once.
template <class F, int E, int W>
__global__ __launch_bounds__(256) void causal_conv_step_kernel(ConvProblem p, const void* state,
                                                              void* new_state, void* yv) {
  using S = typename F::S;
  using IO = RowIO<F, E>;
  const int64_t vecs = (p.channels + E - 1) / E;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.batch * vecs) return;
  int64_t ch;
  const int64_t b = divide(i, vecs, &ch);
  ch *= E;
  float w[W][E], bias[E], a[E];
  typename IO::Raw row[W];
#pragma unroll
  for (int k = 0; k + 1 < W; ++k)
    row[k] = IO::load((const S*)state + (b * (W - 1) + k) * p.channels + ch);
  row[W - 1] = IO::load((const S*)p.x + b * p.x_batch + ch);
  load_filters<E, W>(p, ch, w, bias);
#pragma unroll
  for (int c = 0; c < E; ++c) a[c] = bias[c];
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float v[E];
    IO::unpack(row[k], v);
#pragma unroll
    for (int c = 0; c < E; ++c) a[c] = __builtin_fmaf(w[k][c], v[c], a[c]);
  }
  if (p.silu) {
#pragma unroll
    for (int c = 0; c < E; ++c) a[c] = silu(a[c]);
  }
  IO::store((S*)yv + b * p.channels + ch, IO::pack(a));
#pragma unroll
  for (int k = 0; k + 1 < W; ++k)
    IO::store((S*)new_state + (b * (W - 1) + k) * p.channels + ch, row[k + 1]);
}

// Vectors of E channels can be used when every row starts on E elements.
template <class F> static bool rows_aligned(int E, int64_t channels, const void* a, int64_t s0 = 0,
                                            int64_t s1 = 0) {
  const int64_t bytes = (int64_t)E * (int64_t)sizeof(typename F::S);
  return a == nullptr || ((uintptr_t)a % bytes == 0 && channels % E == 0 && s0 % E == 0 &&
                          s1 % E == 0);
}

constexpr int64_t kGridMost = 1 << 20;              // workgroups; kernels loop beyond it

// Tokens a lane walks: a longer run reads fewer rows and filters twice, as long
// as it leaves enough workgroups.
static int conv_run(const ConvProblem& p, int E, int64_t most, int64_t workgroups) {
  const int64_t lanes = p.batch * ((p.channels + E - 1) / E);
  int run = (int)most;
  while (run > 4 && lanes * ((p.length + run - 1) / run) < workgroups * 256) run /= 2;
  return run;
}

template <class F, int E, int W>
static void fwd_go(const ConvProblem& p, void* y, void* final_state, hipStream_t stream) {
  const int run = conv_run(p, E, 32, 1024);
  const int64_t runs = p.length > 0 ? (p.length + run - 1) / run : 1;
  const int64_t blocks = (p.batch * runs * ((p.channels + E - 1) / E) + 255) / 256;
  const dim3 grid((unsigned)(blocks < kGridMost ? blocks : kGridMost));
  if constexpr (E > 1) {
    if (past_caches(p.batch * p.length * p.channels * (int64_t)sizeof(typename F::S))) {
      causal_conv_kernel<F, E, W, true><<<grid, dim3(256), 0, stream>>>(p, y, final_state, run);
      return;
    }
  }
  causal_conv_kernel<F, E, W, false><<<grid, dim3(256), 0, stream>>>(p, y, final_state, run);
}
template <class F, int W>
static hipError_t fwd_w(const ConvProblem& p, void* y, void* fs, hipStream_t stream) {
  constexpr int E = kVecElems<F>;
  if (rows_aligned<F>(E, p.channels, p.x, p.x_batch, p.x_token) && rows_aligned<F>(E, p.channels, y) &&
      rows_aligned<F>(E, p.channels, fs) && rows_aligned<F>(E, p.channels, p.initial_state)) {
    fwd_go<F, E, W>(p, y, fs, stream);
  } else {
    fwd_go<F, 1, W>(p, y, fs, stream);
  }
  return hipGetLastError();
}

constexpr int kConvGradE = 4;   // channels per lane
static int grad_run(const ConvProblem& p) { return conv_run(p, kConvGradE, 32, 1024); }
static int64_t grad_sets(const ConvProblem& p) {
  const int run = grad_run(p);
  const int64_t per = p.length > 0 ? (p.length + run - 1) / run : 1;
  const int64_t runs = per * p.batch;
  const int64_t sets = (runs + kConvGradWaves - 1) / kConvGradWaves;
  // at most 1024 partial sums per channel, and a grid of at most 2^22 workgroups
  const int64_t cols = (p.channels + 63) / 64, most = (1ll << 22) / cols;
  const int64_t cap = most < 1024 ? most : 1024;
  return sets < cap ? sets : cap;
}
size_t conv_grad_scratch(const ConvProblem& p) {
  return (size_t)(grad_sets(p) * p.channels * (p.width + 1)) * 4;
}

template <class F, int W>
static hipError_t grad_w(const ConvProblem& p, const void* dy, int64_t dy_batch, int64_t dy_token,
                         const void* dfinal, void* dx, float* dweight, float* dbias,
                         void* dinitial, void* scratch, hipStream_t stream) {
  constexpr int E = kConvGradE;
  const int run = grad_run(p);
  const int64_t sets = grad_sets(p);
  float* part = (float*)scratch;
  auto cols = [&](int e) { return ((p.channels + e - 1) / e + 63) / 64; };
  if (sets == 0) {
    // no sequence: the filter sums below are zero
  } else if (rows_aligned<F>(E, p.channels, p.x, p.x_batch, p.x_token) &&
      rows_aligned<F>(E, p.channels, dy, dy_batch, dy_token) &&
      rows_aligned<F>(E, p.channels, dx) && rows_aligned<F>(E, p.channels, dinitial) &&
      rows_aligned<F>(E, p.channels, dfinal) && rows_aligned<F>(E, p.channels, p.initial_state)) {
    causal_conv_grad_kernel<F, E, W, true><<<dim3((unsigned)(sets * cols(E))), dim3(64 * kConvGradWaves),
                                       0, stream>>>(p, dy, dy_batch, dy_token, dfinal, dx, dinitial,
                                                    part, run);
  } else {
    causal_conv_grad_kernel<F, E, W, false><<<dim3((unsigned)(sets * cols(E))), dim3(64 * kConvGradWaves),
                                       0, stream>>>(p, dy, dy_batch, dy_token, dfinal, dx, dinitial,
                                                    part, run);
  }
  const int64_t count = p.channels * (W + 1);
  conv_filter_sum_kernel<<<dim3((unsigned)((count + 63) / 64)), dim3(64 * kSumStrands), 0, stream>>>(
      part, sets, count, W + 1, dweight, dbias);
  return hipGetLastError();
}

template <class F, int W>
static hipError_t step_w(const ConvProblem& p, const void* state, void* new_state, void* y,
                         hipStream_t stream) {
  constexpr int E = kVecElems<F>;
  if (rows_aligned<F>(E, p.channels, p.x, p.x_batch) && rows_aligned<F>(E, p.channels, y) &&
      rows_aligned<F>(E, p.channels, state) && rows_aligned<F>(E, p.channels, new_state)) {
    const int64_t blocks = (p.batch * (p.channels / E) + 255) / 256;
    causal_conv_step_kernel<F, E, W><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(
        p, state, new_state, y);
  } else {
    const int64_t blocks = (p.batch * p.channels + 255) / 256;
    causal_conv_step_kernel<F, 1, W><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(
        p, state, new_state, y);
  }
  return hipGetLastError();
}

// Calls fn with the format and the filter width as constants.
template <class Fn> static hipError_t by_width(int64_t width, Fn&& fn) {
  switch (width) {
    case 1: return fn(std::integral_constant<int, 1>{});
    case 2: return fn(std::integral_constant<int, 2>{});
    case 3: return fn(std::integral_constant<int, 3>{});
    case 4: return fn(std::integral_constant<int, 4>{});
    case 5: return fn(std::integral_constant<int, 5>{});
    case 6: return fn(std::integral_constant<int, 6>{});
    case 7: return fn(std::integral_constant<int, 7>{});
    case 8: return fn(std::integral_constant<int, 8>{});
    default: return hipErrorInvalidValue;
  }
}
template <class Fn> static hipError_t by_format(Fmt fmt, Fn&& fn) {
  switch (fmt) {
    case Fmt::F32: return fn(FmtF32{});
    case Fmt::F16: return fn(FmtF16{});
    case Fmt::BF16: return fn(FmtBF16{});
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_conv(const ConvProblem& p, Fmt fmt, void* y, void* final_state,
                       hipStream_t stream) {
  return by_format(fmt, [&](auto f) {
    return by_width(p.width, [&](auto w) {
      return fwd_w<decltype(f), decltype(w)::value>(p, y, final_state, stream);
    });
  });
}

hipError_t launch_conv_grad(const ConvProblem& p, Fmt fmt, const void* dy, int64_t dy_batch,
                            int64_t dy_token, const void* dfinal, void* dx, float* dweight,
                            float* dbias, void* dinitial, void* scratch, hipStream_t stream) {
  return by_format(fmt, [&](auto f) {
    return by_width(p.width, [&](auto w) {
      return grad_w<decltype(f), decltype(w)::value>(p, dy, dy_batch, dy_token, dfinal, dx, dweight,
                                                     dbias, dinitial, scratch, stream);
    });
  });
}

hipError_t launch_conv_step(const ConvProblem& p, Fmt fmt, const void* state, void* new_state,
                            void* y, hipStream_t stream) {
  return by_format(fmt, [&](auto f) {
    return by_width(p.width, [&](auto w) {
      return step_w<decltype(f), decltype(w)::value>(p, state, new_state, y, stream);
    });
  });
}

}  // namespace sca
