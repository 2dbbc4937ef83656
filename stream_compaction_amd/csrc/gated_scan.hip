// Gated scan: forward and single-token step.
//
//   h[t] = a[t] h[t-1] + w[t] v[t] x[t],  y = h silu(z)      (gates: gated.hpp)
//
// One pass: a workgroup reads its tile of 128 tokens by 128 channels once, finds the
// state that enters it from the tiles before (gated_tile.hpp), and walks its tokens.
//
// 8192 tokens x 4096 channels, bfloat16, rate and input gate: 67 us, 268 MB at 4.0 TB/s
// (the same loads and stores without arithmetic 49 us; vector units 60% busy); 4 x 4096 x
// 4096 float16 with output gate, half of it padding: 71 us, 335 MB at 4.7 TB/s; 45 x 768:
// 7.5 us.  Runs of 16 tokens by 8 waves measured best: 8 tokens 85 us for the first, 4
// waves 82, 16 waves 76.
#include "gated_tile.hpp"

namespace sca {

constexpr int kFwdTokens = 16;                              // of a wave
constexpr int kFwdTile = kFwdTokens * kTileWaves;           // of a workgroup
static_assert(kGatedKeepTokens % kFwdTokens == 0, "a kept state is a wave's first");

template <class F, bool RATE, bool IG, bool Z, Rows2 ROWS>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(4, 4)))
void gated_scan_kernel(GatedProblem p, void* yv, float* final_state, float* starts, uint64_t* scratch,
                       Tiles tiles) {
  using S = typename F::S;
  using PIO = PairIO<F, ROWS>;
  constexpr bool ODD = PIO::ODD;
  using Raw = typename PIO::Raw;
  constexpr int T = kFwdTokens;
  constexpr int eb = sizeof(S);
  // four inputs at once have no room in registers in float32, nor as single channels
  constexpr bool kLateZ = sizeof(S) == 4 || ODD;
  __shared__ TileMaps sh;
  const int wave = wave_id();
  const int D = (int)p.channels;
  const int64_t n = sequence_tokens(p, tiles.b0 + blockIdx.y);
  const Place place = draw_place<true>(tiles, scratch, &sh.tile);
  if (place.run < 0) return;
  const int64_t b = place.b, col = place.col, chunk = place.run;
  const int ch = place.part * kTileChannels + 2 * lane_id();
  const int have = D - ch >= 2 ? 2 : (D - ch == 1 ? 1 : 0);
  // lanes past the last channel work on the last one (pair), unheard
  const int c0 = ODD ? (ch < D ? ch : D - 1) : (ch < D ? ch : D - 2);
  const int c1 = ch + 1 < D ? ch + 1 : D - 1;
  const uint32_t o0 = (uint32_t)c0 * eb, o1 = (uint32_t)c1 * eb;
  const int64_t t0 = chunk * kFwdTile + wave * T;          // this wave's first token
  const uintptr_t yrow = (uintptr_t)yv + ((b * p.length + t0) * D) * eb, ystep = (uintptr_t)D * eb;
  const int room = (int)(p.length - t0 < T ? p.length - t0 : T);   // tokens of the output
  if (chunk * kFwdTile >= n) {                             // no token of this tile exists
    Raw zeros[T];
#pragma unroll
    for (int k = 0; k < T; ++k) zeros[k] = PIO::splat(0.0f);
    PIO::store_rows(yrow, ystep, o0, zeros, room, have);
    if (chunk == 0 && wave == 0 && final_state != nullptr) {
      const float* s0 = p.initial_state == nullptr ? nullptr : p.initial_state + b * D + ch;
      if (have > 0) final_state[b * D + ch] = s0 == nullptr ? 0.0f : s0[0];
      if (have > 1) final_state[b * D + ch + 1] = s0 == nullptr ? 0.0f : s0[1];
    }
    return;
  }
  const int count = (int)(n - t0 <= 0 ? 0 : (n - t0 < T ? n - t0 : T));
  // the rates first: loads return in order, and the first token must not wait for the
  // last one's
  float nr[2] = {0.0f, 0.0f};
  if constexpr (RATE) {
    nr[0] = rate_log2(p.rate[c0]);
    nr[1] = rate_log2(p.rate[c1]);
  }
  // (past the last token it is read again)
  const int64_t first_token = count > 0 ? t0 : n - 1;
  Rows ax((uintptr_t)p.x, p.x_batch, p.x_token, b, first_token, eb);
  Rows af((uintptr_t)p.forget, p.forget_batch, p.forget_token, b, first_token, eb);
  Rows ai((uintptr_t)p.input_gate, p.input_batch, p.input_token, b, first_token, eb);
  Rows az((uintptr_t)p.z, p.z_batch, p.z_token, b, first_token, eb);
  Raw rx[T], rf[T], ri[IG ? T : 1], rz[Z ? T : 1];
#pragma unroll
  for (int k = 0; k < T; ++k) {
    rx[k] = PIO::load(ax.at, o0, o1);
    rf[k] = PIO::load(af.at, o0, o1);
    if constexpr (IG) ri[k] = PIO::load(ai.at, o0, o1);
    if constexpr (Z && !kLateZ) rz[k] = PIO::load(az.at, o0, o1);
    const uintptr_t on = k + 1 < count ? ~(uintptr_t)0 : 0;
    ax.next(on);
    af.next(on);
    ai.next(on);
    if constexpr (!kLateZ) az.next(on);
  }
  float h[2] = {0.0f, 0.0f};                               // what enters the sequence
  if (p.initial_state != nullptr && chunk < kTileGroup) {
    h[0] = p.initial_state[b * D + c0];
    h[1] = p.initial_state[b * D + c1];
  }
  if (count < T) {                                         // tokens that do not exist: a = 1, u = 0
#pragma unroll
    for (int k = 0; k < T; ++k) {
      if (k < count) continue;
      rx[k] = PIO::splat(0.0f);
      rf[k] = PIO::splat(RATE ? -__builtin_huge_valf() : __builtin_huge_valf());
      if constexpr (IG) ri[k] = PIO::splat(0.0f);
    }
  }
  float a[T][2], u[T][2], l[2] = {0.0f, 0.0f}, last[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < T; ++k) {
    float x[2], f[2], v[2];
    PIO::IO::unpack(rx[k], x);
    PIO::IO::unpack(rf[k], f);
    if constexpr (IG) PIO::IO::unpack(ri[k], v);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const Gate g = gate<RATE>(f[c], nr[c]);
      a[k][c] = g.a;
      u[k][c] = g.w * x[c];
      if constexpr (IG) u[k][c] *= sigmoid(v[c]);
      l[c] += g.log_a;
      last[c] = __builtin_fmaf(g.a, last[c], u[k][c]);
    }
    // token after token: left alone, the compiler starts many at once and runs out
    // of registers
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (Z && kLateZ) {
#pragma unroll
    for (int k = 0; k < T; ++k) {
      rz[k] = PIO::load(az.at, o0, o1);
      az.next(k + 1 < count ? ~(uintptr_t)0 : 0);
    }
  }
  put2(sh.l[wave], l[0], l[1]);
  put2(sh.m[wave], half_decay(l[0]), half_decay(l[1]));
  put2(sh.b[wave], last[0], last[1]);
  lds_barrier();
  if (tiles.chunks > 1) {
    const float first[2] = {h[0], h[1]};
    tile_entry(sh, wave, chunk, (n + kFwdTile - 1) / kFwdTile, col, tiles.cols(), scratch,
               tiles.chunks, first, h);
  }
  wave_entry(sh, wave, h);
  if (starts != nullptr && t0 % kGatedKeepTokens == 0 && t0 < n) {
    const int64_t blocks = (p.length + kGatedKeepTokens - 1) / kGatedKeepTokens;
    float* at = starts + (b * blocks + t0 / kGatedKeepTokens) * D + ch;
    if (have > 0) at[0] = h[0];
    if (have > 1) at[1] = h[1];
  }
  Raw out[T];
#pragma unroll
  for (int k = 0; k < T; ++k) {
    float y[2], z[2];
    if constexpr (Z) PIO::IO::unpack(rz[k], z);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      h[c] = __builtin_fmaf(a[k][c], h[c], u[k][c]);
      y[c] = h[c];
      if constexpr (Z) y[c] *= silu(z[c]);
    }
    out[k] = PIO::IO::pack(y);
  }
  if (count < T) {
#pragma unroll
    for (int k = 0; k < T; ++k) out[k] = k < count ? out[k] : PIO::splat(0.0f);
  }
  PIO::store_rows(yrow, ystep, o0, out, room, have);
  if (final_state != nullptr && count > 0 && t0 + count == n) {
    if (have > 0) final_state[b * D + ch] = h[0];
    if (have > 1) final_state[b * D + ch + 1] = h[1];
  }
}

__global__ __launch_bounds__(256) void tile_clear_kernel(uint64_t* scratch, int64_t tickets,
                                                         int64_t words) {
  typedef uint64_t two __attribute__((ext_vector_type(2)));
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words / 2; i += (int64_t)gridDim.x * 256)
    *gptr<two>((uintptr_t)(scratch + 2 * i)) =
        2 * i < tickets ? two{0, 0} : two{~0ull, ~0ull};
}

hipError_t launch_tile_clear(uint64_t* scratch, int64_t tickets, int64_t words, hipStream_t stream) {
  const int64_t blocks = (words / 2 + 255) / 256;
  tile_clear_kernel<<<dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream>>>(scratch, tickets,
                                                                                          words);
  return hipGetLastError();
}

size_t gated_scan_scratch(const GatedProblem& p) { return (size_t)gated_tiles(p, kFwdTile).words() * 8; }

template <class F, bool RATE, bool IG, bool Z>
static hipError_t launch_gated_z(const GatedProblem& p, void* y, float* final_state, float* starts,
                                 uint64_t* scratch, hipStream_t stream) {
  const bool past = past_caches(p.batch * p.length * p.channels * (int64_t)sizeof(typename F::S));
  return launch_tiles(gated_tiles(p, kFwdTile), p.batch, scratch, stream, [&](dim3 grid, const Tiles& t) {
    const dim3 block(kTileThreads);
    if (p.channels % 2 != 0)
      gated_scan_kernel<F, RATE, IG, Z, Rows2::Singles><<<grid, block, 0, stream>>>(
          p, y, final_state, starts, scratch, t);
    else if (past && starts == nullptr)
      gated_scan_kernel<F, RATE, IG, Z, Rows2::PairsOnce><<<grid, block, 0, stream>>>(
          p, y, final_state, starts, scratch, t);
    else if (past)
      gated_scan_kernel<F, RATE, IG, Z, Rows2::PairsPast><<<grid, block, 0, stream>>>(
          p, y, final_state, starts, scratch, t);
    else
      gated_scan_kernel<F, RATE, IG, Z, Rows2::Pairs><<<grid, block, 0, stream>>>(
          p, y, final_state, starts, scratch, t);
  });
}

template <class F, bool RATE>
static hipError_t launch_gated_r(const GatedProblem& p, void* y, float* final_state, float* starts,
                                 uint64_t* s, hipStream_t stream) {
  if (p.input_gate != nullptr)
    return p.z != nullptr ? launch_gated_z<F, RATE, true, true>(p, y, final_state, starts, s, stream)
                          : launch_gated_z<F, RATE, true, false>(p, y, final_state, starts, s, stream);
  return p.z != nullptr ? launch_gated_z<F, RATE, false, true>(p, y, final_state, starts, s, stream)
                        : launch_gated_z<F, RATE, false, false>(p, y, final_state, starts, s, stream);
}

template <class F>
static hipError_t launch_gated_f(const GatedProblem& p, void* y, float* final_state, float* starts,
                                 void* scratch, hipStream_t stream) {
  return p.rate != nullptr
             ? launch_gated_r<F, true>(p, y, final_state, starts, (uint64_t*)scratch, stream)
             : launch_gated_r<F, false>(p, y, final_state, starts, (uint64_t*)scratch, stream);
}

hipError_t launch_gated_scan(const GatedProblem& p, Fmt fmt, void* y, float* final_state,
                             float* starts, void* scratch, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_gated_f<FmtF32>(p, y, final_state, starts, scratch, stream);
    case Fmt::F16: return launch_gated_f<FmtF16>(p, y, final_state, starts, scratch, stream);
    case Fmt::BF16: return launch_gated_f<FmtBF16>(p, y, final_state, starts, scratch, stream);
    default: return hipErrorInvalidValue;
  }
}

template <class F, bool RATE>
__device__ __forceinline__ float gated_token(float h, typename F::S x, typename F::S f,
                                             const typename F::S* ig, float nr) {
  const Gate g = gate<RATE>(widen<F>(f), nr);
  float u = g.w * widen<F>(x);
  if (ig != nullptr) u *= sigmoid(widen<F>(*ig));
  return __builtin_fmaf(g.a, h, u);
}

// One token: a thread per channel (128 x 4096 bfloat16: 4.2 us, 8.4 MB).
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
