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
// What is carried is c[t] = a[t] g[t], from the last token to the first: the same
// maps as the forward's, c -> 2^l c + b, in tiles of 64 tokens (gated_tile.hpp).  The
// states are found again from the tile's first, which the forward kept.  A wave has 8
// tokens: decay, weight and state of each stay in registers with the inputs, the
// sigmoids are computed a second time (all of it kept would leave room for half as
// many waves).
//
// 4 x 2048 x 2048 bfloat16 with rate and input gate: 62 us, 236 MB at 3.8 TB/s; the
// vector units, 75% busy, bound it.  3 x 777 x 522 float32: 12.6 us.
#include "gated_tile.hpp"

namespace sca {

constexpr int kGradTokens = 8;                              // of a wave
constexpr int kGradTile = kGradTokens * kTileWaves;         // of a workgroup
static_assert(kGradTile == kGatedKeepTokens, "a tile starts from a kept state");

// Waves a SIMD: float32's inputs take twice the registers, and with two workgroups a
// CU some of them would go to memory (4 x 2048 x 2304, rate and input gate: 110 us, in four
// waves 136; 4 x 2048 x 2048, output gate: 95 and 100).
template <class F, bool RATE, bool IG, bool Z>
constexpr int kGradWaves = sizeof(typename F::S) == 4 && (RATE || IG || Z) ? 2 : 4;

template <class F, bool RATE, bool IG, bool Z, Rows2 ROWS>
__global__ __launch_bounds__(kTileThreads)
__attribute__((amdgpu_waves_per_eu(kGradWaves<F, RATE, IG, Z>, kGradWaves<F, RATE, IG, Z>)))
void gated_scan_grad_kernel(GatedProblem p, GatedGrads g, uint64_t* scratch, float* partial, Tiles tiles) {
  using S = typename F::S;
  using PIO = PairIO<F, ROWS>;
  constexpr bool ODD = PIO::ODD;
  using IO = typename PIO::IO;
  using Raw = typename PIO::Raw;
  constexpr int T = kGradTokens;
  constexpr int eb = sizeof(S);
  __shared__ TileMaps sh;
  __shared__ float forward_b[kTileWaves][kTileChannels];
  const int wave = wave_id(), turn = kTileWaves - 1 - wave;  // its turn in the walk
  const int D = (int)p.channels;
  const int64_t n = sequence_tokens(p, tiles.b0 + blockIdx.y);
  const Place place = draw_place<false>(tiles, scratch, &sh.tile);
  if (place.run < 0) return;
  const int64_t b = place.b, col = place.col, chunk = tiles.chunks - 1 - place.run;
  const int ch = place.part * kTileChannels + 2 * lane_id();
  const int have = D - ch >= 2 ? 2 : (D - ch == 1 ? 1 : 0);
  // lanes past the last channel work on the last one (pair), unheard
  const int c0 = ODD ? (ch < D ? ch : D - 1) : (ch < D ? ch : D - 2);
  const int c1 = ch + 1 < D ? ch + 1 : D - 1;
  const uint32_t o0 = (uint32_t)c0 * eb, o1 = (uint32_t)c1 * eb;
  const int64_t t0 = chunk * kGradTile + wave * T;         // this wave's first token
  const uintptr_t out = ((b * p.length + t0) * D) * eb, ostep = (uintptr_t)D * eb;
  const int room = (int)(p.length - t0 < T ? p.length - t0 : T);
  if (chunk * kGradTile >= n) {                            // no token of this tile exists
    Raw zeros[T];
#pragma unroll
    for (int k = 0; k < T; ++k) zeros[k] = PIO::splat(0.0f);
    PIO::store_rows((uintptr_t)g.dx + out, ostep, o0, zeros, room, have);
    PIO::store_rows((uintptr_t)g.dforget + out, ostep, o0, zeros, room, have);
    if constexpr (IG) PIO::store_rows((uintptr_t)g.dinput_gate + out, ostep, o0, zeros, room, have);
    if constexpr (Z) PIO::store_rows((uintptr_t)g.dz + out, ostep, o0, zeros, room, have);
    if (wave == 0) {
      float* at = partial + (b * tiles.chunks + chunk) * D + ch;
      if (RATE && have > 0) at[0] = 0.0f;
      if (RATE && have > 1) at[1] = 0.0f;
      if (chunk == 0 && g.dinitial != nullptr) {
        const float* s0 = g.dfinal == nullptr ? nullptr : g.dfinal + b * D + ch;
        if (have > 0) g.dinitial[b * D + ch] = s0 == nullptr ? 0.0f : s0[0];
        if (have > 1) g.dinitial[b * D + ch + 1] = s0 == nullptr ? 0.0f : s0[1];
      }
    }
    return;
  }
  const int count = (int)(n - t0 <= 0 ? 0 : (n - t0 < T ? n - t0 : T));
  // the rates and the state first: loads return in order, and the first token must not
  // wait for the last one's
  float nr[2] = {0.0f, 0.0f}, h[2];
  if constexpr (RATE) {
    nr[0] = rate_log2(p.rate[c0]);
    nr[1] = rate_log2(p.rate[c1]);
  }
  {
    const int64_t blocks = (p.length + kGatedKeepTokens - 1) / kGatedKeepTokens;
    const float* at = g.starts + (b * blocks + chunk) * D;
    h[0] = at[c0];
    h[1] = at[c1];
  }
  // (past the last token it is read again)
  const int64_t first_token = count > 0 ? t0 : n - 1;
  Rows ax((uintptr_t)p.x, p.x_batch, p.x_token, b, first_token, eb);
  Rows af((uintptr_t)p.forget, p.forget_batch, p.forget_token, b, first_token, eb);
  Rows ai((uintptr_t)p.input_gate, p.input_batch, p.input_token, b, first_token, eb);
  Rows az((uintptr_t)p.z, p.z_batch, p.z_token, b, first_token, eb);
  Rows ad((uintptr_t)g.dy, g.dy_batch, g.dy_token, b, first_token, eb);
  Raw rx[T], rf[T], ri[IG ? T : 1], rz[Z ? T : 1], rd[T];
#pragma unroll
  for (int k = 0; k < T; ++k) {
    rx[k] = PIO::load(ax.at, o0, o1);
    rf[k] = PIO::load(af.at, o0, o1);
    if constexpr (IG) ri[k] = PIO::load(ai.at, o0, o1);
    if constexpr (Z) rz[k] = PIO::load(az.at, o0, o1);
    rd[k] = PIO::load(ad.at, o0, o1);
    const uintptr_t on = k + 1 < count ? ~(uintptr_t)0 : 0;
    ax.next(on);
    af.next(on);
    ai.next(on);
    az.next(on);
    ad.next(on);
  }
  const int64_t steps = (n + kGradTile - 1) / kGradTile;
  float c[2] = {0.0f, 0.0f};                               // what enters the sequence from behind
  if (g.dfinal != nullptr && steps - 1 - chunk < kTileGroup) {
    c[0] = g.dfinal[b * D + c0];
    c[1] = g.dfinal[b * D + c1];
  }
  if (count < T) {                                         // tokens that do not exist: a = 1, u = q = 0
#pragma unroll
    for (int k = 0; k < T; ++k) {
      if (k < count) continue;
      rx[k] = rd[k] = PIO::splat(0.0f);
      rf[k] = PIO::splat(RATE ? -__builtin_huge_valf() : __builtin_huge_valf());
      if constexpr (IG) ri[k] = PIO::splat(0.0f);
      if constexpr (Z) rz[k] = PIO::splat(0.0f);
    }
  }
  // hs: first the input's part of each token, then the state before it
  float a[T][2], w[RATE ? T : 1][2], hs[T][2];
  float l[2] = {0.0f, 0.0f}, last[2] = {0.0f, 0.0f}, back[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < T; ++k) {
    float x[2], f[2], v[2];
    IO::unpack(rx[k], x);
    IO::unpack(rf[k], f);
    if constexpr (IG) IO::unpack(ri[k], v);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const Gate gt = gate<RATE>(f[j], nr[j]);
      a[k][j] = gt.a;
      if constexpr (RATE) w[k][j] = gt.w;
      hs[k][j] = gt.w * x[j];
      if constexpr (IG) hs[k][j] *= sigmoid(v[j]);
      l[j] += gt.log_a;
      last[j] = __builtin_fmaf(gt.a, last[j], hs[k][j]);
    }
    __builtin_amdgcn_sched_barrier(0);                     // token after token, as in the forward
  }
#pragma unroll
  for (int k = T - 1; k >= 0; --k) {
    float q[2], z[2];
    IO::unpack(rd[k], q);
    if constexpr (Z) IO::unpack(rz[k], z);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (Z) q[j] *= silu(z[j]);
      back[j] = a[k][j] * (q[j] + back[j]);
    }
  }
  put2(sh.l[turn], l[0], l[1]);
  put2(sh.m[turn], half_decay(l[0]), half_decay(l[1]));
  put2(sh.b[turn], back[0], back[1]);
  put2(forward_b[wave], last[0], last[1]);
  lds_barrier();
  if (tiles.chunks > 1) {
    const float first[2] = {c[0], c[1]};
    tile_entry(sh, turn, steps - 1 - chunk, steps, col, tiles.cols(), scratch, tiles.chunks, first, c);
  }
  wave_entry(sh, turn, c);
  for (int i = 0; i < wave; ++i) {                         // the state that enters this wave's run
    float m[2], fb[2];
    get2(sh.m[kTileWaves - 1 - i], m);
    get2(forward_b[i], fb);
#pragma unroll
    for (int j = 0; j < 2; ++j) h[j] = carry_over(m[j], fb[j], h[j]);
  }
#pragma unroll
  for (int k = 0; k < T; ++k)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float u = hs[k][j];
      hs[k][j] = h[j];
      h[j] = __builtin_fmaf(a[k][j], h[j], u);
    }
  float total[2] = {0.0f, 0.0f};
  const float p_rate[2] = {nr[0] * -kLn2, nr[1] * -kLn2};  // the rates again, at most 1e38: P stays finite
  Raw ox[T], of[T], oi[IG ? T : 1], oz[Z ? T : 1];
#pragma unroll
  for (int k = T - 1; k >= 0; --k) {
    float x[2], f[2], v[2], z[2], d[2], dx[2], df[2], di[2], dz[2];
    IO::unpack(PIO::again(rx[k]), x);
    IO::unpack(PIO::again(rf[k]), f);
    IO::unpack(PIO::again(rd[k]), d);
    if constexpr (IG) IO::unpack(PIO::again(ri[k]), v);
    if constexpr (Z) IO::unpack(PIO::again(rz[k]), z);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float q = d[j];
      if constexpr (Z) {
        q *= silu(z[j]);
        dz[j] = d[j] * h[j] * silu_slope(z[j]);
        h[j] = hs[k][j];
      }
      const Sides s = sides(f[j]);
      Sides vs = {1.0f, 0.0f};
      if constexpr (IG) vs = sides(v[j]);
      const float grad = q + c[j], gv = grad * vs.up;
      const float weight = RATE ? w[RATE ? k : 0][j] : s.down;
      dx[j] = gv * weight;
      if constexpr (IG) di[j] = dx[j] * x[j] * vs.down;
      if constexpr (RATE) {
        // (p / w is 0 where both are)
        const float P = p_rate[j] * s.up, pw = P * rcp_hw(__builtin_fmaxf(weight, 1e-30f));
        const float A = a[k][j];
        const float E = gv * x[j] * (A * A * pw) - grad * (P * A * hs[k][j]);
        df[j] = E * s.down;
        total[j] += E;
      } else {
        df[j] = (grad * hs[k][j] - gv * x[j]) * (s.up * s.down);
      }
      c[j] = a[k][j] * grad;
    }
    ox[k] = IO::pack(dx);
    of[k] = IO::pack(df);
    if constexpr (IG) oi[k] = IO::pack(di);
    if constexpr (Z) oz[k] = IO::pack(dz);
    __builtin_amdgcn_sched_barrier(0);
  }
  if (count < T) {
#pragma unroll
    for (int k = 0; k < T; ++k) {
      const bool on = k < count;
      ox[k] = on ? ox[k] : PIO::splat(0.0f);
      of[k] = on ? of[k] : PIO::splat(0.0f);
      if constexpr (IG) oi[k] = on ? oi[k] : PIO::splat(0.0f);
      if constexpr (Z) oz[k] = on ? oz[k] : PIO::splat(0.0f);
    }
  }
  PIO::store_rows((uintptr_t)g.dx + out, ostep, o0, ox, room, have);
  PIO::store_rows((uintptr_t)g.dforget + out, ostep, o0, of, room, have);
  if constexpr (IG) PIO::store_rows((uintptr_t)g.dinput_gate + out, ostep, o0, oi, room, have);
  if constexpr (Z) PIO::store_rows((uintptr_t)g.dz + out, ostep, o0, oz, room, have);
  if (g.dinitial != nullptr && t0 == 0) {
    if (have > 0) g.dinitial[b * D + ch] = c[0];
    if (have > 1) g.dinitial[b * D + ch + 1] = c[1];
  }
  if constexpr (RATE) {                                    // the tile's sums, wave after wave
    __syncthreads();
    put2(sh.l[wave], total[0], total[1]);
    __syncthreads();
    if (wave == 0) {
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kTileWaves; ++i) {
        float e[2];
        get2(sh.l[i], e);
        sum[0] += e[0];
        sum[1] += e[1];
      }
      float* at = partial + (b * tiles.chunks + chunk) * D + ch;
      if (have > 0) at[0] = sum[0];
      if (have > 1) at[1] = sum[1];
    }
  }
}

// drate from the tiles' sums: 64 channels a workgroup, 16 strands of tiles each, added up in
// 64 bits: a strand has thousands of rows where sequences are many, and in 32 bits equal
// terms drift by as many roundings of the sum.  (4.7 us for 128 tiles of 2048 channels;
// latency.)
__global__ __launch_bounds__(1024) void gated_rate_kernel(const float* partial, const float* rate,
                                                          float* drate, int64_t rows, int64_t channels) {
  __shared__ double strand[16][64];
  const int64_t c = (int64_t)blockIdx.x * 64 + lane_id();
  double sum = 0.0;
  if (c < channels) {
#pragma unroll 8
    for (int64_t i = threadIdx.x / 64; i < rows; i += 16) sum += (double)partial[i * channels + c];
  }
  strand[threadIdx.x / 64][lane_id()] = sum;
  __syncthreads();
  if (threadIdx.x >= 64 || c >= channels) return;
  for (int i = 1; i < 16; ++i) sum += strand[i][lane_id()];
  const float r = rate[c];
  drate[c] = r <= 0.0f ? 0.0f : (float)(sum / (double)r);
}

size_t gated_scan_grad_scratch(const GatedProblem& p) {
  const Tiles t = gated_tiles(p, kGradTile);
  const size_t sums = p.rate == nullptr ? 0 : (size_t)(p.batch * t.chunks * p.channels) * 4;
  return (size_t)t.words() * 8 + sums;
}

template <class F, bool RATE, bool IG, bool Z>
static hipError_t launch_grad_z(const GatedProblem& p, const GatedGrads& g, void* scratch, hipStream_t stream) {
  const Tiles tiles = gated_tiles(p, kGradTile);
  const bool past = past_caches(p.batch * p.length * p.channels * (int64_t)sizeof(typename F::S));
  uint64_t* words = (uint64_t*)scratch;
  float* partial = (float*)(words + tiles.words());
  hipError_t e = hipSuccess;
  if (p.batch > 0)
    e = launch_tiles(tiles, p.batch, words, stream, [&](dim3 grid, const Tiles& t) {
      const dim3 block(kTileThreads);
      if (p.channels % 2 != 0)
        gated_scan_grad_kernel<F, RATE, IG, Z, Rows2::Singles><<<grid, block, 0, stream>>>(p, g, words, partial, t);
      else if (past)
        gated_scan_grad_kernel<F, RATE, IG, Z, Rows2::PairsOnce><<<grid, block, 0, stream>>>(p, g, words, partial, t);
      else
        gated_scan_grad_kernel<F, RATE, IG, Z, Rows2::Pairs><<<grid, block, 0, stream>>>(p, g, words, partial, t);
    });
  if (e != hipSuccess || !RATE) return e;
  gated_rate_kernel<<<dim3((unsigned)((p.channels + 63) / 64)), dim3(1024), 0, stream>>>(
      partial, p.rate, g.drate, p.batch * tiles.chunks, p.channels);
  return hipGetLastError();
}

template <class F, bool RATE>
static hipError_t launch_grad_r(const GatedProblem& p, const GatedGrads& g, void* s, hipStream_t stream) {
  if (p.input_gate != nullptr)
    return p.z != nullptr ? launch_grad_z<F, RATE, true, true>(p, g, s, stream)
                          : launch_grad_z<F, RATE, true, false>(p, g, s, stream);
  return p.z != nullptr ? launch_grad_z<F, RATE, false, true>(p, g, s, stream)
                        : launch_grad_z<F, RATE, false, false>(p, g, s, stream);
}

template <class F>
static hipError_t launch_grad_f(const GatedProblem& p, const GatedGrads& g, void* s, hipStream_t stream) {
  return p.rate != nullptr ? launch_grad_r<F, true>(p, g, s, stream)
                           : launch_grad_r<F, false>(p, g, s, stream);
}

hipError_t launch_gated_scan_grad(const GatedProblem& p, Fmt fmt, const GatedGrads& g,
                                  void* scratch, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_grad_f<FmtF32>(p, g, scratch, stream);
    case Fmt::F16: return launch_grad_f<FmtF16>(p, g, scratch, stream);
    case Fmt::BF16: return launch_grad_f<FmtBF16>(p, g, scratch, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sca
