// Selective scan, forward and single-token step:
//   dt = softplus(dt_raw + dt_bias),  h[t] = exp(dt A) h[t-1] + dt x B,
//   y = (C . h + D x) silu(z)
// per channel, with `states` states each.  See scan_tile.hpp for the mapping.
#include "scan_tile.hpp"

namespace sca {

template <class F, int K, int NG>
__global__ __launch_bounds__(kScanThreads) void selective_scan_kernel(ScanProblem p, void* yv,
                                                                     float* final_state,
                                                                     float* starts, int64_t b0,
                                                                     int64_t tiles) {
  using S = typename F::S;
  using Tile = TileStage<F, K>;
  using Rows = RowStage<F, K, NG>;
  constexpr int TB = 64 * K;
  __shared__ alignas(16) float s_B[NG * TB], s_C[NG * TB];
  __shared__ alignas(16) uint32_t s_x[Tile::WORDS], s_dt[Tile::WORDS], s_z[Tile::WORDS];

  const int lane = lane_id(), wave = wave_id();
  const ScanPlace at = scan_place(p, b0, tiles);
  const int64_t len = scan_length(p, at.b);
  const int N = (int)p.states;
  const bool gate = p.z != nullptr;
  const auto xs = tile_src<F>(p.x, p.x_batch, p.x_token, at.b, at.ch);
  const auto dts = tile_src<F>(p.dt, p.dt_batch, p.dt_token, at.b, at.ch);
  const auto zs = tile_src<F>(p.z, p.z_batch, p.z_token, at.b, at.ch);
  const auto Bs = tile_src<F>(p.B, p.B_batch, p.B_token, at.b, at.g * p.B_group);
  const auto Cs = tile_src<F>(p.C, p.C_batch, p.C_token, at.b, at.g * p.C_group);
  S* y = (S*)yv + at.b * p.length * p.channels + at.ch;
  const bool yvec = (uintptr_t)y % 16 == 0 && (p.channels * (int64_t)sizeof(S)) % 16 == 0;

  // lane n of these registers holds state n of the wave's two channels
  float A2[2], carry[2], Dc[2], bias[2];
  bool live[2];
  int64_t row[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    live[c] = 2 * wave + c < at.nch;
    const int64_t ch = at.ch + 2 * wave + c;
    row[c] = (at.b * p.channels + ch) * N + lane;
    const bool on = live[c] && lane < N;
    A2[c] = on ? p.A[ch * N + lane] * kLog2e : 0.0f;
    carry[c] = on && p.initial_state != nullptr ? p.initial_state[row[c]] : 0.0f;
    Dc[c] = live[c] && p.D != nullptr ? p.D[ch] : 0.0f;
    bias[c] = live[c] && p.dt_bias != nullptr ? p.dt_bias[ch] : 0.0f;
  }

  Tile rx, rdt, rz;
  Rows rB, rC;
  auto fetch = [&](int64_t t0) {
    rx.load(xs, t0, len, at.nch);
    rdt.load(dts, t0, len, at.nch);
    if (gate) rz.load(zs, t0, len, at.nch);
  };
  const int64_t blocks = (len + TB - 1) / TB;
  if (blocks > 0) {
    fetch(0);
    rB.load(Bs, 0, len, 0, N);
    rC.load(Cs, 0, len, 0, N);
  }
  for (int64_t blk = 0; blk < blocks; ++blk) {
    const int64_t t0 = blk * TB;
    __syncthreads();                       // the last block's LDS is free
    rx.put(s_x);
    rdt.put(s_dt);
    if (gate) rz.put(s_z);
    if (starts != nullptr) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (live[c] && lane < N) {
          const int64_t nblk = (p.length + TB - 1) / TB;
          const int64_t ch = at.ch + 2 * wave + c;
          starts[((at.b * nblk + blk) * p.channels + ch) * N + lane] = carry[c];
        }
    }
    rB.put(s_B);
    rC.put(s_C);
    __syncthreads();
    float dt[K][2], u[K][2], acc[K][2], span[2];
    Tile::get(s_x, wave, lane, u);
    Tile::get(s_dt, wave, lane, dt);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float total = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float raw = dt[k][c] + bias[c];
        const float d = p.softplus ? softplus(raw) : raw;
        dt[k][c] = t0 + lane * K + k < len ? d : 0.0f;   // past the end: a = 1, b = 0
        total += dt[k][c];
        acc[k][c] = Dc[c] * u[k][c];
        u[k][c] *= dt[k][c];
      }
      span[c] = total;
    }
    for (int n0 = 0; n0 < N; n0 += NG) {
      if (n0 > 0) {
        __syncthreads();
        rB.put(s_B);
        rC.put(s_C);
        __syncthreads();
      }
      // the next rows (of this block or the next) travel while these are used
      if (n0 + NG < N) {
        rB.load(Bs, t0, len, n0 + NG, N);
        rC.load(Cs, t0, len, n0 + NG, N);
      } else if (blk + 1 < blocks) {
        fetch(t0 + TB);
        rB.load(Bs, t0 + TB, len, 0, N);
        rC.load(Cs, t0 + TB, len, 0, N);
      }
      const int nn = N - n0 < NG ? N - n0 : NG;
      for (int i = 0; i < nn; ++i) {
        const int n = n0 + i;
        float Bk[K], Ck[K];
        plane_read<K>(s_B + i * TB, lane, Bk);
        plane_read<K>(s_C + i * TB, lane, Ck);
        float a[2][K], b[2][K], P[2], H[2], h0[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float An = readlane(A2[c], n);
          float h = 0.0f;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            a[c][k] = exp2_hw(dt[k][c] * An);
            b[c][k] = u[k][c] * Bk[k];
            h = __builtin_fmaf(a[c][k], h, b[c][k]);
          }
          P[c] = exp2_hw(span[c] * An);
          h0[c] = readlane(carry[c], n);
          // the block's start enters through the first lane
          H[c] = __builtin_fmaf(P[c], lane == 0 ? h0[c] : 0.0f, h);
        }
        affine_scan2(H[0], H[1], P[0], P[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          carry[c] = lane == n ? readlane(H[c], kWave - 1) : carry[c];
          float h = dpp<kWaveShr1, 0xf>(H[c], h0[c]);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            h = __builtin_fmaf(a[c][k], h, b[c][k]);
            acc[k][c] = __builtin_fmaf(Ck[k], h, acc[k][c]);
          }
        }
      }
    }
    if (gate) {
      float zv[K][2];
      Tile::get(s_z, wave, lane, zv);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < K; ++k) acc[k][c] *= silu(zv[k][c]);
    }
    Tile::set(s_x, wave, lane, acc);       // the wave's own planes, read above by itself alone
    __syncthreads();
    Tile::store(s_x, y, p.channels, yvec, t0, len, at.nch);
  }
  // tokens past the sequence's end
  for (int64_t i = len * kScanTile + threadIdx.x; i < p.length * kScanTile; i += kScanThreads)
    if (i % kScanTile < at.nch) y[(i / kScanTile) * p.channels + i % kScanTile] = S(0);
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (live[c] && lane < N && final_state != nullptr) final_state[row[c]] = carry[c];
}

// Tokens per lane by length: the smallest block that holds the sequence, up
// to 512 tokens (256 in float32, whose planes are twice as large).  A lane that
// owns more tokens pays the cross-lane scan (about 20 instructions per channel
// and state) fewer times; a block longer than the sequence leaves lanes idle.
static int scan_k(int64_t length, Fmt fmt) {
  if (length <= 64) return 1;
  if (length <= 128) return 2;
  return length <= 256 || fmt == Fmt::F32 ? 4 : 8;
}
int64_t scan_block_tokens(int64_t length, Fmt fmt) { return 64 * scan_k(length, fmt); }

// Workgroups of a launch: grid sizes count work-items in 32 bits, so batches
// beyond that go out as several launches.
constexpr int64_t kMaxGroups = 1ll << 22;

template <class F, int K>
static hipError_t launch_fwd(const ScanProblem& p, void* y, float* final_state, float* starts,
                             hipStream_t stream) {
  const int64_t tiles = (p.channels / p.groups + kScanTile - 1) / kScanTile;
  const int64_t per = tiles * p.groups;
  const int64_t step = kMaxGroups / per < 1 ? 1 : kMaxGroups / per;
  for (int64_t b0 = 0; b0 < p.batch; b0 += step) {
    const int64_t nb = p.batch - b0 < step ? p.batch - b0 : step;
    selective_scan_kernel<F, K, sizeof(typename F::S) == 2 ? 16 : 8>
        <<<dim3((unsigned)(nb * per)), dim3(kScanThreads), 0, stream>>>(p, y, final_state, starts,
                                                                       b0, tiles);
  }
  return hipGetLastError();
}

template <class F>
static hipError_t launch_fwd_f(const ScanProblem& p, Fmt fmt, void* y, float* final_state,
                               float* starts, hipStream_t stream) {
  switch (scan_k(p.length, fmt)) {
    case 1: return launch_fwd<F, 1>(p, y, final_state, starts, stream);
    case 2: return launch_fwd<F, 2>(p, y, final_state, starts, stream);
    case 4: return launch_fwd<F, 4>(p, y, final_state, starts, stream);
    default:
      if constexpr (sizeof(typename F::S) == 2) {
        return launch_fwd<F, 8>(p, y, final_state, starts, stream);
      }
      return hipErrorInvalidValue;
  }
}

hipError_t launch_selective_scan(const ScanProblem& p, Fmt fmt, void* y, float* final_state,
                                 float* starts, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_fwd_f<FmtF32>(p, fmt, y, final_state, starts, stream);
    case Fmt::F16: return launch_fwd_f<FmtF16>(p, fmt, y, final_state, starts, stream);
    case Fmt::BF16: return launch_fwd_f<FmtBF16>(p, fmt, y, final_state, starts, stream);
    default: return hipErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// One token: G lanes (a power of two) share a channel, lane q of them owning
// states q, q + G, ...; the state is read and written once.
// ---------------------------------------------------------------------------
template <class F, int G>
__global__ __launch_bounds__(256) void selective_scan_step_kernel(ScanProblem p,
                                                                 const float* state,
                                                                 float* new_state, void* yv) {
  using S = typename F::S;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G;   // (sequence, channel)
  const int q = threadIdx.x % G;
  const int N = (int)p.states;
  if (i >= p.batch * p.channels) return;                // whole groups of G lanes leave together
  const int64_t b = i / p.channels, ch = i % p.channels;
  const int64_t g = ch / (p.channels / p.groups);
  const float x = widen<F>(((const S*)p.x)[b * p.x_batch + ch]);
  float dt = widen<F>(((const S*)p.dt)[b * p.dt_batch + ch]);
  if (p.dt_bias != nullptr) dt += p.dt_bias[ch];
  if (p.softplus) dt = softplus(dt);
  const float u = dt * x;
  const S* Bp = (const S*)p.B + b * p.B_batch + g * p.B_group;
  const S* Cp = (const S*)p.C + b * p.C_batch + g * p.C_group;
  float acc = 0.0f;
  for (int n = q; n < N; n += G) {
    const float a = exp2_hw(dt * (p.A[ch * N + n] * kLog2e));
    const float h = __builtin_fmaf(a, state[i * N + n], u * widen<F>(Bp[n]));
    new_state[i * N + n] = h;
    acc = __builtin_fmaf(h, widen<F>(Cp[n]), acc);
  }
#pragma unroll
  for (int m = G / 2; m > 0; m /= 2) acc += __shfl_xor(acc, m);
  if (q == 0) {
    float v = p.D != nullptr ? __builtin_fmaf(p.D[ch], x, acc) : acc;
    if (p.z != nullptr) v *= silu(widen<F>(((const S*)p.z)[b * p.z_batch + ch]));
    ((S*)yv)[i] = narrow<F>(v);
  }
}

template <class F>
static hipError_t launch_step_f(const ScanProblem& p, const float* state, float* new_state,
                                void* y, hipStream_t stream) {
  constexpr int G = 16;
  const int64_t blocks = (p.batch * p.channels * G + 255) / 256;
  selective_scan_step_kernel<F, G><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(
      p, state, new_state, y);
  return hipGetLastError();
}

hipError_t launch_selective_scan_step(const ScanProblem& p, Fmt fmt, const float* state,
                                      float* new_state, void* y, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_step_f<FmtF32>(p, state, new_state, y, stream);
    case Fmt::F16: return launch_step_f<FmtF16>(p, state, new_state, y, stream);
    case Fmt::BF16: return launch_step_f<FmtBF16>(p, state, new_state, y, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sca
