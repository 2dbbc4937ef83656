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
                                                                     int64_t tiles,
                                                                     uint32_t count) {
  using S = typename F::S;
  using Tile = TileStage<F, K>;
  using Rows = RowStage<F, K, NG>;
  constexpr int TB = 64 * K;
  __shared__ alignas(16) float s_B[NG * TB], s_C[NG * TB];
  __shared__ alignas(16) uint32_t s_x[Tile::WORDS], s_dt[Tile::WORDS], s_z[Tile::WORDS];

  const int lane = lane_id(), wave = wave_id();
  const uint32_t id = xcd_order(blockIdx.x);
  if (id >= count) return;
  const ScanPlace at = scan_place(p, b0, tiles, id);
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
        <<<dim3(xcd_grid(nb * per)), dim3(kScanThreads), 0, stream>>>(
            p, y, final_state, starts, b0, tiles, (uint32_t)(nb * per));
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
// One token.  Bound by the state: 8 bytes per state and sequence against some
// six operations.  G lanes (a power of two) share a channel, lane q of them
// owning the V states at q V, (q + G) V, ...; V = 4 makes the state's loads and
// stores 16 bytes wide and a wave's contiguous.  A lane takes R sequences of
// its channel at once: A, D and the bias are read once for them and R loads of
// the state are in flight.
// ---------------------------------------------------------------------------
template <class F, int V, int G, int R>
__global__ __launch_bounds__(256) void selective_scan_step_kernel(ScanProblem p,
                                                                 const float* state,
                                                                 float* new_state, void* yv,
                                                                 int64_t first) {
  using S = typename F::S;
  using IO = RowIO<FmtF32, V>;
  using BIO = RowIO<F, V>;
  const uint32_t per = (uint32_t)p.channels * G;        // lanes of one sequence
  const uint32_t cols = (per + 255) / 256;
  const uint32_t at = blockIdx.x % cols * 256 + threadIdx.x;
  const int64_t b0 = first + (int64_t)(blockIdx.x / cols) * R;
  if (at >= per) return;                                // whole groups of G lanes leave together
  const int64_t ch = at / G;
  const int q = at % G, N = (int)p.states;
  const int64_t g = p.groups == 1 ? 0 : (int64_t)((uint32_t)ch / (uint32_t)(p.channels / p.groups));
  const float bias = p.dt_bias != nullptr ? p.dt_bias[ch] : 0.0f;
  float x[R], dt[R], z[R], acc[R];
  bool on[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t b = b0 + r;
    on[r] = b < p.batch;
    x[r] = on[r] ? widen<F>(((const S*)p.x)[b * p.x_batch + ch]) : 0.0f;
    dt[r] = on[r] ? widen<F>(((const S*)p.dt)[b * p.dt_batch + ch]) : 0.0f;
    z[r] = on[r] && p.z != nullptr ? widen<F>(((const S*)p.z)[b * p.z_batch + ch]) : 0.0f;
    acc[r] = 0.0f;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    dt[r] += bias;
    if (p.softplus) dt[r] = softplus(dt[r]);
  }
  for (int n = q * V; n < N; n += G * V) {
    float A[V];
    IO::unpack(IO::load(p.A + ch * N + n, V, V > 1), A);
    typename IO::Raw h0[R];
    typename BIO::Raw Bn[R], Cn[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t b = b0 + r;
      h0[r] = typename IO::Raw{};
      Bn[r] = Cn[r] = typename BIO::Raw{};
      if (!on[r]) continue;
      h0[r] = IO::load(state + (b * p.channels + ch) * N + n, V, V > 1);
      Bn[r] = BIO::load((const S*)p.B + b * p.B_batch + g * p.B_group + n, V, V > 1);
      Cn[r] = BIO::load((const S*)p.C + b * p.C_batch + g * p.C_group + n, V, V > 1);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] *= kLog2e;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float h[V], Bv[V], Cv[V];
      IO::unpack(h0[r], h);
      BIO::unpack(Bn[r], Bv);
      BIO::unpack(Cn[r], Cv);
      const float u = dt[r] * x[r];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = __builtin_fmaf(exp2_hw(dt[r] * A[v]), h[v], u * Bv[v]);
        acc[r] = __builtin_fmaf(h[v], Cv[v], acc[r]);
      }
      if (on[r])
        IO::store(new_state + ((b0 + r) * p.channels + ch) * N + n, IO::pack(h), V, V > 1);
    }
  }
  const float D = p.D != nullptr ? p.D[ch] : 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float a = acc[r];
#pragma unroll
    for (int m = G / 2; m > 0; m /= 2) a += __shfl_xor(a, m);
    if (p.D != nullptr) a = __builtin_fmaf(D, x[r], a);
    if (p.z != nullptr) a *= silu(z[r]);
    if (q == 0 && on[r]) ((S*)yv)[(b0 + r) * p.channels + ch] = narrow<F>(a);
  }
}

template <class F, int V, int G>
static hipError_t launch_step_g(const ScanProblem& p, const float* state, float* new_state,
                                void* y, hipStream_t stream) {
  const int64_t cols = (p.channels * G + 255) / 256;
  // several sequences a lane once that still leaves 2048 workgroups, 8 waves a SIMD
  constexpr int R = 4;
  const bool many = p.batch * cols >= 2048 * R;
  const int64_t step = kMaxGroups / cols < 1 ? 1 : kMaxGroups / cols;
  for (int64_t b0 = 0; b0 < p.batch; b0 += step) {
    const int64_t nb = p.batch - b0 < step ? p.batch - b0 : step;
    if (many) {
      selective_scan_step_kernel<F, V, G, R><<<dim3((unsigned)((nb + R - 1) / R * cols)), dim3(256), 0,
                                               stream>>>(p, state, new_state, y, b0);
    } else {
      selective_scan_step_kernel<F, V, G, 1><<<dim3((unsigned)(nb * cols)), dim3(256), 0, stream>>>(
          p, state, new_state, y, b0);
    }
  }
  return hipGetLastError();
}

template <class F>
static hipError_t launch_step_f(const ScanProblem& p, const float* state, float* new_state,
                                void* y, hipStream_t stream) {
  using S = typename F::S;
  const int64_t bc = 4 * (int64_t)sizeof(S);            // bytes of four states of B or C
  auto rows4 = [&](const void* a, int64_t batch, int64_t group) {
    return (uintptr_t)a % bc == 0 && batch % 4 == 0 && group % 4 == 0;
  };
  const bool vec = p.states % 4 == 0 && (uintptr_t)state % 16 == 0 &&
                   (uintptr_t)new_state % 16 == 0 && (uintptr_t)p.A % 16 == 0 &&
                   rows4(p.B, p.B_batch, p.B_group) && rows4(p.C, p.C_batch, p.C_group);
  if (!vec) return launch_step_g<F, 1, 16>(p, state, new_state, y, stream);
  if (p.states <= 8) return launch_step_g<F, 4, 2>(p, state, new_state, y, stream);
  return launch_step_g<F, 4, 4>(p, state, new_state, y, stream);
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
