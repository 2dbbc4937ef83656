// Gradient of the selective scan (selective_scan.hip has the forward).  With
// q = dy silu(z) and m[t] the gradient with respect to h[t - 1],
//   G[t] = C[t] q[t] + m[t + 1],   m[t] = a[t] G[t]     (a scan from the end),
//   dC[t] = sum_channels q h,      dB[t] = sum_channels G dt x,
//   dx = dt sum_n G B + D q,       ddt = x sum_n G B + sum_n A m h[t - 1],
//   dA = sum_t dt m h[t - 1],      dD = sum_t q x.
//
// A workgroup walks its sequence's blocks from the last to the first.  Each
// block starts from the states the forward kept, recomputes h forward and runs
// m backward, both as wave scans of affine maps (scan_tile.hpp).  Sums over
// states stay in a lane; dB and dC of the workgroup's 16 channels are added
// through LDS, one state at a time, and written as partial sums, which a second
// kernel adds over the workgroups in a fixed order (no atomics: the same bits
// every time).
#include "scan_tile.hpp"

namespace sca {

template <class F, int K> struct GradShape {
  static constexpr int NG = 8;            // states of B and C staged at a time
  static constexpr int TB = 64 * K;
};

// lane l's value from lane `from` of the wave
__device__ __forceinline__ float lane_from(float v, int from) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_ds_bpermute(from * 4, __builtin_bit_cast(int, v)));
}

template <class F, int K>
__global__ __launch_bounds__(kScanThreads) void selective_scan_grad_kernel(
    ScanProblem p, ScanGrads g, float* part, float* part_params, int64_t b0, int64_t tiles,
    uint32_t count) {
  using S = typename F::S;
  using Tile = TileStage<F, K>;
  constexpr int NG = GradShape<F, K>::NG, TB = GradShape<F, K>::TB;
  using Rows = RowStage<F, K, NG>;
  __shared__ alignas(16) float s_B[NG * TB], s_C[NG * TB], s_ex[kScanWaves * 2 * TB];
  __shared__ alignas(16) uint32_t s_x[Tile::WORDS], s_dt[Tile::WORDS], s_z[Tile::WORDS], s_dy[Tile::WORDS];

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
  const auto dys = tile_src<F>(g.dy, g.dy_batch, g.dy_token, at.b, at.ch);
  const auto Bs = tile_src<F>(p.B, p.B_batch, p.B_token, at.b, at.g * p.B_group);
  const auto Cs = tile_src<F>(p.C, p.C_batch, p.C_token, at.b, at.g * p.C_group);
  const int64_t out0 = at.b * p.length * p.channels + at.ch;
  S* dx = (S*)g.dx + out0;
  S* ddt = (S*)g.ddt + out0;
  S* dz = gate ? (S*)g.dz + out0 : nullptr;
  const bool whole = (p.channels * (int64_t)sizeof(S)) % 16 == 0;
  const bool xvec = whole && (uintptr_t)dx % 16 == 0, dtvec = whole && (uintptr_t)ddt % 16 == 0;
  const bool zvec = whole && (uintptr_t)dz % 16 == 0;

  // lane n of these registers holds state n of the wave's two channels
  float A2[2], m_carry[2], dA[2] = {0.0f, 0.0f}, Dc[2], bias[2];
  float dD[2] = {0.0f, 0.0f}, dbias[2] = {0.0f, 0.0f};
  bool live[2];
  int64_t row[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    live[c] = 2 * wave + c < at.nch;
    const int64_t ch = at.ch + 2 * wave + c;
    row[c] = (at.b * p.channels + ch) * N + lane;
    const bool on = live[c] && lane < N;
    A2[c] = on ? p.A[ch * N + lane] * kLog2e : 0.0f;
    m_carry[c] = on && g.dfinal != nullptr ? g.dfinal[row[c]] : 0.0f;
    Dc[c] = live[c] && p.D != nullptr ? p.D[ch] : 0.0f;
    bias[c] = live[c] && p.dt_bias != nullptr ? p.dt_bias[ch] : 0.0f;
  }

  const int64_t nblk = (p.length + TB - 1) / TB;
  const int64_t blocks = (len + TB - 1) / TB;
  const int64_t group = at.b * p.groups + at.g;
  for (int64_t blk = blocks - 1; blk >= 0; --blk) {
    const int64_t t0 = blk * TB;
    Rows rB, rC;
    {
      Tile rx, rdt, rz, rdy;
      rx.load(xs, t0, len, at.nch);
      rdt.load(dts, t0, len, at.nch);
      rdy.load(dys, t0, len, at.nch);
      if (gate) rz.load(zs, t0, len, at.nch);
      rB.load(Bs, t0, len, 0, N);
      rC.load(Cs, t0, len, 0, N);
      __syncthreads();                     // the last block's LDS is free
      rx.put(s_x);
      rdt.put(s_dt);
      rdy.put(s_dy);
      if (gate) rz.put(s_z);
      rB.put(s_B);
      rC.put(s_C);
    }
    float start[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t ch = at.ch + 2 * wave + c;
      start[c] = live[c] && lane < N
                     ? g.starts[((at.b * nblk + blk) * p.channels + ch) * N + lane]
                     : 0.0f;
    }
    __syncthreads();
    float dt[K][2], u[K][2], q[K][2], span[2];
    float gb[K][2] = {}, da[K][2] = {}, ysum[K][2] = {};
    Tile::get(s_dt, wave, lane, dt);
    Tile::get(s_x, wave, lane, u);
    Tile::get(s_dy, wave, lane, q);
    if (gate) {
      float zv[K][2];
      Tile::get(s_z, wave, lane, zv);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c) q[k][c] *= silu(zv[k][c]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float total = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float raw = dt[k][c] + bias[c];
        const float d = p.softplus ? softplus(raw) : raw;
        dt[k][c] = t0 + lane * K + k < len ? d : 0.0f;   // past the end: a = 1, b = 0
        total += dt[k][c];
        dD[c] = __builtin_fmaf(q[k][c], u[k][c], dD[c]);
        u[k][c] *= dt[k][c];
      }
      span[c] = total;
    }
    for (int n0 = 0; n0 < N; n0 += NG) {
      if (n0 > 0) {
        rB.put(s_B);
        rC.put(s_C);
        __syncthreads();
      }
      if (n0 + NG < N) {
        rB.load(Bs, t0, len, n0 + NG, N);
        rC.load(Cs, t0, len, n0 + NG, N);
      }
      const int nn = N - n0 < NG ? N - n0 : NG;
      for (int i = 0; i < nn; ++i) {
        const int n = n0 + i;
        float Bk[K], Ck[K], dBk[K], dCk[K];
        plane_read<K>(s_B + i * TB, lane, Bk);
        plane_read<K>(s_C + i * TB, lane, Ck);
        float a[2][K], h[2][K], P[2], H[2], h0[2], M[2], m0[2], An[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          An[c] = readlane(A2[c], n);
          float hl = 0.0f, ml = 0.0f;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            a[c][k] = exp2_hw(dt[k][c] * An[c]);
            h[c][k] = u[k][c] * Bk[k];
            hl = __builtin_fmaf(a[c][k], hl, h[c][k]);
          }
#pragma unroll
          for (int k = K - 1; k >= 0; --k) ml = a[c][k] * __builtin_fmaf(Ck[k], q[k][c], ml);
          P[c] = exp2_hw(span[c] * An[c]);
          h0[c] = readlane(start[c], n);
          m0[c] = readlane(m_carry[c], n);
          H[c] = __builtin_fmaf(P[c], lane == 0 ? h0[c] : 0.0f, hl);
          M[c] = __builtin_fmaf(P[c], lane == kWave - 1 ? m0[c] : 0.0f, ml);
        }
        // the backward scan runs over the lanes in reverse
        float R[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          M[c] = lane_from(M[c], kWave - 1 - lane);
          R[c] = lane_from(P[c], kWave - 1 - lane);
        }
        affine_scan2(H[0], H[1], P[0], P[1]);
        affine_scan2(M[0], M[1], R[0], R[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float hin = dpp<kWaveShr1, 0xf>(H[c], h0[c]);
          const float last = readlane(M[c], kWave - 1);
          m_carry[c] = lane == n ? last : m_carry[c];
          const float back = lane_from(M[c], kWave - 2 - lane);
          float m = lane == kWave - 1 ? m0[c] : back;
          float hk = hin;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            hk = __builtin_fmaf(a[c][k], hk, h[c][k]);
            h[c][k] = hk;
            const float dC = q[k][c] * hk;
            dCk[k] = c == 0 ? dC : dCk[k] + dC;
            ysum[k][c] = __builtin_fmaf(Ck[k], hk, ysum[k][c]);
          }
          float dAl = 0.0f;
#pragma unroll
          for (int k = K - 1; k >= 0; --k) {
            const float G = __builtin_fmaf(Ck[k], q[k][c], m);
            m = a[c][k] * G;
            const float dB = G * u[k][c];
            dBk[k] = c == 0 ? dB : dBk[k] + dB;
            gb[k][c] = __builtin_fmaf(G, Bk[k], gb[k][c]);
            const float w = m * (k > 0 ? h[c][k > 0 ? k - 1 : 0] : hin);
            da[k][c] = __builtin_fmaf(w, An[c], da[k][c]);
            dAl = __builtin_fmaf(w, dt[k][c], dAl);
          }
          const float dAn = wave_sum(dAl);
          dA[c] += lane == n ? dAn : 0.0f;
        }
        plane_write<K>(s_ex + (wave * 2 + 0) * TB, lane, dBk);
        plane_write<K>(s_ex + (wave * 2 + 1) * TB, lane, dCk);
        __syncthreads();
        float* to = part + (((group * tiles + at.tile) * nblk + blk) * N + n) * (2 * TB);
        for (int j = threadIdx.x; j < 2 * TB; j += kScanThreads) {
          float v = s_ex[j];
#pragma unroll
          for (int w = 1; w < kScanWaves; ++w) v += s_ex[w * 2 * TB + j];
          to[j] = v;
        }
        __syncthreads();
      }
    }
    // the block's outputs, through the waves' own planes
    float xv[K][2], out[K][2];
    Tile::get(s_x, wave, lane, xv);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) out[k][c] = __builtin_fmaf(gb[k][c], dt[k][c], Dc[c] * q[k][c]);
    Tile::set(s_x, wave, lane, out);
    Tile::get(s_dt, wave, lane, out);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float raw = out[k][c] + bias[c];
        float v = __builtin_fmaf(gb[k][c], xv[k][c], da[k][c] * kLn2);
        if (p.softplus) v *= sigmoid(raw);
        v = t0 + lane * K + k < len ? v : 0.0f;
        dbias[c] += v;
        out[k][c] = v;
      }
    Tile::set(s_dt, wave, lane, out);
    if (gate) {
      float zv[K][2];
      Tile::get(s_z, wave, lane, zv);
      Tile::get(s_dy, wave, lane, out);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          out[k][c] *= __builtin_fmaf(Dc[c], xv[k][c], ysum[k][c]) * silu_slope(zv[k][c]);
      Tile::set(s_z, wave, lane, out);
    }
    __syncthreads();
    Tile::store(s_x, dx, p.channels, xvec, t0, len, at.nch);
    Tile::store(s_dt, ddt, p.channels, dtvec, t0, len, at.nch);
    if (gate) Tile::store(s_z, dz, p.channels, zvec, t0, len, at.nch);
  }
  // tokens past the sequence's end
  for (int64_t i = len * kScanTile + threadIdx.x; i < p.length * kScanTile; i += kScanThreads)
    if (i % kScanTile < at.nch) {
      const int64_t o = (i / kScanTile) * p.channels + i % kScanTile;
      dx[o] = S(0);
      ddt[o] = S(0);
      if (gate) dz[o] = S(0);
    }
  // sums over this sequence: [batch][channels * states | channels | channels]
  float* params = part_params + at.b * p.channels * (N + 2);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int64_t ch = at.ch + 2 * wave + c;
    const float sD = wave_sum(dD[c]), sb = wave_sum(dbias[c]);
    if (!live[c]) continue;
    if (lane < N) {
      params[ch * N + lane] = dA[c];
      if (g.dinitial != nullptr) g.dinitial[row[c]] = m_carry[c];
    }
    if (lane == 0) {
      params[p.channels * N + ch] = sD;
      params[p.channels * (N + 1) + ch] = sb;
    }
  }
}

// dB and dC: the sums over the workgroups of a group's channels, 64 tokens of
// one array per workgroup, turned from one state per plane to one token per row.
template <class F, int K>
__global__ __launch_bounds__(256) void scan_rows_sum_kernel(ScanProblem p, const float* part,
                                                           void* dBv, void* dCv, int64_t tiles) {
  using S = typename F::S;
  constexpr int TB = 64 * K;
  __shared__ alignas(16) float s_v[64 * 65];
  const int lane = lane_id(), wave = wave_id();
  const int N = (int)p.states;
  const int64_t nblk = (p.length + TB - 1) / TB;
  const int64_t total = p.batch * p.groups * nblk * K * 2;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int arr = (int)(w % 2), seg = (int)(w / 2 % K);
    const int64_t blk = w / (2 * K) % nblk, group = w / (2 * K) / nblk;
    const int64_t b = group / p.groups, gi = group % p.groups;
    const bool any = blk * TB < scan_length(p, b);
    for (int n = wave; n < N; n += 4) {
      float v = 0.0f;
      if (any) {
        const float* src = part + ((group * tiles * nblk + blk) * N + n) * (2 * TB) + arr * TB +
                           seg * 64 + lane;
        const int64_t step = nblk * N * (2 * TB);
#pragma unroll 4
        for (int64_t t = 0; t < tiles; ++t) v += src[t * step];
      }
      s_v[lane * 65 + n] = v;
    }
    __syncthreads();
    S* out = (S*)(arr == 0 ? dBv : dCv);
    for (int i = threadIdx.x; i < 64 * N; i += 256) {
      const int l = i / N, n = i % N;
      const int64_t t = blk * TB + plane_token<K>(seg * 64 + l);
      if (t < p.length)
        out[((b * p.length + t) * p.groups + gi) * N + n] = narrow<F>(s_v[l * 65 + n]);
    }
    __syncthreads();
  }
}

// dA, dD and ddt_bias: sums over the batch, in order.
__global__ __launch_bounds__(256) void scan_params_sum_kernel(const float* part, int64_t batch,
                                                             int64_t channels, int64_t states,
                                                             float* dA, float* dD, float* dbias) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, count = channels * (states + 2);
  if (i >= count) return;
  float v = 0.0f;
  for (int64_t b = 0; b < batch; ++b) v += part[b * count + i];
  if (i < channels * states) {
    dA[i] = v;
  } else if (i < channels * (states + 1)) {
    if (dD != nullptr) dD[i - channels * states] = v;
  } else if (dbias != nullptr) {
    dbias[i - channels * (states + 1)] = v;
  }
}

namespace {
int64_t grad_tiles(const ScanProblem& p) {
  return (p.channels / p.groups + kScanTile - 1) / kScanTile;
}
size_t rows_part_floats(const ScanProblem& p, Fmt fmt) {
  const int64_t tb = scan_block_tokens(p.length, fmt);
  const int64_t nblk = (p.length + tb - 1) / tb;
  return (size_t)(p.batch * p.groups * grad_tiles(p) * nblk * p.states * 2 * tb);
}
}  // namespace

size_t selective_scan_grad_scratch(const ScanProblem& p, Fmt fmt) {
  return 4 * (rows_part_floats(p, fmt) + (size_t)(p.batch * p.channels * (p.states + 2)));
}

constexpr int64_t kMaxGroups = 1ll << 22;   // workgroups per launch

template <class F, int K>
static hipError_t launch_grad(const ScanProblem& p, Fmt fmt, const ScanGrads& g, void* scratch,
                              hipStream_t stream) {
  const int64_t tiles = grad_tiles(p);
  const int64_t per = tiles * p.groups;
  const int64_t step = kMaxGroups / per < 1 ? 1 : kMaxGroups / per;
  float* part = (float*)scratch;
  float* params = part + rows_part_floats(p, fmt);
  for (int64_t b0 = 0; b0 < p.batch; b0 += step) {
    const int64_t nb = p.batch - b0 < step ? p.batch - b0 : step;
    selective_scan_grad_kernel<F, K><<<dim3(xcd_grid(nb * per)), dim3(kScanThreads), 0, stream>>>(
        p, g, part, params, b0, tiles, (uint32_t)(nb * per));
  }
  constexpr int TB = 64 * K;
  const int64_t nblk = (p.length + TB - 1) / TB;
  const int64_t sums = p.batch * p.groups * nblk * K * 2;
  if (sums > 0)
    scan_rows_sum_kernel<F, K><<<dim3((unsigned)(sums < (1 << 20) ? sums : 1 << 20)), dim3(256), 0,
                                 stream>>>(p, part, g.dB, g.dC, tiles);
  const int64_t count = p.channels * (p.states + 2);
  scan_params_sum_kernel<<<dim3((unsigned)((count + 255) / 256)), dim3(256), 0, stream>>>(
      params, p.batch, p.channels, p.states, g.dA, g.dD, g.ddt_bias);
  return hipGetLastError();
}

template <class F>
static hipError_t launch_grad_f(const ScanProblem& p, Fmt fmt, const ScanGrads& g, void* scratch,
                                hipStream_t stream) {
  switch (scan_block_tokens(p.length, fmt) / 64) {
    case 1: return launch_grad<F, 1>(p, fmt, g, scratch, stream);
    case 2: return launch_grad<F, 2>(p, fmt, g, scratch, stream);
    case 4: return launch_grad<F, 4>(p, fmt, g, scratch, stream);
    case 8:
      if constexpr (sizeof(typename F::S) == 2) return launch_grad<F, 8>(p, fmt, g, scratch, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_selective_scan_grad(const ScanProblem& p, Fmt fmt, const ScanGrads& g,
                                      void* scratch, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_grad_f<FmtF32>(p, fmt, g, scratch, stream);
    case Fmt::F16: return launch_grad_f<FmtF16>(p, fmt, g, scratch, stream);
    case Fmt::BF16: return launch_grad_f<FmtBF16>(p, fmt, g, scratch, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sca
