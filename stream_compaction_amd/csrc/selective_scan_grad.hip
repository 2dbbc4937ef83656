// Gradient of the selective scan (selective_scan.hip has the forward).  With
// q = dy silu(z) and m[t] the gradient with respect to h[t - 1],
//   G[t] = C[t] q[t] + m[t + 1],   m[t] = a[t] G[t]     (from the last token),
//   dC[t] = sum_channels q h,      dB[t] = sum_channels G dt x,
//   dx = dt sum_n G B + D q,       ddt = x sum_n G B + sum_n A m h[t - 1],
//   dA = sum_t dt m h[t - 1],      dD = sum_t q x.
//
// A workgroup walks its sequence in blocks of 16 tokens from the last to the
// first.  A block's states are computed again from the one that the forward
// kept before it, and stay in registers with the decays (16 of each per lane);
// then m goes backward over them.  Bound by vector instructions: 12 products and
// sums per token and state, and 8 to 9 for the sums over 16 states (dx, ddt, dz)
// and 16 channels (dB, dC).  dB and dC of the workgroup's channels go out as
// partial sums, which a second kernel adds over the workgroups in a fixed order
// (no atomics: the same bits every time).
//
// Measured (traced), bf16, 16 states, 4 x 2048 x 2048 with gate: 284 us, and 12 + 5
// us for the two kernels of partial sums (67 MB); two waves per SIMD, vector units
// 82% busy, 28 instructions per token and state.  One tile of channels per workgroup
// instead of two takes 5% longer for twice the partial sums.
#include "scan_tile.hpp"

namespace sca {

namespace {

constexpr int kT = kKeep;               // tokens per block
constexpr int kPS = kT + 4;             // stride of planes of one value per token
constexpr int kPlane = kScanTile * kPS;

// Sums over the 16 lanes of a row of 16 values: lane l gets value l.  A lane adds
// its partner's share of the values it keeps: 8, then 4 lanes apart by additions
// that write one half of the lanes, closer by selects.  Instructions between a
// write and the DPP read of the same register: at least two throughout.  The
// first eight values are written before the others are read: early clobbers.
__device__ __forceinline__ float lanes_sum(float (&v)[16], int l) {
#define SCA_FAR(A, B)                                                          \
  "v_add_f32_dpp " A ", " A ", " A " row_ror:8 row_mask:0xf bank_mask:0x3\n\t"   \
  "v_add_f32_dpp " A ", " B ", " B " row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
#define SCA_NEAR(A, B)                                                         \
  "v_add_f32_dpp " A ", " A ", " A " row_ror:12 row_mask:0xf bank_mask:0x5\n\t"  \
  "v_add_f32_dpp " A ", " B ", " B " row_ror:4 row_mask:0xf bank_mask:0xa\n\t"
  asm("s_nop 1\n\t"
      SCA_FAR("%0", "%8") SCA_FAR("%1", "%9") SCA_FAR("%2", "%10") SCA_FAR("%3", "%11")
      SCA_FAR("%4", "%12") SCA_FAR("%5", "%13") SCA_FAR("%6", "%14") SCA_FAR("%7", "%15")
      SCA_NEAR("%0", "%4") SCA_NEAR("%1", "%5") SCA_NEAR("%2", "%6") SCA_NEAR("%3", "%7")
      "s_nop 1"
      : "+&v"(v[0]), "+&v"(v[1]), "+&v"(v[2]), "+&v"(v[3]), "+&v"(v[4]), "+&v"(v[5]),
        "+&v"(v[6]), "+&v"(v[7])
      : "v"(v[8]), "v"(v[9]), "v"(v[10]), "v"(v[11]), "v"(v[12]), "v"(v[13]), "v"(v[14]), "v"(v[15]));
#undef SCA_FAR
#undef SCA_NEAR
  const bool b1 = (l & 2) != 0, b0 = (l & 1) != 0;
  float s[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float keep = b1 ? v[t + 2] : v[t], give = b1 ? v[t] : v[t + 2];
    s[t] = keep + dpp<0x4e, 0xf>(give, 0.0f);          // quad_perm [2, 3, 0, 1]
  }
  const float keep = b0 ? s[1] : s[0], give = b0 ? s[0] : s[1];
  return keep + dpp<0xb1, 0xf>(give, 0.0f);            // quad_perm [1, 0, 3, 2]
}

}  // namespace

// TL tiles of 16 channels, four waves each.  ENDS: only find m before each chunk
// of a split scan (but the first) from zero after it, and the sum of its steps.
template <class F, int NS, bool GATE, int TL, bool ALL, bool ENDS>
__global__ __launch_bounds__(256 * TL) void selective_scan_grad_kernel(
    ScanProblem p, ScanGrads g, float* part, float* part_params, ScanSplit split, int64_t b0,
    int64_t tiles, uint32_t count) {
  using S = typename F::S;
  typedef float vec4 __attribute__((ext_vector_type(4)));
  constexpr int RL = 2 / TL;            // rows of B and C that a thread stages
  constexpr int SUMS = GATE ? 3 : 2;
  __shared__ alignas(16) float s_x[2][TL][3 * kPlane];            // steps, steps times x, q
  __shared__ alignas(16) float s_bc[2][2][NS * kPlane];           // B, C
  __shared__ alignas(16) float s_sum[2][TL][SUMS][4 * kPlane];    // over a wave's states
  __shared__ alignas(16) float s_dbc[2][TL][2][NS * 16 * kT];     // over a tile's channels
  __shared__ alignas(16) float s_none[ALL ? 1 : kT];     // u and q of states that do not exist

  const uint32_t id = xcd_order(blockIdx.x);
  if (id >= count) return;
  // chunk by chunk; a chunk is worked on like a sequence that begins at `first`
  const uint32_t per = ENDS ? count / (split.chunks - 1) : count / split.chunks;
  const int64_t chunk = id / per + (ENDS ? 1 : 0), first = chunk * split.tokens;
  const ScanPlace at = scan_place(p, b0, tiles, id % per, kScanTile * TL);
  auto within = [&](int64_t n) {
    return n <= first ? 0 : (n - first < split.tokens ? n - first : split.tokens);
  };
  const int64_t len = within(scan_length(p, at.b)), padded = within(p.length);
  const int N = (int)p.states;
  const int tid = (int)threadIdx.x, lane = lane_id(), wave = wave_id();
  const int tl = wave / 4, row = lane / 16, cl = lane % 16;
  const int n0 = wave % 4 * 4 + row;            // this lane's states: n0, n0 + 16, ...
  // channels of this wave's tile (none for a tile past the group's last channel)
  const int nch = (int)at.nch - tl * kScanTile < kScanTile ? (int)at.nch - tl * kScanTile : kScanTile;
  const int64_t tch = at.ch + tl * kScanTile, ch = tch + cl;

  // staging: this thread's token and channel, and its token and state of each 16
  const int tok = tid % 256 / 16, c = tid % 16;
  const bool on = c < nch;
  const int64_t cch = on ? tch + c : at.ch;     // a channel that exists
  struct Src {
    const S *base, *p;
    int64_t token;
  };
  auto source = [&](const void* a, int64_t batch, int64_t token, int64_t off) {
    Src s;
    s.base = s.p = (const S*)a + at.b * batch + first * token + off;
    s.token = token;
    return s;
  };
  Src xs = source(p.x, p.x_batch, p.x_token, cch), dts = source(p.dt, p.dt_batch, p.dt_token, cch);
  Src dys = source(g.dy, g.dy_batch, g.dy_token, cch);
  Src zs = GATE ? source(p.z, p.z_batch, p.z_token, cch) : xs;
  Src rows[RL][NS];
#pragma unroll
  for (int r = 0; r < RL; ++r)
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int n = s * 16 + c < N ? s * 16 + c : 0;
      rows[r][s] = r + tl == 0 ? source(p.B, p.B_batch, p.B_token, at.g * p.B_group + n)
                               : source(p.C, p.C_batch, p.C_token, at.g * p.C_group + n);
    }
  const float Dc = on && p.D != nullptr ? p.D[cch] : 0.0f;
  const float bias = on && p.dt_bias != nullptr ? p.dt_bias[cch] : 0.0f;
  float dD = 0.0f, dbias = 0.0f;

  float A2[NS], m[NS], dA[NS] = {};
  bool mine[NS];
  const int64_t srow = (at.b * p.channels + ch) * N;
  const float* kept[NS];                        // of the block before the one last fetched
  const int64_t nkeep = (p.length + kKeep - 1) / kKeep;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int n = n0 + s * 16;
    mine[s] = cl < nch && n < N;
    A2[s] = mine[s] ? p.A[ch * N + n] * kLog2e : kNoState;
    m[s] = !ENDS && mine[s] && g.dfinal != nullptr ? g.dfinal[srow + n] : 0.0f;
    const int64_t from = (at.b * nkeep + first / kKeep) * p.channels + (mine[s] ? ch : at.ch);
    kept[s] = g.starts + from * N + (mine[s] ? n : 0);
  }

  if (!ALL && tid < kT) s_none[tid] = 0.0f;

  float span = 0.0f;                            // ENDS: sum of the channel's steps
  if constexpr (!ENDS) {
    // m after the chunk, from the chunks after it (eight loads at a time)
#pragma unroll 8
    for (int64_t c = split.chunks - 1; c > chunk; --c) {
      const int64_t r = (at.b * split.chunks + c) * p.channels + (cl < nch ? ch : at.ch);
      const float passed = split.spans[r];
#pragma unroll
      for (int s = 0; s < NS; ++s)
        m[s] = carried(passed * A2[s], m[s]) + (mine[s] ? split.ends[r * N + n0 + s * 16] : 0.0f);
    }
  }

  struct Fetched { S x, dt, dy, z, rows[RL][NS]; float h[NS]; } f;
  auto each = [&](auto&& fn) {
    fn(xs);
    fn(dts);
    fn(dys);
    fn(zs);
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
      for (int s = 0; s < NS; ++s) fn(rows[r][s]);
  };
  auto seek = [&](int64_t blk) {                // the last token that exists at the latest
    const int64_t t = blk * kT + tok;
    each([&](Src& s) { s.p = s.base + (t < len ? t : len - 1) * s.token; });
  };
  auto fetch = [&](int64_t blk) {
    f.x = *gptr<const S>((uintptr_t)xs.p);
    f.dt = *gptr<const S>((uintptr_t)dts.p);
    f.dy = *gptr<const S>((uintptr_t)dys.p);
    f.z = *gptr<const S>((uintptr_t)zs.p);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
      for (int r = 0; r < RL; ++r) f.rows[r][s] = *gptr<const S>((uintptr_t)rows[r][s].p);
      if constexpr (!ENDS) f.h[s] = kept[s][blk * p.channels * N];
    }
  };

  // what a block's outputs need beside the sums
  struct Rest { float x, dt, skip, slope, gate; };
  auto stage = [&](int64_t t, int buf, Rest& rest, float (&start)[NS]) {
    // past either end of the sequence, and in channels past the last: a = 1, b = 0
    const bool token = t >= 0 && t < len, exists = token && on;
    const float x = widen<F>(f.x), raw = widen<F>(f.dt) + bias, dy = widen<F>(f.dy);
    const float soft = softplus(raw), sig = sigmoid(raw);
    float d = p.softplus ? soft : raw;
    d = exists ? d : 0.0f;
    float q = dy;
    if constexpr (GATE) {
      const float z = widen<F>(f.z);
      q = dy * silu(z);
      rest.gate = dy * silu_slope(z);
    }
    q = exists ? q : 0.0f;
    const float u = exists ? d * x : 0.0f;
    float* to = s_x[buf][tl] + c * kPS + tok;
    to[0] = d;
    to[kPlane] = u;
    to[2 * kPlane] = q;
    rest.x = x;
    rest.dt = d;
    rest.skip = Dc * q;
    rest.slope = p.softplus ? sig : 1.0f;
    dD += exists ? q * x : 0.0f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const bool real = token && s * 16 + c < N;
#pragma unroll
      for (int r = 0; r < RL; ++r)
        s_bc[buf][r + tl][(s * 16 + c) * kPS + tok] = real ? widen<F>(f.rows[r][s]) : 0.0f;
      if constexpr (!ENDS) start[s] = mine[s] ? f.h[s] : 0.0f;
    }
  };

  auto walk = [&](int buf, const float (&start)[NS]) {
    const float* xp = s_x[buf][tl] + cl * kPS;
    float dt[16], u[16], q[16], vG[16], vA[16], vY[16];
#pragma unroll
    for (int t = 0; t < 16; t += 4) {
      const vec4 a = *(const vec4*)(xp + t);
#pragma unroll
      for (int i = 0; i < 4; ++i) dt[t + i] = a[i];
    }
    // u and q as state s of this lane takes them
    auto take = [&](int s) {
      if (s > 0 && ALL) return;
      const float* up = ALL || mine[s] ? xp + kPlane : s_none;
      const float* qp = ALL || mine[s] ? xp + 2 * kPlane : s_none;
#pragma unroll
      for (int t = 0; t < 16; t += 4) {
        const vec4 b = *(const vec4*)(up + t), e = *(const vec4*)(qp + t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[t + i] = b[i];
          q[t + i] = e[i];
        }
      }
    };
    if constexpr (ENDS) {
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 16; ++t) sum += dt[t];
      span += sum;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const float C = s_bc[buf][1][(s * 16 + n0) * kPS + cl];
        take(s);
        for_tokens([&](auto tc) {
          constexpr int t = 15 - decltype(tc)::value;
          m[s] = exp2_hw(dt[t] * A2[s]) * __builtin_fmaf(row_bcast<t>(C), q[t], m[s]);
        }, std::make_integer_sequence<int, 16>{});
      }
      return;
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int bc = (s * 16 + n0) * kPS + cl;
      const float B = s_bc[buf][0][bc], C = s_bc[buf][1][bc];
      take(s);
      float a[16], h[16], v[16], now = start[s];
      for_tokens([&](auto tc) {
        constexpr int t = decltype(tc)::value;
        a[t] = exp2_hw(dt[t] * A2[s]);
        now = __builtin_fmaf(a[t], now, row_bcast<t>(B) * u[t]);
        h[t] = now;
        v[t] = q[t] * now;
        if constexpr (GATE) {
          // (the asm keeps a product beside its broadcast, which else does not fold)
          if (s == 0) {
            vY[t] = row_bcast<t>(C) * now;
          } else {
            vY[t] = __builtin_fmaf(row_bcast<t>(C), now, vY[t]);
          }
          asm volatile("" : "+v"(vY[t]));
        }
      }, std::make_integer_sequence<int, 16>{});
      float* out = s_dbc[buf][tl][0] + (s * 16 + n0) * kT + cl;
      out[NS * 16 * kT] = lanes_sum(v, cl);
      // other registers to the compiler: broadcasts shared by two products do not fold
      float Bb = B, Cb = C;
      asm volatile("" : "+v"(Bb), "+v"(Cb));
      float dAb = 0.0f;                         // of the block: shorter chains of additions
      for_tokens([&](auto tc) {
        constexpr int t = 15 - decltype(tc)::value;
        float G = __builtin_fmaf(row_bcast<t>(Cb), q[t], m[s]);
        asm volatile("" : "+v"(G));
        v[t] = G * u[t];
        if (s == 0) {
          vG[t] = row_bcast<t>(Bb) * G;
        } else {
          vG[t] = __builtin_fmaf(row_bcast<t>(Bb), G, vG[t]);
        }
        asm volatile("" : "+v"(vG[t]));
        m[s] = a[t] * G;
        const float w = m[s] * (t > 0 ? h[t > 0 ? t - 1 : 0] : start[s]);
        vA[t] = s == 0 ? w * A2[s] : __builtin_fmaf(w, A2[s], vA[t]);
        dAb = __builtin_fmaf(w, dt[t], dAb);
      }, std::make_integer_sequence<int, 16>{});
      dA[s] += dAb;
      out[0] = lanes_sum(v, cl);
    }
    const int to = (wave % 4 * 16 + cl) * kPS + row * 4;
    auto put = [&](int k, const float (&v)[16]) {
      float sums[4];
      rows_sum(v, sums);
      *(vec4*)(s_sum[buf][tl][k] + to) = vec4{sums[0], sums[1], sums[2], sums[3]};
    };
    put(0, vG);
    put(1, vA);
    if constexpr (GATE) put(SUMS - 1, vY);
  };

  const int64_t out0 = (at.b * p.length + first) * p.channels + tch + c;
  const int64_t group = at.b * p.groups + at.g;
  float* part0 = part + ((group * tiles + at.tile) * p.length + first) * (2 * N);
  auto finish = [&](const Rest& rest, int64_t blk, int buf) {
    const int64_t t = blk * kT + tok;
    auto total = [&](int k) {
      const float* from = s_sum[buf][tl][k] + c * kPS + tok;
      return (from[0] + from[kPlane]) + (from[2 * kPlane] + from[3 * kPlane]);
    };
    const float gb = total(0), da = total(1);
    const float ddt = __builtin_fmaf(gb, rest.x, da * kLn2) * rest.slope;
    if (t < len) {
      dbias += ddt;
      const int64_t o = out0 + t * p.channels;
      if (on) {
        ((S*)g.dx)[o] = narrow<F>(__builtin_fmaf(gb, rest.dt, rest.skip));
        ((S*)g.ddt)[o] = narrow<F>(ddt);
        if constexpr (GATE)
          ((S*)g.dz)[o] = narrow<F>(rest.gate * __builtin_fmaf(Dc, rest.x, total(SUMS - 1)));
      }
    }
    // this workgroup's part of dB and dC, [token][2][states]
#pragma unroll
    for (int k = 0; k < 2 * NS; k += TL) {
      const int j = k + tl, arr = j / NS, n = j % NS * 16 + c;
      if (t >= len || n >= N) continue;
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < TL; ++i) v += s_dbc[buf][i][arr][n * kT + tok];
      part0[t * (2 * N) + arr * N + n] = v;
    }
  };

  const int64_t blocks = (len + kT - 1) / kT;
  Rest rest[2];
  float start[2][NS];
  auto back = [&](int64_t blk) {                // from block blk to blk - 1, all of it exists
    if (blk > 0) each([&](Src& s) { s.p -= kT * s.token; });
  };
  // block blk is staged in buffer `buf`, the block before it in f
  auto step = [&](int64_t blk, int buf) {
    stage((blk - 1) * kT + tok, buf ^ 1, rest[buf ^ 1], start[buf ^ 1]);
    back(blk - 1);
    fetch(blk > 2 ? blk - 2 : 0);
    walk(buf, start[buf]);
    lds_barrier();
    if constexpr (!ENDS) finish(rest[buf], blk, buf);
  };
  if (blocks > 0) {
    seek(blocks - 1);
    fetch(blocks - 1);
    stage((blocks - 1) * kT + tok, 0, rest[0], start[0]);
    if (blocks > 1) seek(blocks - 2);
    fetch(blocks > 1 ? blocks - 2 : 0);
    lds_barrier();
    for (int64_t blk = blocks - 1; blk >= 0; blk -= 2) {
      step(blk, 0);
      if (blk == 0) break;
      step(blk - 1, 1);
    }
  }
  if constexpr (ENDS) {
    const int64_t r = (at.b * split.chunks + chunk) * p.channels + ch;
    if (wave == 0 && row == 0 && cl < nch) split.spans[r] = span;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (mine[s]) split.ends[r * N + n0 + s * 16] = m[s];
    return;
  }
  // tokens past the sequence's end
  const int width = kScanTile * TL;
  for (int64_t i = len * width + tid; i < padded * width; i += 256 * TL)
    if (i % width < at.nch) {
      const int64_t o = (at.b * p.length + first + i / width) * p.channels + at.ch + i % width;
      ((S*)g.dx)[o] = S(0);
      ((S*)g.ddt)[o] = S(0);
      if constexpr (GATE) ((S*)g.dz)[o] = S(0);
    }
  // sums over this chunk: [batch][chunks][channels * states | channels | channels]
  float* params = part_params + (at.b * split.chunks + chunk) * p.channels * (N + 2);
  __syncthreads();
  float* sums = &s_sum[0][0][0][0];
  sums[tid] = dD;
  sums[256 * TL + tid] = dbias;
  __syncthreads();
  if (tid < 2 * width) {
    const int k = tid / width, j = tid % width;
    float v = 0.0f;
#pragma unroll
    for (int t = 0; t < kT; ++t) v += sums[k * 256 * TL + j / 16 * 256 + t * 16 + j % 16];
    if (j < at.nch) params[p.channels * (N + k) + at.ch + j] = v;
  }
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (mine[s]) {
      params[ch * N + n0 + s * 16] = dA[s];
      if (g.dinitial != nullptr && chunk == 0) g.dinitial[srow + n0 + s * 16] = m[s];
    }
}

// dB and dC: the sums over the workgroups of a group's channels.
template <class F>
__global__ __launch_bounds__(256) void scan_rows_sum_kernel(ScanProblem p, const float* part,
                                                           void* dBv, void* dCv, int64_t tiles) {
  using S = typename F::S;
  const int64_t N = p.states, per = p.length * 2 * N, total = p.batch * p.groups * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    int64_t j, e, gi;
    const int64_t group = divide(i, per, &j), t = divide(j, 2 * N, &e);
    const int64_t b = divide(group, p.groups, &gi);
    float v = 0.0f;
    if (t < scan_length(p, b)) {
      const float* src = part + group * tiles * per + j;
#pragma unroll 8
      for (int64_t k = 0; k < tiles; ++k) v += src[k * per];
    }
    const int64_t o = ((b * p.length + t) * p.groups + gi) * N;
    if (e < N) {
      ((S*)dBv)[o + e] = narrow<F>(v);
    } else {
      ((S*)dCv)[o + e - N] = narrow<F>(v);
    }
  }
}

// dA, dD and ddt_bias: sums over the batch and its chunks, in order.
__global__ __launch_bounds__(256) void scan_params_sum_kernel(const float* part, int64_t batch,
                                                             int64_t channels, int64_t states,
                                                             float* dA, float* dD, float* dbias) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, count = channels * (states + 2);
  if (i >= count) return;
  float v = 0.0f;
#pragma unroll 8
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
// Tiles per workgroup: two halve the partial sums of dB and dC, where a group
// has two tiles, that leaves a workgroup for every CU, and the registers hold it.
int grad_tiles_each(const ScanProblem& p) {
  const int64_t tiles = (p.channels / p.groups + kScanTile - 1) / kScanTile;
  return tiles > 1 && p.states <= 16 && p.batch * p.groups * ((tiles + 1) / 2) >= 256 ? 2 : 1;
}
int64_t grad_tiles(const ScanProblem& p) {
  const int64_t width = kScanTile * grad_tiles_each(p);
  return (p.channels / p.groups + width - 1) / width;
}
size_t rows_part_floats(const ScanProblem& p) {
  return (size_t)(p.batch * p.groups * grad_tiles(p) * p.length * 2 * p.states);
}
}  // namespace

size_t selective_scan_grad_scratch(const ScanProblem& p) {
  int64_t tokens;
  const int64_t chunks = scan_chunks(p, &tokens);
  return 4 * (rows_part_floats(p) + (size_t)(p.batch * chunks * p.channels * (p.states + 2))) +
         selective_scan_scratch(p);
}

constexpr int64_t kMaxGroups = 1ll << 22;   // workgroups per launch

template <class F>
static hipError_t launch_grad(const ScanProblem& p, const ScanGrads& g, void* scratch,
                              hipStream_t stream) {
  const int64_t tiles = grad_tiles(p);
  const int64_t per = tiles * p.groups;
  const int64_t step = kMaxGroups / per < 1 ? 1 : kMaxGroups / per;
  float* part = (float*)scratch;
  float* params = part + rows_part_floats(p);
  ScanSplit split{};
  split.chunks = (uint32_t)scan_chunks(p, &split.tokens);
  split.ends = params + p.batch * split.chunks * p.channels * (p.states + 2);
  split.spans = split.ends + p.batch * split.chunks * p.channels * p.states;
  for (int64_t b0 = 0; b0 < p.batch; b0 += step) {
    const int64_t nb = p.batch - b0 < step ? p.batch - b0 : step;
    auto launch = [&](auto ns, auto gate, auto tl, auto all) {
      constexpr int TL = decltype(tl)::value, NS = decltype(ns)::value;
      constexpr bool GATE = decltype(gate)::value, ALL = decltype(all)::value;
      if constexpr (TL == 1) {
        if (split.chunks > 1) {
          const int64_t count = nb * per * (split.chunks - 1);
          selective_scan_grad_kernel<F, NS, GATE, TL, ALL, true>
              <<<dim3(xcd_grid(count)), dim3(256), 0, stream>>>(
              p, g, part, params, split, b0, tiles, (uint32_t)count);
        }
      }
      const int64_t count = nb * per * split.chunks;
      selective_scan_grad_kernel<F, NS, GATE, TL, ALL, false>
          <<<dim3(xcd_grid(count)), dim3(256 * TL), 0, stream>>>(
          p, g, part, params, split, b0, tiles, (uint32_t)count);
    };
    auto go = [&](auto ns, auto gate, auto tl) {
      constexpr int NS = decltype(ns)::value;
      if constexpr (NS > 1) {
        if (scan_all_states<NS>(p)) return launch(ns, gate, tl, std::true_type{});
      }
      launch(ns, gate, tl, std::false_type{});
    };
    auto by_tiles = [&](auto ns, auto gate) {
      if constexpr (decltype(ns)::value == 1) {
        if (grad_tiles_each(p) == 2) return go(ns, gate, std::integral_constant<int, 2>{});
      }
      go(ns, gate, std::integral_constant<int, 1>{});
    };
    auto by_gate = [&](auto ns) {
      if (p.z != nullptr) {
        by_tiles(ns, std::true_type{});
      } else {
        by_tiles(ns, std::false_type{});
      }
    };
    if (p.states <= 16) {
      by_gate(std::integral_constant<int, 1>{});
    } else if (p.states <= 32) {
      by_gate(std::integral_constant<int, 2>{});
    } else {
      by_gate(std::integral_constant<int, 4>{});
    }
  }
  const int64_t sums = (p.batch * p.groups * p.length * 2 * p.states + 255) / 256;
  if (sums > 0)
    scan_rows_sum_kernel<F><<<dim3((unsigned)(sums < (1 << 20) ? sums : 1 << 20)), dim3(256), 0,
                              stream>>>(p, part, g.dB, g.dC, tiles);
  const int64_t count = p.channels * (p.states + 2);
  scan_params_sum_kernel<<<dim3((unsigned)((count + 255) / 256)), dim3(256), 0, stream>>>(
      params, p.batch * split.chunks, p.channels, p.states, g.dA, g.dD, g.ddt_bias);
  return hipGetLastError();
}

hipError_t launch_selective_scan_grad(const ScanProblem& p, Fmt fmt, const ScanGrads& g,
                                      void* scratch, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_grad<FmtF32>(p, g, scratch, stream);
    case Fmt::F16: return launch_grad<FmtF16>(p, g, scratch, stream);
    case Fmt::BF16: return launch_grad<FmtBF16>(p, g, scratch, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sca
