// Selective scan, forward and single-token step:
//   dt = softplus(dt_raw + dt_bias),  h[t] = exp(dt A) h[t-1] + dt x B,
//   y = (C . h + D x) silu(z)
// per channel, with `states` states each.  See scan_tile.hpp for the mapping.
#include "scan_tile.hpp"

namespace sca {

namespace {

// Forward.  A lane owns one channel and NS of its states and walks the tokens in
// order: per token and state a product and an exponential for the decay, a
// product for the input, a multiply-add for the state and a product with C,
// which is what the definition asks for and no more, so the kernel is bound by
// these vector instructions.  Lanes 16 r .. 16 r + 15 of wave w hold 16
// channels' state w 4 + r (+ 16, ...): B and C are the same for a row of 16
// lanes, so a lane holds them for one of 16 tokens and the products take them by
// DPP row broadcast, without an instruction or an LDS read per token.
//
// A workgroup (4 waves) owns 16 channels of one sequence, in blocks of T tokens.
// Its threads turn dt into steps and products with x, once per element, and
// stage them and B and C in LDS as float32 planes of one value per token; the
// sums over a wave's states are left there too, and the block's outputs are put
// together from them during the next block's walk.  Everything is buffered twice:
// one barrier per block.
//
// Measured (traced), 16 states, softplus and gate: bf16 8192 x 4096 277 us (1.9e12
// updates a second; one wave per SIMD, vector units 57% busy, the rest is latency),
// f16, a batch of 4 with 8192 of 16384 tokens 204 us (three waves, 93%).  The
// definition's own instructions alone would take 93 us; a block's 291
// instructions per wave are 128 + 32 exponentials for them, 48 for the sums over
// rows and some 83 for steps, gate and staging.  Tokens across lanes with wave
// scans of affine maps, the arrangement before, took 302 and 342 us: its second
// pass over every token and the scans cost more than the sums over rows here.
constexpr int kT = 32;                  // tokens per block
constexpr int kPS = kT + 4;             // plane stride: 16 channels' 16-byte reads, and the
                                        // pairs' stores, fall on different banks
constexpr int kPlane = kScanTile * kPS;
constexpr int kFwdThreads = 256;        // T tokens of 8 channel pairs

}  // namespace

// What a launch does: all; also keep the state before every kKeep tokens in
// `starts`, for the gradient; or find the chunks' ends of a split scan alone.
enum class Pass { Run, Keep, Ends };

template <class F, int NS, bool VEC, bool ALL, Pass PASS>
__global__ __launch_bounds__(kFwdThreads) void selective_scan_kernel(
    ScanProblem p, void* yv, float* final_state, float* starts, ScanSplit split, int64_t b0,
    int64_t tiles, uint32_t count) {
  constexpr bool KEEP = PASS == Pass::Keep, ENDS = PASS == Pass::Ends;
  using S = typename F::S;
  using IO = RowIO<F, 2>;
  typedef float vec4 __attribute__((ext_vector_type(4)));
  __shared__ alignas(16) float s_x[2][2 * kPlane];           // steps, steps times x
  __shared__ alignas(16) float s_bc[2][2 * NS * kPlane];     // B, C
  __shared__ alignas(16) float s_part[2][ENDS ? 1 : 4 * kPlane];   // per wave
  __shared__ alignas(16) float s_none[ALL ? 1 : kT];         // products of states that do not exist

  const uint32_t id = xcd_order(blockIdx.x);
  if (id >= count) return;
  // chunk by chunk; a chunk is worked on like a sequence that begins at `first`
  const uint32_t per = ENDS ? count / (split.chunks - 1) : count / split.chunks;
  const int64_t chunk = id / per, first = chunk * split.tokens;
  const ScanPlace at = scan_place(p, b0, tiles, id % per, kScanTile);
  auto within = [&](int64_t n) {
    return n <= first ? 0 : (n - first < split.tokens ? n - first : split.tokens);
  };
  const int64_t whole = scan_length(p, at.b), len = within(whole), padded = within(p.length);
  const int N = (int)p.states, nch = (int)at.nch;
  const bool gate = p.z != nullptr;
  const int tid = (int)threadIdx.x, lane = lane_id(), wave = wave_id();
  const int row = lane / 16, cl = lane % 16;
  const int n0 = wave * 4 + row;                // this lane's states: n0, n0 + 16, ...
  const int64_t ch = at.ch + cl;

  // staging: this thread's token and two channels (and two states of each 16)
  const int tok = tid / 8, pair = tid % 8;
  const bool stager = pair * 2 < nch;
  float* keep = KEEP ? starts + ((at.b * ((p.length + kKeep - 1) / kKeep) + first / kKeep) * p.channels +
                                 ch) * N + n0
                     : nullptr;
  using Src = PairSrc<F, VEC>;
  using Raw = Pair<F, VEC>;
  Src xs(p.x, p.x_batch, p.x_token, at.b, at.ch + first * p.x_token, nch);
  Src dts(p.dt, p.dt_batch, p.dt_token, at.b, at.ch + first * p.dt_token, nch);
  // without a gate x stands in, unused
  const int64_t z_token = gate ? p.z_token : p.x_token;
  Src zs(gate ? p.z : p.x, gate ? p.z_batch : p.x_batch, z_token, at.b, at.ch + first * z_token,
         nch);
  Src Bs[NS], Cs[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    // the states past the last 16 that exist read the first ones, unused
    const int n = s * 16 < N ? s * 16 : 0;
    Bs[s] = Src(p.B, p.B_batch, p.B_token, at.b,
                at.g * p.B_group + n + first * p.B_token, N - n);
    Cs[s] = Src(p.C, p.C_batch, p.C_token, at.b,
                at.g * p.C_group + n + first * p.C_token, N - n);
  }
  S* y = (S*)yv + (at.b * p.length + first) * p.channels + at.ch;
  float Dc[2], bias[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool on = pair * 2 + i < nch;
    Dc[i] = on && p.D != nullptr ? p.D[at.ch + pair * 2 + i] : 0.0f;
    bias[i] = on && p.dt_bias != nullptr ? p.dt_bias[at.ch + pair * 2 + i] : 0.0f;
  }
  float A2[NS], h[NS];
  bool mine[NS];
  const int64_t srow = (at.b * p.channels + ch) * N;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int n = n0 + s * 16;
    mine[s] = cl < nch && n < N;
    A2[s] = mine[s] ? p.A[ch * N + n] * kLog2e : kNoState;
    h[s] = !ENDS && mine[s] && p.initial_state != nullptr ? p.initial_state[srow + n] : 0.0f;
  }

  if (!ALL && tid < kT) s_none[tid] = 0.0f;

  float span = 0.0f;                            // ENDS: sum of the channel's steps
  if constexpr (!ENDS) {
    // the chunk's start, from the chunks before (eight loads at a time)
#pragma unroll 8
    for (int64_t c = 0; c < chunk; ++c) {
      const int64_t r = (at.b * split.chunks + c) * p.channels + (cl < nch ? ch : at.ch);
      const float passed = split.spans[r];
#pragma unroll
      for (int s = 0; s < NS; ++s)
        h[s] = carried(passed * A2[s], h[s]) + (mine[s] ? split.ends[r * N + n0 + s * 16] : 0.0f);
    }
  }
  // the next block travels while one is worked on
  struct Fetched { Raw x, dt, z, B[NS], C[NS]; };
  auto seek = [&](int64_t t0) {
    xs.seek(t0, len);
    dts.seek(t0, len);
    zs.seek(t0, len);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      Bs[s].seek(t0, len);
      Cs[s].seek(t0, len);
    }
  };
  auto fetch = [&](Fetched& f) {
    f.x = xs.load();
    f.dt = dts.load();
    if constexpr (!ENDS) f.z = zs.load();
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      f.B[s] = Bs[s].load();
      if constexpr (!ENDS) f.C[s] = Cs[s].load();
    }
    xs.advance(kT);
    dts.advance(kT);
    zs.advance(kT);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      Bs[s].advance(kT);
      Cs[s].advance(kT);
    }
  };
  // what a block's outputs need beside the sums: D x and the gate's factor
  struct Rest { float skip[2], factor[2]; };
  // The fetched block into buffer `buf`; tokens past the end get step 0 (a = 1,
  // b = 0).  Without branches, so that it is scheduled into the walk's waits.
  auto stage = [&](const Fetched& f, bool exists, int buf, Rest& rest) {
    float x[2], dt[2], v[2];
    f.x.unpack(x);
    f.dt.unpack(dt);
    if constexpr (!ENDS) f.z.unpack(v);
    float* to = s_x[buf] + pair * 2 * kPS + tok;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float raw = dt[i] + bias[i];
      const float soft = softplus(raw);
      const float d = p.softplus ? soft : raw;
      to[i * kPS] = exists ? d : 0.0f;
      to[kPlane + i * kPS] = exists ? d * x[i] : 0.0f;
      if constexpr (!ENDS) {
        rest.skip[i] = Dc[i] * x[i];
        const float factor = silu(v[i]);
        rest.factor[i] = gate ? factor : 1.0f;
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      float* bc = s_bc[buf] + (s * 16 + pair * 2) * kPS + tok;
      const int n = s * 16 + pair * 2;
      const bool on0 = exists && n < N, on1 = exists && n + 1 < N;
      f.B[s].unpack_if(on0, on1, v);
      bc[0] = v[0];
      bc[kPS] = v[1];
      if constexpr (!ENDS) {
        f.C[s].unpack_if(on0, on1, v);
        bc[NS * kPlane] = v[0];
        bc[NS * kPlane + kPS] = v[1];
      }
    }
  };
  auto walk = [&](int64_t t0, int buf) {
    auto products = [&](int s) {
      return ALL || mine[s] ? s_x[buf] + kPlane + cl * kPS : s_none;
    };
#pragma unroll
    for (int sub = 0; sub < kT; sub += 16) {
      const float* xp = s_x[buf] + cl * kPS + sub;
      float dt[16], u[16], v[16], sums[4];
#pragma unroll
      for (int t = 0; t < 16; t += 4) {
        const vec4 d = *(const vec4*)(xp + t), w = *(const vec4*)(products(0) + sub + t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dt[t + i] = d[i];
          u[t + i] = w[i];
        }
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (!ALL && s > 0) {
#pragma unroll
          for (int t = 0; t < 16; t += 4) {
            const vec4 w = *(const vec4*)(products(s) + sub + t);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[t + i] = w[i];
          }
        }
        if (KEEP && mine[s] && t0 + sub < len) keep[s * 16] = h[s];
        const float* bc = s_bc[buf] + (s * 16 + n0) * kPS + sub + cl;
        const float B = bc[0], C = ENDS ? 0.0f : bc[NS * kPlane];
        for_tokens([&](auto tc) {
          constexpr int t = decltype(tc)::value;
          const float a = exp2_hw(dt[t] * A2[s]);
          h[s] = __builtin_fmaf(a, h[s], row_bcast<t>(B) * u[t]);
          if constexpr (ENDS) return;
          if (s == 0) {
            v[t] = row_bcast<t>(C) * h[s];
          } else {
            v[t] = __builtin_fmaf(row_bcast<t>(C), h[s], v[t]);
          }
          // the product stays beside its broadcast, which else does not fold into it
          asm volatile("" : "+v"(v[t]));
        }, std::make_integer_sequence<int, 16>{});
      }
      if constexpr (ENDS) {
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 16; ++t) sum += dt[t];
        span += sum;
        continue;
      }
      rows_sum(v, sums);
      *(vec4*)(s_part[buf] + (wave * 16 + cl) * kPS + sub + row * 4) =
          vec4{sums[0], sums[1], sums[2], sums[3]};
      if (KEEP) keep += p.channels * N;
    }
  };
  const uint32_t off = (uint32_t)((tok * p.channels + pair * 2) * (int64_t)sizeof(S));
  auto finish = [&](const Rest& rest, int64_t t0, int buf) {
    float out[2];
    const float* from = s_part[buf] + pair * 2 * kPS + tok;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v = rest.skip[i];
#pragma unroll
      for (int w = 0; w < 4; ++w) v += from[w * kPlane + i * kPS];
      out[i] = v * rest.factor[i];
    }
    const bool live = t0 >= 0 && t0 + tok < len;
    const S* to = y + t0 * p.channels;
    if constexpr (VEC) {
      store_if(to, off, live && stager, IO::pack(out));
    } else {
      store_if(to, off, live && pair * 2 < nch, narrow<F>(out[0]));
      store_if(to, off + (uint32_t)sizeof(S), live && pair * 2 + 1 < nch, narrow<F>(out[1]));
    }
  };

  const int64_t blocks = (len + kT - 1) / kT;
  Fetched f;
  // Block t0 is staged in buffer `buf`, the block after it in f; the outputs of the
  // block before it (none for the first) are due.  No branch between the barriers
  // but the last blocks' seek: all of it is scheduled together.
  Rest rest[2] = {};
  auto step = [&](int64_t t0, int buf) {
    if (t0 + 3 * kT > len) seek(t0 + 2 * kT);
    if constexpr (!ENDS) finish(rest[buf ^ 1], t0 - kT, buf ^ 1);
    stage(f, t0 + kT + tok < len, buf ^ 1, rest[buf ^ 1]);
    fetch(f);
    walk(t0, buf);
    lds_barrier();
  };
  if (blocks > 0) {
    seek(0);
    fetch(f);
    stage(f, tok < len, 0, rest[0]);
    if (2 * kT > len) seek(kT);
    fetch(f);
    lds_barrier();
    int64_t blk = 0;
    for (; blk + 1 < blocks; blk += 2) {
      step(blk * kT, 0);
      step((blk + 1) * kT, 1);
    }
    if (blk < blocks) step(blk * kT, 0);
    if constexpr (!ENDS) {
      if (blocks & 1) {
        finish(rest[0], (blocks - 1) * kT, 0);
      } else {
        finish(rest[1], (blocks - 1) * kT, 1);
      }
    }
  }
  if constexpr (ENDS) {
    const int64_t r = (at.b * split.chunks + chunk) * p.channels + ch;
    if (wave == 0 && row == 0 && cl < nch) split.spans[r] = span;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (mine[s]) split.ends[r * N + n0 + s * 16] = h[s];
    return;
  }
  // tokens past the sequence's end
  for (int64_t i = len * kScanTile + tid; i < padded * kScanTile; i += kFwdThreads)
    if (i % kScanTile < nch) y[(i / kScanTile) * p.channels + i % kScanTile] = S(0);
  // the final state is the chunk's in which the sequence ends
  const bool ends_here = whole > first ? whole - first <= split.tokens : chunk == 0 && whole == 0;
  if (final_state == nullptr || !ends_here) return;
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (mine[s]) final_state[srow + n0 + s * 16] = h[s];
}

// Workgroups of a launch: grid sizes count work-items in 32 bits, so batches
// beyond that go out as several launches.
constexpr int64_t kMaxGroups = 1ll << 21;

// Chunks by an estimate in tokens' time.  With w waves per SIMD (256 workgroups
// are one) a token takes 1 + 0.5 (w - 1) times as long as with up to one; the
// first pass costs 0.6 of the second and leaves out one chunk; its launch and the
// chunks' starts stand for 150 + 8 n tokens.  The split must win a fifth.  Forward
// / gradient, split against whole, 16 states in bf16: 8192 x 64 channels 28 / 53 us
// against 263 / 717, 2048 x 512 24 / 49 against 69 / 192, 2 x 4096 x 768 71 / 154
// against 134 / 377, 8192 x 2048 160 / 385 against 266 / 748, 7 x 1024 x 300 38 / 79
// against 38 / 105.  From 256 workgroups on (8192 x 4096) the estimate gains
// nothing.
int64_t scan_chunks(const ScanProblem& p, int64_t* tokens) {
  const int64_t groups = (p.channels / p.groups + kScanTile - 1) / kScanTile * p.groups * p.batch;
  *tokens = p.length > 0 ? p.length : 1;
  if (groups == 0 || groups >= 256 || p.length < 512) return 1;
  int64_t best = p.length * 8 / 10, chunks = 1;
  for (int64_t n = 2; n <= 32 && n * 128 <= p.length; ++n) {
    const int64_t over = groups * n > 256 ? groups * n - 256 : 0;
    const int64_t each = p.length / n * (10 * n + 6 * (n - 1)) / (10 * n);
    const int64_t time = each * (25600 + 50 * over) / 25600 + 150 + 8 * n;
    if (time < best) {
      best = time;
      chunks = n;
    }
  }
  if (chunks == 1) return 1;
  *tokens = ((p.length + chunks - 1) / chunks + kT - 1) / kT * kT;
  return (p.length + *tokens - 1) / *tokens;
}
size_t selective_scan_scratch(const ScanProblem& p) {
  int64_t tokens;
  const int64_t chunks = scan_chunks(p, &tokens);
  return chunks == 1 ? 0 : (size_t)(p.batch * chunks * p.channels * (p.states + 1)) * 4;
}

template <class F, int NS, bool VEC, bool ALL>
static void fwd_launch(const ScanProblem& p, void* y, float* final_state, float* starts,
                   const ScanSplit& split, hipStream_t stream) {
  const int64_t tiles = (p.channels / p.groups + kScanTile - 1) / kScanTile;
  const int64_t per = tiles * p.groups;
  const int64_t step = kMaxGroups / per < 1 ? 1 : kMaxGroups / per;
  for (int64_t b0 = 0; b0 < p.batch; b0 += step) {
    const int64_t nb = p.batch - b0 < step ? p.batch - b0 : step;
    auto go = [&](auto pass, int64_t chunks) {
      const int64_t count = nb * per * chunks;
      selective_scan_kernel<F, NS, VEC, ALL, decltype(pass)::value>
          <<<dim3(xcd_grid(count)), dim3(kFwdThreads), 0, stream>>>(
              p, y, final_state, starts, split, b0, tiles, (uint32_t)count);
    };
    if (split.chunks > 1) go(std::integral_constant<Pass, Pass::Ends>{}, split.chunks - 1);
    if (starts != nullptr) {
      go(std::integral_constant<Pass, Pass::Keep>{}, split.chunks);
    } else {
      go(std::integral_constant<Pass, Pass::Run>{}, split.chunks);
    }
  }
}

template <class F, int NS, bool VEC>
static void fwd_go(const ScanProblem& p, void* y, float* final_state, float* starts,
                   const ScanSplit& split, hipStream_t stream) {
  if constexpr (NS > 1) {
    if (scan_all_states<NS>(p))
      return fwd_launch<F, NS, VEC, true>(p, y, final_state, starts, split, stream);
  }
  fwd_launch<F, NS, VEC, false>(p, y, final_state, starts, split, stream);
}

template <class F>
static hipError_t launch_fwd(const ScanProblem& p, void* y, float* final_state, float* starts,
                             void* scratch, hipStream_t stream) {
  ScanSplit split{};
  split.chunks = 1;
  split.tokens = p.length > 0 ? p.length : 1;
  if (scratch != nullptr) {
    split.chunks = (uint32_t)scan_chunks(p, &split.tokens);
    split.ends = (float*)scratch;
    split.spans = split.ends + p.batch * split.chunks * p.channels * p.states;
  }
  auto by_states = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    if (p.states <= 16) {
      fwd_go<F, 1, VEC>(p, y, final_state, starts, split, stream);
    } else if (p.states <= 32) {
      fwd_go<F, 2, VEC>(p, y, final_state, starts, split, stream);
    } else {
      fwd_go<F, 4, VEC>(p, y, final_state, starts, split, stream);
    }
  };
  if (scan_pairs<F>(p, y)) {
    by_states(std::true_type{});
  } else {
    by_states(std::false_type{});
  }
  return hipGetLastError();
}

hipError_t launch_selective_scan(const ScanProblem& p, Fmt fmt, void* y, float* final_state,
                                 float* starts, void* scratch, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_fwd<FmtF32>(p, y, final_state, starts, scratch, stream);
    case Fmt::F16: return launch_fwd<FmtF16>(p, y, final_state, starts, scratch, stream);
    case Fmt::BF16: return launch_fwd<FmtBF16>(p, y, final_state, starts, scratch, stream);
    default: return hipErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// One token.  Bound by the state: 8 bytes per state and sequence against some
// six operations.  G lanes (a power of two) share a channel, lane q of them
// owning the V states at q V, (q + G) V, ...; V = 4 makes the state's loads and
// stores 16 bytes wide and a wave's contiguous.  A lane takes R sequences of
// its channel at once: A, D and the bias are read once for them and R loads of
// the state are in flight.  128 x 4096 x 16 in bf16 (72 MB), three states in turn,
// which the last-level cache holds in part: R = 2 16.4 us (4.4 TB/s), R = 4 20.2 us,
// whose registers leave fewer waves; six in turn: R = 2 20.5 us (3.5 TB/s).  A launch owns the
// sequences [first, end): what a lane's R reach past `end` is the next launch's,
// and to be moved once only.
// ---------------------------------------------------------------------------
template <class F, int V, int G, int R>
__global__ __launch_bounds__(256) void selective_scan_step_kernel(ScanProblem p,
                                                                 const float* state,
                                                                 float* new_state, void* yv,
                                                                 int64_t first, int64_t end) {
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
    on[r] = b < end;
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
    IO::unpack(IO::load(p.A + ch * N + n), A);
    typename IO::Raw h0[R];
    typename BIO::Raw Bn[R], Cn[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t b = b0 + r;
      h0[r] = typename IO::Raw{};
      Bn[r] = Cn[r] = typename BIO::Raw{};
      if (!on[r]) continue;
      h0[r] = IO::load(state + (b * p.channels + ch) * N + n);
      Bn[r] = BIO::load((const S*)p.B + b * p.B_batch + g * p.B_group + n);
      Cn[r] = BIO::load((const S*)p.C + b * p.C_batch + g * p.C_group + n);
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
        IO::store(new_state + ((b0 + r) * p.channels + ch) * N + n, IO::pack(h));
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
  constexpr int R = 2;
  const bool many = p.batch * cols >= 2048 * R;
  const int64_t step = kMaxGroups / cols < 1 ? 1 : kMaxGroups / cols;
  for (int64_t b0 = 0; b0 < p.batch; b0 += step) {
    const int64_t nb = p.batch - b0 < step ? p.batch - b0 : step;
    if (many) {
      selective_scan_step_kernel<F, V, G, R><<<dim3((unsigned)((nb + R - 1) / R * cols)), dim3(256), 0,
                                               stream>>>(p, state, new_state, y, b0, b0 + nb);
    } else {
      selective_scan_step_kernel<F, V, G, 1><<<dim3((unsigned)(nb * cols)), dim3(256), 0, stream>>>(
          p, state, new_state, y, b0, b0 + nb);
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
