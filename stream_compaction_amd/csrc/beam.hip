// Beam search: the best continuations of a batch of beams, and the beams' states
// moved to where they go on.
//
// A continuation of beam j by token v has the score
//   S[j, v] = score[j] + ((l[v] - m) - log(sum over u of exp(l[u] - m))),
// l being the beam's logits and m their maximum; formed in 64 bits, as the scores
// that compete lie closer together than float32's rounding of a sum over a
// vocabulary.  The `count` greatest are chosen in a total order: score, then the
// lower beam, the greater logit, the lower token.
//
// Two launches.  The first reads each logit once: a workgroup keeps a segment of a
// beam's row in registers, finds its maximum and its sum of exponentials, and its
// `count` greatest logits (within a beam the order by score is that by logit).  A
// bound for these comes from the lanes' maxima: in a wave where `count` lanes hold
// something as great as T, T bounds the choice from below, and what is not below it
// is little.  The second launch joins segments and beams, a workgroup a batch entry.
#include "sequence.hpp"

namespace sca {

namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamWaves = kBeamThreads / 64;
constexpr int kListed = 1024;                // candidates of a segment that are ranked
constexpr int kJoinThreads = 1024;
constexpr int kJoinWaves = kJoinThreads / 64;
constexpr int kJoined = 2048;                // candidates of a batch entry that are ranked
constexpr uint32_t kMaskedKey = 0x007fffffu; // order_key(-inf)

// A float's place in the order of all floats (-0 being 0); NaNs are masked logits.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __builtin_bit_cast(float, (k >> 31) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_value64(uint64_t k) {
  return __builtin_bit_cast(double, (k >> 63) ? k & 0x7fffffffffffffffull : ~k);
}

// 2^t for -1000 <= t <= 0, to 4e-11 of it: t = n + f with |f| <= 1/2, a polynomial of
// degree 7 (least maximum of the relative error, fitted there), n to the exponent.
__device__ __forceinline__ double exp2_64(double t) {
  const double shift = 6755399441055744.0;   // 1.5 x 2^52: the sum's last digits are n
  const double r = t + shift, f = t - (r - shift);
  double v = __builtin_fma(f, 1.5201921452474336e-05, 0.00015469291140648007);
  v = __builtin_fma(f, v, 0.0013333922564236862);
  v = __builtin_fma(f, v, 0.009618027253677558);
  v = __builtin_fma(f, v, 0.05550410353447074);
  v = __builtin_fma(f, v, 0.24022651198157435);
  v = __builtin_fma(f, v, 0.6931471807284468);
  v = __builtin_fma(f, v, 0.9999999999616814);
  const uint64_t b = __builtin_bit_cast(uint64_t, v) + (__builtin_bit_cast(uint64_t, r) << 52);
  return __builtin_bit_cast(double, b);
}
constexpr double kLog2e64 = 1.4426950408889634074;

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v = __builtin_fmaxf(v, __shfl_xor(v, m));
  return v;
}

// The greatest T, a multiple of 2^LOW, that at least `count` lanes' keys are not below.
template <int LOW>
__device__ __forceinline__ uint32_t lanes_bound(uint32_t key, int count) {
  uint32_t t = 0;
#pragma unroll
  for (int bit = 31; bit >= LOW; --bit) {
    const uint32_t c = t | (1u << bit);
    if (__builtin_popcountll(__ballot(key >= c)) >= count) t = c;
  }
  // (a 16-bit type's keys end in zeros, below 0 in ones)
  return (t >> 31) ? t : t | ((1u << LOW) - 1);
}

struct Found {                               // of a segment
  float most;
  float pad;
  double sum;
};

struct SegmentShared {
  uint64_t list[kListed];
  double sum[kBeamWaves];
  float most[kBeamWaves];
  uint32_t bound[kBeamWaves], part[kBeamWaves];
  uint32_t listed;
};

// A workgroup's sum of a number of each thread.
__device__ __forceinline__ uint32_t group_sum(uint32_t v, SegmentShared& s, int wave) {
#pragma unroll
  for (int m = 32; m > 0; m /= 2) v += (uint32_t)__shfl_xor((int)v, m);
  __syncthreads();
  if (lane_id() == 0) s.part[wave] = v;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < kBeamWaves; ++w) all += s.part[w];
  return all;
}

}  // namespace

// A segment: 256 NV vectors of 16 bytes.  Entries are (order_key << 32 | ~token), so that the greater entry
// comes first; 0 is none.
template <class F, int NV>
__global__ __launch_bounds__(kBeamThreads) void beam_segment_kernel(BeamProblem p, uint64_t* best,
                                                                   Found* found, int64_t row0,
                                                                   int64_t segments) {
  using S = typename F::S;
  constexpr int E = kVecElems<F>;
  constexpr int kBits = std::is_same_v<F, FmtBF16> ? 16 : (std::is_same_v<F, FmtF16> ? 13 : 0);
  __shared__ SegmentShared sh;
  const int wave = wave_id(), tid = (int)threadIdx.x, count = (int)p.count;
  int64_t seg, j;
  const int64_t row = row0 + divide((int64_t)blockIdx.x, segments, &seg);
  const int64_t b = divide(row, p.beams, &j);
  if (p.finished != nullptr && p.finished[row] != 0) return;     // none of its logits is asked for
  const S* logits = (const S*)p.logits + b * p.logits_batch + j * p.logits_beam;
  if (tid == 0) sh.listed = 0;
  // The row's last vector ends with it and may begin among those of the one before,
  // which are left out.  What a thread adds up depends on the vocabulary alone, not
  // on where the row lies: equal rows have equal sums.
  const int64_t v0 = seg * (kBeamThreads * NV) + tid;
  auto begin = [&](int64_t vec) { return vec * E < p.vocab - E ? vec * E : p.vocab - E; };
  float v[NV][E];
  if (p.vocab >= E) {
    u32x4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      raw[i] = RowIO<F, E>::load_any(logits + begin(v0 + i * kBeamThreads), E);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      RowIO<F, E>::unpack(raw[i], v[i]);
      const int64_t skip = (v0 + i * kBeamThreads) * E - begin(v0 + i * kBeamThreads);
#pragma unroll
      for (int e = 0; e < E; ++e)
        v[i][e] = e >= skip && v[i][e] == v[i][e] ? v[i][e] : -__builtin_huge_valf();
    }
  } else {                                   // less than a vector: the first thread's
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[i][e] = -__builtin_huge_valf();
        if (i == 0 && v0 == 0 && e >= E - p.vocab) {
          const float l = widen<F>(logits[e - (E - p.vocab)]);
          v[i][e] = l == l ? l : v[i][e];
        }
      }
  }
  float most = v[0][0];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) most = __builtin_fmaxf(most, v[i][e]);
  const uint32_t mine = order_key(most);
  const uint32_t bound = lanes_bound<kBits>(mine, count);
  const float wmost = wave_max(most);
  if (lane_id() == 0) {
    sh.most[wave] = wmost;
    sh.bound[wave] = bound;
  }
  __syncthreads();
  float top = sh.most[0];
  uint32_t least = sh.bound[0];
#pragma unroll
  for (int w = 1; w < kBeamWaves; ++w) {
    top = __builtin_fmaxf(top, sh.most[w]);
    least = least > sh.bound[w] ? least : sh.bound[w];
  }
  uint64_t* out = best + (row * segments + seg) * count;
  if (top == -__builtin_huge_valf()) {                           // all masked
    if (tid < count) out[tid] = 0;
    if (tid == 0) found[row * segments + seg] = Found{top, 0.0f, 0.0};
    return;
  }
  // what is above the bound, then what is equal to it
  least = least > kMaskedKey ? least : kMaskedKey + 1;
  auto entry = [&](int i, int e) {
    const uint32_t token = (uint32_t)(begin(v0 + i * kBeamThreads) + e);
    return ((uint64_t)order_key(v[i][e]) << 32) | (uint32_t)~token;
  };
  float edge = key_value(least);
  auto above = [&]() {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v[i][e] > edge) {
          const uint32_t k = __hip_atomic_fetch_add(&sh.listed, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
          if (k < (uint32_t)kListed) sh.list[k] = entry(i, e);
        }
  };
  if (most > edge) above();
  double sum = 0.0;
  if (top == __builtin_huge_valf()) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) sum += v[i][e] == top ? 1.0 : 0.0;
  } else {
    const double off = -(double)top * kLog2e64;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e)
        sum += exp2_64(__builtin_fmax(__builtin_fma((double)v[i][e], kLog2e64, off), -1000.0));
  }
  sum = wave_sum(sum);
  if (lane_id() == 0) sh.sum[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    double all = sh.sum[0];
#pragma unroll
    for (int w = 1; w < kBeamWaves; ++w) all += sh.sum[w];
    found[row * segments + seg] = Found{top, 0.0f, all};
  }
  uint32_t n = sh.listed;
  if (n > (uint32_t)kListed) {
    // too much above the bound (great logits side by side): the count-th greatest
    // itself, bit by bit
    uint32_t t = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = t | (1u << bit);
      uint32_t k = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) k += order_key(v[i][e]) >= c ? 1u : 0u;
      if (group_sum(k, sh, wave) >= (uint32_t)count) t = c;
    }
    edge = key_value(t > kMaskedKey ? t : kMaskedKey + 1);
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    above();
    __syncthreads();
    n = sh.listed;
  }
  if (n < (uint32_t)count) {
    // those equal to the bound, in token order, as many as are asked for
    uint32_t open = (uint32_t)count - n, taken = n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t k = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) k += v[i][e] == edge ? 1u : 0u;
      uint32_t before = wave_scan_incl<Op::Add>(k);
      __syncthreads();
      if (lane_id() == 63) sh.part[wave] = before;
      __syncthreads();
      before -= k;
      uint32_t all = 0;
#pragma unroll
      for (int w = 0; w < kBeamWaves; ++w) {
        before += w < wave ? sh.part[w] : 0;
        all += sh.part[w];
      }
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v[i][e] == edge) {
          if (before < open) sh.list[taken + before] = entry(i, e);
          ++before;
        }
      const uint32_t got = all < open ? all : open;
      taken += got;
      open -= got;
    }
    n = taken;
  }
  __syncthreads();
  for (uint32_t i = tid; i < n; i += kBeamThreads) {
    const uint64_t mine64 = sh.list[i];
    uint32_t rank = 0;
    for (uint32_t k = 0; k < n; ++k) rank += sh.list[k] > mine64 ? 1u : 0u;
    if (rank < (uint32_t)count) out[rank] = mine64;
  }
  if (tid >= (int)n && tid < count) out[tid] = 0;
}

namespace {

// A candidate in the order of the choice: score, lower beam, greater logit, lower token.
struct Candidate {
  uint64_t score;                            // order_key64; 0 is none
  uint32_t beam;
  uint32_t pad;
  uint64_t entry;
};
__device__ __forceinline__ bool beats(const Candidate& a, const Candidate& b) {
  if (a.score != b.score) return a.score > b.score;
  if (a.beam != b.beam) return a.beam < b.beam;
  return a.entry > b.entry;
}

struct JoinShared {
  Candidate list[kJoined];
  double lse[64];                            // log of the sum of exponentials
  float most[64], score[64];
  uint32_t bound[kJoinWaves];
  uint32_t listed;
  Candidate wave_best[kJoinWaves];
};

}  // namespace

__global__ __launch_bounds__(kJoinThreads) void beam_join_kernel(BeamProblem p, const uint64_t* best,
                                                                 const Found* found, float* scores,
                                                                 int32_t* parents, int32_t* tokens,
                                                                 int64_t b0, int64_t segments) {
  __shared__ JoinShared sh;
  const int wave = wave_id(), tid = (int)threadIdx.x, count = (int)p.count, beams = (int)p.beams;
  const int64_t b = b0 + blockIdx.x, row0 = b * beams;
  if (tid == 0) sh.listed = 0;
  for (int j = wave; j < beams; j += kJoinWaves) {
    const Found* f = found + (row0 + j) * segments;
    const bool done = p.finished != nullptr && p.finished[row0 + j] != 0;
    float most = -__builtin_huge_valf();
    double sum = 0.0;
    if (!done) {
      for (int64_t s = lane_id(); s < segments; s += 64) most = __builtin_fmaxf(most, f[s].most);
      most = wave_max(most);
      for (int64_t s = lane_id(); s < segments; s += 64) {
        const float m = f[s].most;
        const double part = f[s].sum;
        if (m == most) sum += part;
        else if (m > -__builtin_huge_valf()) sum += part * exp((double)m - (double)most);
      }
      sum = wave_sum(sum);
    }
    if (lane_id() == 0) {
      sh.most[j] = most;
      sh.lse[j] = done ? 0.0 : log(sum);
      sh.score[j] = p.scores[row0 + j];
    }
  }
  __syncthreads();
  const int64_t per = segments * count, total = per * beams;
  // candidate i of the batch entry
  auto candidate = [&](int64_t i) {
    int64_t k;
    const int j = (int)divide(i, per, &k);
    Candidate c{0, (uint32_t)j, 0, 0};
    const double base = (double)sh.score[j];
    double s;
    if (p.finished != nullptr && p.finished[row0 + j] != 0) {
      if (k != 0) return c;
      c.entry = (uint32_t)~(uint32_t)p.end_token;
      s = base;
    } else {
      c.entry = best[row0 * per + i];
      if (c.entry == 0) return c;
      const float l = key_value((uint32_t)(c.entry >> 32)), m = sh.most[j];
      s = base + ((l == m ? 0.0 : (double)l - (double)m) - sh.lse[j]);
    }
    if (s > -__builtin_huge_val()) c.score = order_key64(s);      // (no NaN)
    return c;
  };
  uint64_t mine = 0;
  for (int64_t i = tid; i < total; i += kJoinThreads) {
    const uint64_t s = candidate(i).score;
    mine = mine > s ? mine : s;
  }
  const uint32_t bound = lanes_bound<0>((uint32_t)(mine >> 32), count);
  if (lane_id() == 0) sh.bound[wave] = bound;
  __syncthreads();
  uint32_t least = 1;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) least = least > sh.bound[w] ? least : sh.bound[w];
  if ((uint32_t)(mine >> 32) >= least)
    for (int64_t i = tid; i < total; i += kJoinThreads) {
      const Candidate c = candidate(i);
      if ((uint32_t)(c.score >> 32) < least) continue;
      const uint32_t k = __hip_atomic_fetch_add(&sh.listed, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      if (k < (uint32_t)kJoined) sh.list[k] = c;
    }
  __syncthreads();
  uint32_t n = sh.listed;
  if (n > (uint32_t)kJoined) {
    // too many: one after the other, the best of those behind the one before
    Candidate last{~0ull, 0, 0, ~0ull};
    n = 0;
    for (int k = 0; k < count; ++k) {
      Candidate top{0, 0, 0, 0};
      for (int64_t i = tid; i < total; i += kJoinThreads) {
        const Candidate c = candidate(i);
        if (c.score != 0 && beats(last, c) && beats(c, top)) top = c;
      }
      for (int m = 32; m > 0; m /= 2) {
        Candidate o{__shfl_xor((unsigned long long)top.score, m), (uint32_t)__shfl_xor((int)top.beam, m), 0,
                    __shfl_xor((unsigned long long)top.entry, m)};
        if (beats(o, top)) top = o;
      }
      __syncthreads();
      if (lane_id() == 0) sh.wave_best[wave] = top;
      __syncthreads();
      top = sh.wave_best[0];
      for (int w = 1; w < kJoinWaves; ++w)
        if (beats(sh.wave_best[w], top)) top = sh.wave_best[w];
      if (top.score == 0) break;
      if (tid == 0) sh.list[n] = top;
      ++n;
      last = top;
    }
    __syncthreads();
  }
  const int64_t out = b * count;
  for (uint32_t i = tid; i < n; i += kJoinThreads) {
    const Candidate c = sh.list[i];
    uint32_t rank = 0;
    for (uint32_t k = 0; k < n; ++k) rank += beats(sh.list[k], c) ? 1u : 0u;
    if (rank >= (uint32_t)count) continue;
    scores[out + rank] = (float)key_value64(c.score);
    parents[out + rank] = (int32_t)c.beam;
    tokens[out + rank] = (int32_t)~(uint32_t)c.entry;
  }
  if (n >= (uint32_t)count || wave != 0) return;
  // fewer than asked for have a chance: the first of the others, in order
  uint32_t filled = n;
  for (int64_t f0 = 0; filled < (uint32_t)count; f0 += 64) {
    const int64_t f = f0 + lane_id();
    int64_t v;
    const int64_t j = divide(f, p.vocab, &v);
    bool on = j < p.beams;
    for (uint32_t k = 0; k < n; ++k)
      if (sh.list[k].beam == (uint32_t)j && (uint32_t)~(uint32_t)sh.list[k].entry == (uint32_t)v) on = false;
    const uint64_t all = __ballot(on);
    const uint32_t at = filled + (uint32_t)__builtin_popcountll(all & ((1ull << lane_id()) - 1));
    if (on && at < (uint32_t)count) {
      scores[out + at] = -__builtin_huge_valf();
      parents[out + at] = (int32_t)j;
      tokens[out + at] = (int32_t)v;
    }
    filled += (uint32_t)__builtin_popcountll(all);
  }
}

namespace {

// Vectors a thread: as many as still leave a workgroup for every CU, so that a few
// rows are read by the whole chip.
template <class F> int beam_vectors(const BeamProblem& p) {
  const int64_t vecs = (p.vocab + kVecElems<F> - 1) / kVecElems<F>, rows = p.batch * p.beams;
  for (int nv = 4; nv > 1; nv /= 2)
    if (rows * (vecs / (kBeamThreads * nv)) >= 512) return nv;
  return 1;
}
template <class F> int64_t beam_segments(const BeamProblem& p, int nv) {
  const int64_t vecs = (p.vocab + kVecElems<F> - 1) / kVecElems<F>;
  return (vecs + kBeamThreads * nv - 1) / (kBeamThreads * nv);
}

template <class F, int NV>
hipError_t launch_segments(const BeamProblem& p, uint64_t* best, Found* found, int64_t segments,
                           hipStream_t stream) {
  const int64_t rows = p.batch * p.beams, most = (1ll << 22) / segments, step = most < 1 ? 1 : most;
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t n = rows - r < step ? rows - r : step;
    beam_segment_kernel<F, NV><<<dim3((unsigned)(n * segments)), dim3(kBeamThreads), 0, stream>>>(
        p, best, found, r, segments);
  }
  return hipGetLastError();
}

template <class F> size_t beam_scratch_f(const BeamProblem& p) {
  const size_t segs = (size_t)(p.batch * p.beams) * (size_t)beam_segments<F>(p, beam_vectors<F>(p));
  return segs * (sizeof(Found) + 8 * (size_t)p.count);
}

template <class F>
hipError_t launch_beam_f(const BeamProblem& p, float* scores, int32_t* parents, int32_t* tokens,
                         void* scratch, hipStream_t stream) {
  const int nv = beam_vectors<F>(p);
  const int64_t segments = beam_segments<F>(p, nv);
  Found* found = (Found*)scratch;
  uint64_t* best = (uint64_t*)(found + p.batch * p.beams * segments);
  hipError_t e;
  switch (nv) {
    case 4: e = launch_segments<F, 4>(p, best, found, segments, stream); break;
    case 2: e = launch_segments<F, 2>(p, best, found, segments, stream); break;
    default: e = launch_segments<F, 1>(p, best, found, segments, stream); break;
  }
  if (e != hipSuccess) return e;
  for (int64_t b = 0; b < p.batch; b += 1 << 21) {
    const int64_t n = p.batch - b < (1 << 21) ? p.batch - b : 1 << 21;
    beam_join_kernel<<<dim3((unsigned)n), dim3(kJoinThreads), 0, stream>>>(p, best, found, scores, parents,
                                                                          tokens, b, segments);
  }
  return hipGetLastError();
}

}  // namespace

size_t beam_select_scratch(const BeamProblem& p, Fmt fmt) {
  switch (fmt) {
    case Fmt::F32: return beam_scratch_f<FmtF32>(p);
    case Fmt::F16: return beam_scratch_f<FmtF16>(p);
    case Fmt::BF16: return beam_scratch_f<FmtBF16>(p);
    default: return 0;
  }
}

hipError_t launch_beam_select(const BeamProblem& p, Fmt fmt, float* scores, int32_t* parents,
                              int32_t* tokens, void* scratch, hipStream_t stream) {
  switch (fmt) {
    case Fmt::F32: return launch_beam_f<FmtF32>(p, scores, parents, tokens, scratch, stream);
    case Fmt::F16: return launch_beam_f<FmtF16>(p, scores, parents, tokens, scratch, stream);
    case Fmt::BF16: return launch_beam_f<FmtBF16>(p, scores, parents, tokens, scratch, stream);
    default: return hipErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// States to their new beams: new[b, j] = old[b, parent[b, j]].  A thread has one
// column of 16 bytes (fewer where there are many beams, to hold a column of all of
// them in registers) in every beam of a batch entry: it reads all it moves before it
// writes, so that the states can be moved in place, where beams that go on as
// themselves are neither read nor written.  All tensors go out in one launch (64 of
// them a launch).
// ---------------------------------------------------------------------------
namespace {

constexpr int kMoved = 64;                   // tensors a launch
struct Moves {
  uintptr_t from[kMoved], to[kMoved];
  int64_t bytes[kMoved];                     // of a row
  uint32_t first[kMoved + 1];                // its first block of columns, of a batch entry
  int count;
};

template <class V> __device__ __forceinline__ V load_loose(uintptr_t a) {
  typedef V Loose __attribute__((aligned(1)));
  return *gptr<const Loose>(a);
}
template <class V> __device__ __forceinline__ void store_loose(uintptr_t a, V v) {
  typedef V Loose __attribute__((aligned(1)));
  *gptr<Loose>(a) = v;
}

template <int NB, class V>
__device__ __forceinline__ void move_column(uintptr_t from, uintptr_t to, int64_t bytes, const int* parent,
                                            uint64_t moves) {
  // (every load is issued: a register that only a branch writes costs many more)
  V v[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) v[j] = load_loose<V>(from + (uintptr_t)(parent[j] * bytes));
#pragma unroll
  for (int j = 0; j < NB; ++j)
    if ((moves >> j) & 1) store_loose<V>(to + (uintptr_t)(j * bytes), v[j]);
}

}  // namespace

template <int NB, class V>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4, 8)))
void beam_reorder_kernel(Moves m, const int32_t* parents, int64_t b0,
                                                           int beams) {
  const int64_t blocks = m.first[m.count];
  int64_t block;
  const int64_t b = b0 + divide((int64_t)blockIdx.x, blocks, &block);
  int t = 0;
  while (t + 1 < m.count && (uint32_t)block >= m.first[t + 1]) ++t;
  const bool in_place = m.from[t] == m.to[t];
  int parent[NB];
  uint64_t moves = 0;                        // by beam
  int some = 0;                              // a row that is read
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int q = j < beams ? parents[b * beams + j] : j;
    parent[j] = __builtin_amdgcn_readfirstlane(q >= 0 && q < beams ? q : j);
    if (j < beams && !(in_place && parent[j] == j)) {
      moves |= 1ull << j;
      some = parent[j];
    }
  }
  if (moves == 0) return;
#pragma unroll
  for (int j = 0; j < NB; ++j) parent[j] = (moves >> j) & 1 ? parent[j] : some;
  const int64_t bytes = m.bytes[t], whole = bytes / (int64_t)sizeof(V);
  const int64_t col = (block - m.first[t]) * 256 + threadIdx.x;
  const uintptr_t skip = (uintptr_t)(b * beams * bytes);
  const uintptr_t from = m.from[t] + skip, to = m.to[t] + skip;
  if (col < whole) {
    move_column<NB, V>(from + (uintptr_t)col * sizeof(V), to + (uintptr_t)col * sizeof(V), bytes, parent, moves);
  } else if (col - whole < bytes % (int64_t)sizeof(V)) {         // a row's last bytes, one a thread
    const uintptr_t at = (uintptr_t)(whole * (int64_t)sizeof(V) + (col - whole));
    move_column<NB, uint8_t>(from + at, to + at, bytes, parent, moves);
  }
}

template <int NB, class V>
static hipError_t launch_moves(const void* const* states, void* const* new_states, const int64_t* row_bytes,
                               int64_t tensors, const int32_t* parents, int64_t batch, int64_t beams,
                               hipStream_t stream) {
  constexpr int64_t kMostBlocks = 1ll << 23;
  for (int64_t t = 0; t < tensors;) {
    Moves m{};
    int64_t blocks = 0;
    for (; t < tensors && m.count < kMoved; ++t) {
      if (row_bytes[t] == 0) continue;
      const int64_t cols = row_bytes[t] / (int64_t)sizeof(V) + row_bytes[t] % (int64_t)sizeof(V);
      const int64_t need = (cols + 255) / 256;
      if (m.count > 0 && blocks + need > kMostBlocks) break;
      m.from[m.count] = (uintptr_t)states[t];
      m.to[m.count] = (uintptr_t)new_states[t];
      m.bytes[m.count] = row_bytes[t];
      m.first[m.count] = (uint32_t)blocks;
      blocks += need;
      m.first[++m.count] = (uint32_t)blocks;
    }
    if (m.count == 0) break;
    const int64_t step = blocks >= kMostBlocks ? 1 : kMostBlocks / blocks;
    for (int64_t b = 0; b < batch; b += step) {
      const int64_t n = batch - b < step ? batch - b : step;
      beam_reorder_kernel<NB, V><<<dim3((unsigned)(n * blocks)), dim3(256), 0, stream>>>(m, parents, b, (int)beams);
    }
  }
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const void* const* states, void* const* new_states,
                               const int64_t* row_bytes, int64_t tensors, const int32_t* parents,
                               int64_t batch, int64_t beams, hipStream_t stream) {
  if (beams <= 4) return launch_moves<4, u32x4>(states, new_states, row_bytes, tensors, parents, batch, beams, stream);
  if (beams <= 8) return launch_moves<8, u32x4>(states, new_states, row_bytes, tensors, parents, batch, beams, stream);
  if (beams <= 16) return launch_moves<16, u32x4>(states, new_states, row_bytes, tensors, parents, batch, beams, stream);
  if (beams <= 32) return launch_moves<32, u32x2>(states, new_states, row_bytes, tensors, parents, batch, beams, stream);
  return launch_moves<64, uint32_t>(states, new_states, row_bytes, tensors, parents, batch, beams, stream);
}

}  // namespace sca
