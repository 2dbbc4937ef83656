// Beam search: the best continuations of a batch of beams, and the beams' states
// moved to where they go on.
//
// A continuation of beam j by token v has the score
//   S[j, v] = score[j] + ((l[v] - m) - log(sum over u of exp(l[u] - m))),
// l being the beam's logits and m their maximum; formed in 64 bits, as the scores
// that compete lie closer together than float32's rounding of a sum over a
// vocabulary.  Every exponential is of a difference from a maximum, so that rows
// which are one another plus a constant have equal scores, and a token that is
// certain has its beam's own.  The `count` greatest are chosen in a total order:
// score, then the lower beam, the greater logit, the lower token.
//
// Two launches.  The first reads each logit once: a workgroup keeps a segment of a
// beam's row in registers, finds its maximum, then its sum of exponentials and its
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

// exp(x) for -690 <= x <= 0: 1 at 0, and within (5e-16 + 2e-17 |x|) of itself (the second
// by log2(e)'s own rounding).  x log2(e) is n + f with |f| <= 1/2: n comes from the last
// digits of a sum with 1.5 x 2^52, f from the same product with n taken off in one
// rounding; 2^f is a polynomial of degree 10 that is 1 at 0 (relative error 3e-16, fitted
// there by exchange), and n is added to its exponent.
__device__ __forceinline__ double exp_64(double x) {
  const double shift = 6755399441055744.0, log2e = 1.4426950408889634074;
  const double r = __builtin_fma(x, log2e, shift), f = __builtin_fma(x, log2e, shift - r);
  double v = __builtin_fma(f, 7.1117595466171784e-09, 1.0210506490815314e-07);
  v = __builtin_fma(f, v, 1.3215235630301141e-06);
  v = __builtin_fma(f, v, 1.5252647747511752e-05);
  v = __builtin_fma(f, v, 0.0001540353080082534);
  v = __builtin_fma(f, v, 0.001333355824648106);
  v = __builtin_fma(f, v, 0.009618129107380713);
  v = __builtin_fma(f, v, 0.05550410866434658);
  v = __builtin_fma(f, v, 0.24022650695910472);
  v = __builtin_fma(f, v, 0.6931471805599516);
  v = __builtin_fma(f, v, 1.0);
  u32x2 b = __builtin_bit_cast(u32x2, v);
  b.y += __builtin_bit_cast(u32x2, r).x << 20;
  return __builtin_bit_cast(double, b);
}
// exp(x - most) for x <= most; 1e-300, which adds nothing, for what is masked (-infinity
// or NaN) or much smaller.
__device__ __forceinline__ double exp_below(double x, double most) {
  return exp_64(__builtin_fmax(x - most, -690.0));
}

// All lanes' sum and maximum, in every lane.
__device__ __forceinline__ double wave_sum(double v) {
  return readlane(wave_scan_incl<Op::Add>(v), 63);
}
__device__ __forceinline__ float wave_max(float v) {
  return readlane(wave_scan_incl<Op::Max>(v), 63);
}

// The ranks of n entries of `list` by `threads` threads, added up in `rank`, which is
// zero: several threads an entry where there are fewer entries than threads.  The
// caller waits before it reads them.
template <class T>
__device__ __forceinline__ void add_ranks(const T* list, uint32_t* rank, uint32_t n, uint32_t threads) {
  uint32_t wide = 32;
  while (wide < n && wide < threads) wide *= 2;
  const uint32_t parts = threads / wide, part = threadIdx.x / wide;
  for (uint32_t i = threadIdx.x % wide; i < n; i += wide) {
    const T mine = list[i];
    uint32_t above = 0;
#pragma unroll 4
    for (uint32_t k = part; k < n; k += parts) above += list[k] > mine ? 1u : 0u;
    if (above != 0)
      __hip_atomic_fetch_add(&rank[i], above, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  }
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
  return t;
}
// Two bounds for the `count` greatest of a segment, from its waves' lanes: a wave in
// which `count` lanes reach a value gives one alone; the least of what a quarter of them
// reach in each of the four gives another.  The greater holds: as a rule the second,
// which leaves some 20 entries for 16 (the first 50); where all that is great lies in one
// wave the first.  The low bits of the keys are left out as far as a 16-bit type has
// none (its keys end in zeros, below 0 in ones), and in float32 the last 12.
struct Bounds { uint32_t alone, together; };
template <class F>
__device__ __forceinline__ Bounds lanes_bounds(uint32_t key, int count) {
  constexpr int LOW = std::is_same_v<F, FmtBF16> ? 16 : (std::is_same_v<F, FmtF16> ? 13 : 12);
  constexpr uint32_t ones = sizeof(typename F::S) == 2 ? (1u << LOW) - 1 : 0;
  const uint32_t t = lanes_bound<LOW>(key, count), u = lanes_bound<LOW>(key, (count + kBeamWaves - 1) / kBeamWaves);
  return Bounds{(t >> 31) ? t : t | ones, (u >> 31) ? u : u | ones};
}
__device__ __forceinline__ uint32_t joint_bound(const Bounds* waves) {
  uint32_t alone = waves[0].alone, together = waves[0].together;
#pragma unroll
  for (int w = 1; w < kBeamWaves; ++w) {
    alone = alone > waves[w].alone ? alone : waves[w].alone;
    together = together < waves[w].together ? together : waves[w].together;
  }
  return alone > together ? alone : together;
}

// Of a segment: its greatest logit, and its sum of exp(l - most); of +infinity, how many
// logits are that.
struct Found {
  float most;
  double sum;
};

struct SegmentShared {
  uint64_t by_wave[kBeamWaves][kListed / kBeamWaves], list[kListed];
  uint32_t rank[kListed];
  double sum[kBeamWaves];
  float most[kBeamWaves];
  Bounds bound[kBeamWaves];
  uint32_t part[kBeamWaves], listed[kBeamWaves];
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

// A segment: `length` vectors of 16 bytes, at most 256 NV.  Entries are (order_key << 32
// | ~token), so that the greater entry comes first; 0 is none.
//
// 32 x 8 rows of 50000 bfloat16 logits, count 16: 20 us, of which some 7 the 64-bit
// exponentials (19 instructions a logit) and 4 the choice; the vector units are 69% busy.
// 128 x 4 rows in float32, a fifth of them finished: 28.5 us, 2.9 TB/s.  (Exponentials of the
// logits as they are, with 4 instructions fewer, took 17.2 and 25, but a row plus a constant
// had another sum.  Relative to a wave's maximum, before the barrier, 19.8 and 28.8.)
template <class F, int NV>
__global__ __launch_bounds__(kBeamThreads) void beam_segment_kernel(BeamProblem p, uint64_t* best,
                                                                   Found* found, int64_t row0,
                                                                   int64_t segments, int64_t length) {
  using S = typename F::S;
  constexpr int E = kVecElems<F>;
  __shared__ SegmentShared sh;
  const int wave = wave_id(), tid = (int)threadIdx.x, count = (int)p.count;
  int64_t seg, j;
  const int64_t row = row0 + divide((int64_t)blockIdx.x, segments, &seg);
  const int64_t b = divide(row, p.beams, &j);
  if (p.finished != nullptr && p.finished[row] != 0) return;     // none of its logits is asked for
  const S* logits = (const S*)p.logits + b * p.logits_batch + j * p.logits_beam;
  // The row's last vector ends with it and may begin among those of the one before,
  // which are left out.  What a thread adds up depends on the vocabulary alone, not
  // on where the row lies: equal rows have equal sums.
  // (below 2^31 logits and a segment more: 32 bits without a sign)
  const uint32_t vocab = (uint32_t)p.vocab;
  const uint32_t s0 = (uint32_t)(seg * length), v0 = s0 + (uint32_t)tid, vend = s0 + (uint32_t)length;
  const bool whole = vocab >= E;
  auto begin = [&](uint32_t vec) { return whole && vec * E < vocab - E ? vec * E : vocab - E; };
  using IO = RowIO<F, E>;
  u32x4 raw[NV];                             // as they are: 16-bit logits two to a register
  if (whole) {
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = IO::load_any(logits + begin(v0 + i * kBeamThreads), E);
  } else {                                   // less than a vector: the first thread's
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[e] = -__builtin_huge_valf();
        if (i == 0 && tid == 0 && e + (int)vocab >= E) v[e] = widen<F>(logits[e + (int)vocab - E]);
      }
      raw[i] = IO::pack(v);
    }
  }
  // Vector i's logits.  A NaN is smaller and greater than nothing and equal to nothing,
  // so that it counts for nothing below.
  auto values = [&](int i, float (&v)[E]) {
    uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) materialize(w[k]);         // unpacked each time, not kept so
    raw[i] = u32x4{w[0], w[1], w[2], w[3]};
    IO::unpack(raw[i], v);
  };
  float most = -__builtin_huge_valf();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[E];
    const uint32_t vec = v0 + i * kBeamThreads, skip = vec < vend ? vec * E - begin(vec) : E;
    if (skip > 0 && whole) {
      IO::unpack(raw[i], v);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = (uint32_t)e >= skip ? v[e] : -__builtin_huge_valf();
      raw[i] = IO::pack(v);
    }
    values(i, v);
#pragma unroll
    for (int e = 0; e < E; ++e) most = __builtin_elementwise_maximum(most, v[e]);
    // vector after vector: each when it is there, with the registers of one
    __builtin_amdgcn_sched_barrier(0);
  }
  // (that maximum is NaN wherever an operand is; one that passes NaNs over would need the
  // signalling ones made quiet first, an instruction more a logit)
  if (__ballot(most != most) != 0) {
    most = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[E];
      values(i, v);
#pragma unroll
      for (int e = 0; e < E; ++e) most = v[e] > most ? v[e] : most;
    }
  }
  const uint32_t mine = order_key(most);
  const Bounds bound = lanes_bounds<F>(mine, count);
  const float wmost = wave_max(most);
  if (lane_id() == 0) {
    sh.most[wave] = wmost;
    sh.bound[wave] = bound;
  }
  __syncthreads();
  float top = sh.most[0];
  uint32_t least = joint_bound(sh.bound);
#pragma unroll
  for (int w = 1; w < kBeamWaves; ++w) top = __builtin_fmaxf(top, sh.most[w]);
  uint64_t* out = best + (row * segments + seg) * count;
  if (top == -__builtin_huge_valf()) {                           // all masked
    if (tid < count) out[tid] = 0;
    if (tid == 0) found[row * segments + seg] = Found{top, 0.0};
    return;
  }
  // what is above the bound, then what is equal to it
  least = least > kMaskedKey ? least : kMaskedKey + 1;
  // What is chosen is first held as its value and where it lies (the thread, and which
  // of its logits), a few instructions each; the entry is made of that by a lane each.
  auto hold = [&](int ie, float v) {
    return ((uint64_t)__builtin_bit_cast(uint32_t, v) << 32) | ((uint32_t)ie * kBeamThreads + (uint32_t)tid);
  };
  auto entry = [&](uint64_t held) {
    const uint32_t at = (uint32_t)held, ie = at / kBeamThreads;
    const uint32_t vec = s0 + at % kBeamThreads + ie / E * kBeamThreads;
    const uint32_t token = begin(vec) + ie % E;
    return ((uint64_t)order_key(__builtin_bit_cast(float, (uint32_t)(held >> 32))) << 32) | (uint32_t)~token;
  };
  float edge = key_value(least);
  // each wave lists what is above the edge for itself; n: how many there were
  auto above = [&](int i, const float (&v)[E], uint32_t& n) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint64_t on = __ballot(v[e] > edge);
      if (on == 0) continue;
      const uint32_t k = n + (uint32_t)__builtin_popcountll(on & ((1ull << lane_id()) - 1));
      if (v[e] > edge && k < (uint32_t)(kListed / kBeamWaves)) sh.by_wave[wave][k] = hold(i * E + e, v[e]);
      n += (uint32_t)__builtin_popcountll(on);
    }
  };
  // the exponentials and the list, in one walk
  const bool some = wmost > edge;
  uint32_t listed = 0;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[E];
    values(i, v);
#pragma unroll
    for (int e = 0; e < E; ++e) sum += exp_below((double)v[e], (double)top);
    materialize(sum);
    __builtin_amdgcn_sched_barrier(0);
    if (some) above(i, v, listed);
  }
  if (top == __builtin_huge_valf()) {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[E];
      values(i, v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += v[e] == top ? 1.0 : 0.0;
    }
  }
  sum = wave_sum(sum);
  if (lane_id() == 0) {
    sh.sum[wave] = sum;
    sh.listed[wave] = listed;
  }
  __syncthreads();
  if (tid == 0) {
    double all = sh.sum[0];
#pragma unroll
    for (int w = 1; w < kBeamWaves; ++w) all += sh.sum[w];
    found[row * segments + seg] = Found{top, all};
  }
  bool over = false;
#pragma unroll
  for (int w = 0; w < kBeamWaves; ++w) over |= sh.listed[w] > (uint32_t)(kListed / kBeamWaves);
  if (over) {
    // too much above the bound (great logits side by side): the count-th greatest
    // itself, bit by bit
    uint32_t t = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = t | (1u << bit);
      const float low = key_value(c > kMaskedKey ? c : kMaskedKey + 1);
      uint32_t k = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[E];
        values(i, v);
#pragma unroll
        for (int e = 0; e < E; ++e) k += v[e] >= low ? 1u : 0u;
      }
      if (group_sum(k, sh, wave) >= (uint32_t)count) t = c;
    }
    edge = key_value(t > kMaskedKey ? t : kMaskedKey + 1);
    listed = 0;                              // fewer than `count`
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[E];
      values(i, v);
      above(i, v, listed);
    }
    __syncthreads();
    if (lane_id() == 0) sh.listed[wave] = listed;
    __syncthreads();
  }
  uint32_t n = 0, place = 0;                 // the waves' lists, one behind the other
#pragma unroll
  for (int w = 0; w < kBeamWaves; ++w) {
    place += w < wave ? sh.listed[w] : 0;
    n += sh.listed[w];
  }
  if (n >= (uint32_t)count && n <= 64) {
    // as a rule: one wave ranks an entry a lane, the others are done
    if (wave != 0) return;
    uint32_t k = (uint32_t)lane_id(), w = 0;
#pragma unroll
    for (int i = 0; i + 1 < kBeamWaves; ++i) {
      const bool beyond = w == (uint32_t)i && k >= sh.listed[i];
      k -= beyond ? sh.listed[i] : 0;
      w += beyond ? 1 : 0;
    }
    const uint64_t own = (uint32_t)lane_id() < n ? entry(sh.by_wave[w][k]) : 0;
    uint32_t rank = 0;
    for (uint32_t i = 0; i < n; ++i) rank += readlane(own, (int)i) > own ? 1u : 0u;
    if ((uint32_t)lane_id() < n && rank < (uint32_t)count) out[rank] = own;
    return;
  }
  for (uint32_t i = lane_id(); i < listed; i += 64) sh.list[place + i] = entry(sh.by_wave[wave][i]);
  for (int i = tid; i < kListed; i += kBeamThreads) sh.rank[i] = 0;
  if (n < (uint32_t)count) {
    // those equal to the bound, in token order, as many as are asked for
    uint32_t open = (uint32_t)count - n, taken = n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[E];
      values(i, v);
      uint32_t k = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) k += v[e] == edge ? 1u : 0u;
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
        if (v[e] == edge) {
          if (before < open) sh.list[taken + before] = entry(hold(i * E + e, v[e]));
          ++before;
        }
      const uint32_t got = all < open ? all : open;
      taken += got;
      open -= got;
    }
    n = taken;
  }
  __syncthreads();
  add_ranks(sh.list, sh.rank, n, kBeamThreads);
  __syncthreads();
  for (uint32_t i = tid; i < n; i += kBeamThreads)
    if (sh.rank[i] < (uint32_t)count) out[sh.rank[i]] = sh.list[i];
  if (tid >= (int)n && tid < count) out[tid] = 0;
}

namespace {

// A candidate in the order of the choice: score, lower beam, greater logit, lower token.
struct Candidate {
  uint64_t score;                            // order_key64; 0 is none
  uint64_t entry;
  uint32_t beam;
};
__device__ __forceinline__ bool operator>(const Candidate& a, const Candidate& b) {
  if (a.score != b.score) return a.score > b.score;
  if (a.beam != b.beam) return a.beam < b.beam;
  return a.entry > b.entry;
}

struct JoinShared {
  Candidate list[kJoined];
  uint32_t rank[kJoined];
  double lse[64];                            // log of the sum of exp(logit - most)
  float most[64], score[64];
  bool done[64];
  uint32_t bound[kJoinWaves];
  uint32_t listed;
  Candidate wave_best[kJoinWaves];
};

}  // namespace

// A workgroup a batch entry: 5 us for one of 4 beams and 12 segments, 6.5 for 32 of 8
// beams and 5 segments; latency, as three steps read what the one before found.
__global__ __launch_bounds__(kJoinThreads) void beam_join_kernel(BeamProblem p, const uint64_t* best,
                                                                 const Found* found, float* scores,
                                                                 int32_t* parents, int32_t* tokens,
                                                                 int64_t b0, int64_t segments) {
  __shared__ JoinShared sh;
  const int wave = wave_id(), tid = (int)threadIdx.x, count = (int)p.count, beams = (int)p.beams;
  const int64_t b = b0 + blockIdx.x, row0 = b * beams;
  const int64_t per = segments * count, total = per * beams;
  // a thread's first candidates, read while the beams' sums are joined
  constexpr int R = 4;
  uint64_t held[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = tid + r * kJoinThreads;
    held[r] = best[row0 * per + (i < total ? i : total - 1)];
  }
  if (tid == 0) sh.listed = 0;
  for (int i = tid; i < kJoined; i += kJoinThreads) sh.rank[i] = 0;
  for (int j = wave; j < beams; j += kJoinWaves) {
    // (a finished beam's segments hold nothing, and are read all the same: their loads
    // need not wait for the mark's)
    const Found* f = found + (row0 + j) * segments;
    const Found own = f[lane_id() < segments ? lane_id() : 0];
    const float score = p.scores[row0 + j];
    const bool done = p.finished != nullptr && p.finished[row0 + j] != 0;
    float most = own.most;
    for (int64_t s = lane_id() + 64; s < segments; s += 64) most = __builtin_fmaxf(most, f[s].most);
    most = wave_max(most);
    auto part = [&](const Found& v) {
      return v.most == most ? v.sum : v.sum * exp_below((double)v.most, (double)most);
    };
    double sum = lane_id() < segments ? part(own) : 0.0;
    for (int64_t s = lane_id() + 64; s < segments; s += 64) sum += part(f[s]);
    sum = wave_sum(sum);
    if (lane_id() == 0) {
      sh.most[j] = most;
      sh.lse[j] = log(sum);
      sh.score[j] = score;
      sh.done[j] = done;
    }
  }
  __syncthreads();
  // candidate i of the batch entry, whose entry is known
  auto candidate = [&](int64_t i, uint64_t entry) {
    int64_t k;
    const int j = (int)divide(i, per, &k);
    Candidate c{0, entry, (uint32_t)j};
    const double base = (double)sh.score[j];
    double s;
    if (sh.done[j]) {
      if (k != 0) return c;
      c.entry = (uint32_t)~(uint32_t)p.end_token;
      s = base;
    } else {
      if (entry == 0) return c;
      const float l = key_value((uint32_t)(entry >> 32)), m = sh.most[j];
      // (beside an infinite logit only such have a chance)
      s = base + ((l == m ? 0.0 : (double)l - (double)m) - sh.lse[j]);
    }
    if (s > -__builtin_huge_val()) c.score = order_key64(s);      // (no NaN)
    return c;
  };
  uint64_t mine = 0, first[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = tid + r * kJoinThreads;
    first[r] = i < total ? candidate(i, held[r]).score : 0;
    mine = mine > first[r] ? mine : first[r];
  }
  for (int64_t i = tid + R * kJoinThreads; i < total; i += kJoinThreads) {
    const uint64_t s = candidate(i, best[row0 * per + i]).score;
    mine = mine > s ? mine : s;
  }
  const uint32_t bound = lanes_bound<12>((uint32_t)(mine >> 32), count);
  if (lane_id() == 0) sh.bound[wave] = bound;
  __syncthreads();
  uint32_t least = 1;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) least = least > sh.bound[w] ? least : sh.bound[w];
  auto list = [&](const Candidate& c) {
    const uint32_t k = __hip_atomic_fetch_add(&sh.listed, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    if (k < (uint32_t)kJoined) sh.list[k] = c;
  };
  if ((uint32_t)(mine >> 32) >= least) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if ((uint32_t)(first[r] >> 32) >= least) list(candidate(tid + r * kJoinThreads, held[r]));
    for (int64_t i = tid + R * kJoinThreads; i < total; i += kJoinThreads) {
      const Candidate c = candidate(i, best[row0 * per + i]);
      if ((uint32_t)(c.score >> 32) >= least) list(c);
    }
  }
  __syncthreads();
  uint32_t n = sh.listed;
  if (n > (uint32_t)kJoined) {
    // too many: one after the other, the best of those behind the one before
    Candidate last{~0ull, ~0ull, 0};
    n = 0;
    for (int k = 0; k < count; ++k) {
      Candidate top{0, 0, 0};
      for (int64_t i = tid; i < total; i += kJoinThreads) {
        const Candidate c = candidate(i, best[row0 * per + i]);
        if (c.score != 0 && last > c && c > top) top = c;
      }
      for (int m = 32; m > 0; m /= 2) {
        const Candidate o{__shfl_xor((unsigned long long)top.score, m),
                          __shfl_xor((unsigned long long)top.entry, m),
                          (uint32_t)__shfl_xor((int)top.beam, m)};
        if (o > top) top = o;
      }
      __syncthreads();
      if (lane_id() == 0) sh.wave_best[wave] = top;
      __syncthreads();
      top = sh.wave_best[0];
      for (int w = 1; w < kJoinWaves; ++w)
        if (sh.wave_best[w] > top) top = sh.wave_best[w];
      if (top.score == 0) break;
      if (tid == 0) sh.list[n] = top;
      ++n;
      last = top;
    }
    __syncthreads();
  }
  add_ranks(sh.list, sh.rank, n, kJoinThreads);
  __syncthreads();
  const int64_t out = b * count;
  for (uint32_t i = tid; i < n; i += kJoinThreads) {
    const Candidate c = sh.list[i];
    const uint32_t rank = sh.rank[i];
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

// How rows are cut: segments of equal length, at most 8 vectors a thread.  A
// workgroup costs what 2 (float32: 4) vectors a thread cost beside its own, and a CU
// goes through its workgroups one after the other as far as arithmetic is concerned,
// the first few waits apart.  So a few rows are cut fine, for the whole chip, many
// rows coarse, where their length fits whole vectors best: 256 rows of 50000 in
// bfloat16 take 5 segments of 1250.
struct Cut { int64_t segments, length; int vectors; };
template <class F> Cut beam_cut(const BeamProblem& p) {
  const int64_t vecs = (p.vocab + kVecElems<F> - 1) / kVecElems<F>, rows = p.batch * p.beams;
  const int64_t least = (vecs + 8 * kBeamThreads - 1) / (8 * kBeamThreads);
  const int64_t most = (vecs + kBeamThreads - 1) / kBeamThreads;
  constexpr int64_t own = sizeof(typename F::S) == 4 ? 4 : 2;
  Cut best{};
  int64_t lowest = 0;
  for (int64_t s = least; s <= most; ++s) {
    const int64_t length = (vecs + s - 1) / s, nv = (length + kBeamThreads - 1) / kBeamThreads;
    const int64_t cost = (own + nv) * ((rows * s + 255) / 256 + 4);
    if (best.segments == 0 || cost < lowest) {
      best = Cut{(vecs + length - 1) / length, length, (int)nv};
      lowest = cost;
    }
    if (s >= least + 64 && s < most) s = most - 1;     // (a very long row: no need to look at all)
  }
  return best;
}

template <class F, int NV>
hipError_t launch_segments(const BeamProblem& p, uint64_t* best, Found* found, int64_t segments,
                           int64_t length, hipStream_t stream) {
  const int64_t rows = p.batch * p.beams, most = (1ll << 22) / segments, step = most < 1 ? 1 : most;
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t n = rows - r < step ? rows - r : step;
    beam_segment_kernel<F, NV><<<dim3((unsigned)(n * segments)), dim3(kBeamThreads), 0, stream>>>(
        p, best, found, r, segments, length);
  }
  return hipGetLastError();
}

template <class F> size_t beam_scratch_f(const BeamProblem& p) {
  const size_t segs = (size_t)(p.batch * p.beams) * (size_t)beam_cut<F>(p).segments;
  return segs * (sizeof(Found) + 8 * (size_t)p.count);
}

template <class F>
hipError_t launch_beam_f(const BeamProblem& p, float* scores, int32_t* parents, int32_t* tokens,
                         void* scratch, hipStream_t stream) {
  const Cut cut = beam_cut<F>(p);
  const int64_t segments = cut.segments;
  Found* found = (Found*)scratch;
  uint64_t* best = (uint64_t*)(found + p.batch * p.beams * segments);
  hipError_t e;
  switch (cut.vectors) {
    case 8: e = launch_segments<F, 8>(p, best, found, segments, cut.length, stream); break;
    case 7: e = launch_segments<F, 7>(p, best, found, segments, cut.length, stream); break;
    case 6: e = launch_segments<F, 6>(p, best, found, segments, cut.length, stream); break;
    case 5: e = launch_segments<F, 5>(p, best, found, segments, cut.length, stream); break;
    case 4: e = launch_segments<F, 4>(p, best, found, segments, cut.length, stream); break;
    case 3: e = launch_segments<F, 3>(p, best, found, segments, cut.length, stream); break;
    case 2: e = launch_segments<F, 2>(p, best, found, segments, cut.length, stream); break;
    default: e = launch_segments<F, 1>(p, best, found, segments, cut.length, stream); break;
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
// them a launch).  8 layers' states of 32 x 8 beams, 587 MB: 164 us with 339 MB read
// (each parent's row once, in however many beams it goes on), 5.6 TB/s.
// ---------------------------------------------------------------------------
namespace {

constexpr int kMoved = 64;                   // tensors a launch
#ifndef SCA_REORDER_BLOCKS
#define SCA_REORDER_BLOCKS (1ll << 23)
#endif
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
template <bool PAST, class V> __device__ __forceinline__ void store_loose(uintptr_t a, V v) {
  typedef V Loose __attribute__((aligned(1)));
  if constexpr (PAST) {
    __builtin_nontemporal_store(v, gptr<Loose>(a));
  } else {
    *gptr<Loose>(a) = v;
  }
}

// States that the 256 MB last-level cache cannot hold are stored past the caches: 587
// MB of new states 164 us, by other stores 172.
inline bool states_past_caches(int64_t bytes) { return bytes > (256ll << 20); }

template <int NB, bool PAST, class V>
__device__ __forceinline__ void move_column(uintptr_t from, uintptr_t to, int64_t bytes, const int* parent,
                                            uint64_t moves) {
  // (every load is issued: a register that only a branch writes costs many more)
  V v[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) v[j] = load_loose<V>(from + (uintptr_t)(parent[j] * bytes));
#pragma unroll
  for (int j = 0; j < NB; ++j)
    if ((moves >> j) & 1) store_loose<PAST, V>(to + (uintptr_t)(j * bytes), v[j]);
}

}  // namespace

template <int NB, class V, bool PAST>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4, 8)))
void beam_reorder_kernel(Moves m, const int32_t* parents, int64_t b0, uint32_t first, uint32_t blocks,
                         int beams) {
  // blocks: of a batch entry in this launch, from the first one on
  int64_t block;
  const int64_t b = b0 + divide((int64_t)blockIdx.x, blocks, &block);
  block += first;
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
    move_column<NB, PAST, V>(from + (uintptr_t)col * sizeof(V), to + (uintptr_t)col * sizeof(V), bytes, parent, moves);
  } else if (col - whole < bytes % (int64_t)sizeof(V)) {         // a row's last bytes, one a thread
    const uintptr_t at = (uintptr_t)(whole * (int64_t)sizeof(V) + (col - whole));
    move_column<NB, PAST, uint8_t>(from + at, to + at, bytes, parent, moves);
  }
}

template <int NB, class V>
static hipError_t launch_moves(const void* const* states, void* const* new_states, const int64_t* row_bytes,
                               int64_t tensors, const int32_t* parents, int64_t batch, int64_t beams,
                               hipStream_t stream) {
  // Workgroups of a launch: 2^31 threads, where an axis ends at 2^32.  A longer row (32 GB)
  // goes out in several launches: no column reads what another writes, in place either.
  constexpr int64_t kMostBlocks = SCA_REORDER_BLOCKS;
  int64_t all = 0;
  for (int64_t t = 0; t < tensors; ++t) all += batch * beams * row_bytes[t];
  const bool past = states_past_caches(all);
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
      for (int64_t first = 0; first < blocks; first += kMostBlocks) {
        const int64_t part = blocks - first < kMostBlocks ? blocks - first : kMostBlocks;
        const dim3 grid((unsigned)(n * part));
        if (past)
          beam_reorder_kernel<NB, V, true><<<grid, dim3(256), 0, stream>>>(m, parents, b, (uint32_t)first,
                                                                           (uint32_t)part, (int)beams);
        else
          beam_reorder_kernel<NB, V, false><<<grid, dim3(256), 0, stream>>>(m, parents, b, (uint32_t)first,
                                                                            (uint32_t)part, (int)beams);
      }
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
