// Token embedding, out[i] = scale * weight[ids[i]], and the gradient of its
// table, dweight[v] = scale * sum over the tokens i with ids[i] = v of dout[i].
// Ids outside [0, rows) stand for masked tokens: their output is zero and they
// add to no row.
//
// The gradient sorts the tokens by id (the library's radix sort, stable), so
// that each table row is the sum of one run of sorted tokens, taken in token
// order: no float atomics, the same bits every time.  The sorted tokens are cut
// into segments; a wave sums the runs of its segment (one table column
// block), writes the rows whose run lies inside, and leaves the sums of runs
// that cross a border to a second kernel.
//
// Both directions are bound by memory.  Measured, bf16, 16384 tokens with a
// language's frequencies, a table of 50000 x 2048: lookup of the 5850 rows that
// occur (91 MB) 17 us, 23 where no cache holds any of them; gradient (272 MB) 70
// us: 44 us for sort and zeros, 19 for the segments, 9 for the borders.  Gradients
// past the short sort's limit: 16385 tokens 134 us, 32768 149 (339 MB), 131072 265
// (743 MB), 524288 703 (2.4 GB).
#include "sequence.hpp"

namespace sca {

namespace {

template <class I>
__device__ __forceinline__ int64_t token_row(const I* ids, int64_t i, int64_t rows) {
  const int64_t v = (int64_t)ids[i];
  return v >= 0 && v < rows ? v : -1;
}

}  // namespace

template <class F, int E, bool ALIGNED, bool PAST, class I>
__global__ __launch_bounds__(256) void embedding_kernel(const void* weight, const I* ids,
                                                       void* out, int64_t tokens, int64_t rows,
                                                       int64_t channels, int64_t row_stride,
                                                       float scale) {
  using S = typename F::S;
  using IO = RowIO<F, E>;
  const int64_t vecs = (channels + E - 1) / E, total = tokens * vecs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / vecs, ch = i % vecs * E;
    const int64_t row = token_row(ids, t, rows);
    typename IO::Raw r{};
    if (row >= 0) {
      float v[E];
      IO::unpack(IO::template get<ALIGNED>((const S*)weight + row * row_stride + ch, channels - ch), v);
#pragma unroll
      for (int c = 0; c < E; ++c) v[c] *= scale;
      r = IO::pack(v);
    }
    if constexpr (ALIGNED) {
      IO::template store_past<PAST>((S*)out + t * channels + ch, r);
    } else {
      IO::store_any((S*)out + t * channels + ch, r, channels - ch);
    }
  }
}

// Sort keys and positions; a masked token gets the key `rows`, past every row.
template <class I>
__global__ __launch_bounds__(256) void embedding_keys_kernel(const I* ids, int64_t tokens,
                                                            int64_t rows, uint32_t* keys,
                                                            uint32_t* pos) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= tokens) return;
  const int64_t row = token_row(ids, i, rows);
  keys[i] = (uint32_t)(row < 0 ? rows : row);
  pos[i] = (uint32_t)i;
}

__global__ __launch_bounds__(256) void embedding_zero_kernel(uint4* out, int64_t vecs, uint8_t* tail,
                                                            int tail_bytes) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < vecs; i += step)
    __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, gptr<u32x4>((uintptr_t)(out + i)));
  if (blockIdx.x == 0 && (int)threadIdx.x < tail_bytes) tail[threadIdx.x] = 0;
}

// The whole gradient of a very short list in one launch, where launches cost
// more than the work.  Every wave holds all ids in registers, one per lane of
// kFewIds registers; it owns 64 E channels of the rows r, r + step, ... (step
// apart, so that the rows of frequent tokens, which lie together, are on
// different waves), finds a row's tokens by ballots, and adds them in token
// order, 16 loads at a time.  For up to 256 tokens: the longest run, all of them in
// one row, is then 16 groups of loads (256 ids of a 3000 x 800 bf16 table: 8.8 us
// against 17.2 the other way with a language's frequencies, 22 against 17 all in
// one row).
constexpr int kFewIds = 4;
constexpr int64_t kFewTokens = 64 * kFewIds;

template <class F, class G, int E, bool ALIGNED, class I>
__global__ __launch_bounds__(256) void embedding_few_kernel(const void* dout, const I* ids,
                                                           void* dweight, int tokens, int64_t rows,
                                                           int64_t channels, int64_t row_stride,
                                                           float scale, uint32_t cols, uint32_t step) {
  using S = typename F::S;
  using IO = RowIO<F, E>;
  constexpr int OE = E < kVecElems<G> ? E : kVecElems<G>;
  using OIO = RowIO<G, OE>;
  constexpr int kAhead = 16;
  const int lane = lane_id();
  const uint32_t wave = blockIdx.x * 4 + (uint32_t)wave_id();
  const int64_t ch = ((int64_t)(wave % cols) * 64 + lane) * E;
  uint32_t key[kFewIds];                 // masked tokens: no row
#pragma unroll
  for (int k = 0; k < kFewIds; ++k)
    key[k] = k * 64 + lane < tokens ? (uint32_t)token_row(ids, k * 64 + lane, rows) : ~0u;
  const bool live = ch < channels;
  if (wave >= step * cols) return;
  for (uint64_t row = wave / cols; row < (uint64_t)rows; row += step) {
    float sum[E] = {};
#pragma unroll
    for (int k = 0; k < kFewIds; ++k) {
      uint64_t left = __ballot(key[k] == (uint32_t)row);
      while (left != 0) {
        typename IO::Raw raw[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          raw[j] = typename IO::Raw{};
          if (left == 0) continue;
          const int64_t i = k * 64 + __builtin_ctzll(left);
          left &= left - 1;
          if (live)
            raw[j] = IO::template get<ALIGNED>((const S*)dout + i * row_stride + ch, channels - ch);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          float v[E];
          IO::unpack(raw[j], v);
#pragma unroll
          for (int c = 0; c < E; ++c) sum[c] += v[c];     // past the last token: + 0
        }
      }
    }
    if (!live) continue;
    typename G::S* to = (typename G::S*)dweight + (int64_t)row * channels + ch;
#pragma unroll
    for (int h = 0; h < E; h += OE) {
      float o[OE];
#pragma unroll
      for (int c = 0; c < OE; ++c) o[c] = sum[h + c] * scale;
      if (ALIGNED || h < channels - ch)
        OIO::template put<ALIGNED>(to + h, OIO::pack(o), channels - ch - h);
    }
  }
}

// The sort of a short list, in one launch.  A workgroup owns `bucket` (at most
// 256) table rows and reads all ids: those below its rows tell where its part
// of the sorted list begins, so workgroups need nothing of one another.  It
// counts its rows per wave (a wave owns consecutive tokens) and places its
// tokens in token order.  It also writes zeros to its rows: the segments'
// kernel overwrites those that have a token, which costs less than waiting for
// the counts before the first store (the barriers between wait
// for LDS alone).  Every id is read by every workgroup, from
// L2: 64 MB for 16384 ids and 512 workgroups, against the four passes over the
// list and the seven launches of the general path.
constexpr int kBucketRows = 256;
constexpr int kBucketWaves = 16;
constexpr int kBucketIds = 16;           // ids per lane
constexpr int64_t kBucketTokens = 64 * kBucketWaves * kBucketIds;

// The workgroup's threads write zeros to [a, e), whose ends are multiples of
// `unit` (2 or 4) bytes.
__device__ __forceinline__ void zero_span(uintptr_t a, uintptr_t e, int unit) {
  const uintptr_t a16 = (a + 15) & ~(uintptr_t)15;
  const uintptr_t lo = a16 < e ? a16 : e, hi = lo + ((e - lo) & ~(uintptr_t)15);
  const uintptr_t t = threadIdx.x;
  for (uintptr_t i = lo + t * 16; i < hi; i += 64 * kBucketWaves * 16)
    __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, gptr<u32x4>(i));
  const uintptr_t head = a + t * unit, tail = hi + t * unit;
  if (unit == 4) {
    if (head < lo) *gptr<uint32_t>(head) = 0;
    if (tail < e) *gptr<uint32_t>(tail) = 0;
  } else {
    if (head < lo) *gptr<uint16_t>(head) = 0;
    if (tail < e) *gptr<uint16_t>(tail) = 0;
  }
}

template <class I>
__global__ __launch_bounds__(64 * kBucketWaves) void embedding_bucket_kernel(
    const I* ids, int tokens, int64_t rows, int bucket, uint32_t* __restrict__ keys,
    uint32_t* __restrict__ pos, char* __restrict__ dweight,
    int64_t row_bytes, int unit) {
  __shared__ uint32_t s_off[kBucketWaves][kBucketRows];
  __shared__ uint32_t s_start[kBucketRows];
  __shared__ uint32_t s_below[kBucketWaves], s_sum[kBucketRows / 64];
  const int lane = lane_id(), wave = wave_id();
  const uint32_t lo = blockIdx.x * (uint32_t)bucket;      // rows are at most 2^17 here
  const int its = (tokens + 64 * kBucketWaves - 1) / (64 * kBucketWaves);
  const int first = wave * its * 64 + lane;
  constexpr uint32_t kNone = ~0u;
  uint32_t rel[kBucketIds];              // row within the bucket
  uint32_t below = 0;
#pragma unroll
  for (int b = 0; b < kBucketRows; b += 64) s_off[wave][b + lane] = 0;
  uint32_t row[kBucketIds];              // masked tokens are above every row
#pragma unroll
  for (int k = 0; k < kBucketIds; ++k) {
    const int i = first + k * 64;
    row[k] = k < its && i < tokens ? (uint32_t)token_row(ids, i, rows) : kNone;
  }
  // half of the workgroups write their zeros before the sort, half after it, so
  // that some always keep the memory busy
  auto clear = [&]() {
    const int64_t left = rows - lo, mine = left < bucket ? left : bucket;
    const uintptr_t a = (uintptr_t)dweight + (uintptr_t)(lo * row_bytes);
    zero_span(a, a + (uintptr_t)(mine * row_bytes), unit);
  };
  const bool late = blockIdx.x / 8 % 2 != 0;
  if (!late) clear();
#pragma unroll
  for (int k = 0; k < kBucketIds; ++k) {
    below += (uint32_t)__popcll(__ballot(row[k] < lo));
    rel[k] = row[k] - lo < (uint32_t)bucket ? row[k] - lo : kNone;
    if (rel[k] != kNone) atomicAdd(&s_off[wave][rel[k]], 1u);
  }
  if (lane == 0) s_below[wave] = below;
  lds_barrier();
  uint32_t count = 0, incl = 0;
  if (threadIdx.x < kBucketRows) {
    // per row: where each wave's tokens begin among the row's, and their number
#pragma unroll
    for (int w = 0; w < kBucketWaves; ++w) {
      const uint32_t v = s_off[w][threadIdx.x];
      s_off[w][threadIdx.x] = count;
      count += v;
    }
    incl = wave_scan_incl<Op::Add>(count);
    if (lane == kWave - 1) s_sum[wave] = incl;
  }
  lds_barrier();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kBucketWaves; ++w) base += s_below[w];
#pragma unroll
  for (int w = 0; w < kBucketRows / 64; ++w) {
    if (threadIdx.x < kBucketRows && w < wave) incl += s_sum[w];
    all += s_sum[w];
  }
  if (threadIdx.x < kBucketRows) s_start[threadIdx.x] = base + incl - count;
  lds_barrier();

#pragma unroll
  for (int k = 0; k < kBucketIds; ++k) {
    const uint32_t r = rel[k];
    const bool on = r != kNone;
    uint64_t same = __ballot(on);
    if (same == 0) continue;
    // lanes with the same row
#pragma unroll
    for (int bit = 0; bit < 8; ++bit) {
      const uint64_t set = __ballot((r >> bit & 1) != 0);
      same &= (r >> bit & 1) != 0 ? set : ~set;
    }
    if (on) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      uint32_t* mine = &s_off[wave][r];
      const uint32_t before = __hip_atomic_load(mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
      const uint32_t at = s_start[r] + before + rank;
      keys[at] = lo + r;
      pos[at] = (uint32_t)(first + k * 64);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // the wave's LDS accesses are in order: all lanes have read
      if (rank == 0)
        __hip_atomic_store(mine, before + (uint32_t)__popcll(same), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_WAVEFRONT);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
  // masked tokens sort last
  if (blockIdx.x == gridDim.x - 1)
    for (int i = (int)(base + all) + (int)threadIdx.x; i < tokens; i += 64 * kBucketWaves) {
      keys[i] = (uint32_t)rows;
      pos[i] = 0;
    }
  if (late) clear();
}

constexpr int kSegAhead = 8;      // gradient rows loaded together

// A wave sums segment `seg` of the sorted tokens over one block of 64 E
// channels.  part[seg][0] gets the sum of the run that began before the
// segment, part[seg][1] that of the run that continues past it (both float32);
// a run that covers the whole segment and goes on at both ends is in [0].
template <class F, class G, int E, bool ALIGNED>
__global__ __launch_bounds__(256) void embedding_segment_kernel(
    const void* dout, const uint32_t* keys, const uint32_t* pos, void* dweight, float* part,
    int64_t tokens, int64_t rows, int64_t channels, int64_t row_stride, float scale, int seg_tokens) {
  using S = typename F::S;
  using IO = RowIO<F, E>;
  constexpr int OE = E < kVecElems<G> ? E : kVecElems<G>;   // outputs per store
  using OIO = RowIO<G, OE>;
  const int lane = lane_id();
  const int64_t blocks = (channels + 64 * E - 1) / (64 * E);
  const int64_t total = (tokens + seg_tokens - 1) / seg_tokens * blocks;
  for (int64_t w = (int64_t)blockIdx.x * 4 + wave_id(); w < total; w += (int64_t)gridDim.x * 4) {
    int64_t col;
    const int64_t seg = divide(w, blocks, &col), s0 = seg * seg_tokens;
    const int64_t ch = (col * 64 + lane) * E, n = channels - ch;
    const int cnt = (int)(tokens - s0 < seg_tokens ? tokens - s0 : seg_tokens);
    // lane l holds the key and position of token s0 + l, lane seg_tokens the next
    // segment's first key, and `before` the last segment's last
    uint32_t key = ~0u, at = 0;
    if (lane <= cnt && s0 + lane < tokens) {
      key = keys[s0 + lane];
      at = lane < cnt ? pos[s0 + lane] : 0;
    }
    const uint32_t before = s0 > 0 ? keys[s0 - 1] : ~0u;
    float* out_part = part + seg * 2 * channels + ch;
    float sum[E] = {};
    bool whole = true;               // the current run began in this segment
    {
      const uint32_t first = (uint32_t)__builtin_amdgcn_readlane((int)key, 0);
      whole = first != before;
    }
    for (int j0 = 0; j0 < cnt; j0 += kSegAhead) {
      typename IO::Raw raw[kSegAhead];
#pragma unroll
      for (int j = 0; j < kSegAhead; ++j) {
        raw[j] = typename IO::Raw{};
        const int64_t i = (uint32_t)__builtin_amdgcn_readlane((int)at, j0 + j);
        if (j0 + j < cnt && n > 0) raw[j] = IO::template get<ALIGNED>((const S*)dout + i * row_stride + ch, n);
      }
#pragma unroll
      for (int j = 0; j < kSegAhead; ++j) {
        if (j0 + j >= cnt) continue;
        const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)key, j0 + j);
        const uint32_t next = (uint32_t)__builtin_amdgcn_readlane((int)key, j0 + j + 1);
        if (k >= (uint32_t)rows) continue;               // masked tokens sort last
        float v[E];
        IO::unpack(raw[j], v);
#pragma unroll
        for (int c = 0; c < E; ++c) sum[c] += v[c];
        const bool last = j0 + j + 1 == cnt;
        if (k == next && !last) continue;
        // the run ends here, or the segment does
        const bool open = last && k == next;
        if (n > 0) {
          if (whole && !open) {
            typename G::S* to = (typename G::S*)dweight + (int64_t)k * channels + ch;
#pragma unroll
            for (int h = 0; h < E; h += OE) {
              float o[OE];
#pragma unroll
              for (int c = 0; c < OE; ++c) o[c] = sum[h + c] * scale;
              if (ALIGNED || h < n) OIO::template put<ALIGNED>(to + h, OIO::pack(o), n - h);
            }
          } else {
            float* to = out_part + (whole ? channels : 0);
#pragma unroll
            for (int c = 0; c < E; ++c)
              if (ALIGNED || c < n) to[c] = sum[c];
          }
        }
#pragma unroll
        for (int c = 0; c < E; ++c) sum[c] = 0.0f;
        whole = true;
      }
    }
  }
}

// Runs that cross segments: the workgroup of the segment in which such a run
// begins adds its pieces in order and writes the row (256 E channels of it).  A
// frequent token's run crosses many segments: kAhead of them are looked at
// together.
template <class G, int E, bool ALIGNED>
__global__ __launch_bounds__(256) void embedding_border_kernel(const uint32_t* __restrict__ keys,
                                                              void* __restrict__ dweight,
                                                              const float* __restrict__ part,
                                                              int64_t tokens, int64_t rows,
                                                              int64_t channels, float scale,
                                                              int seg_tokens) {
  using IO = RowIO<FmtF32, E>;
  constexpr int kAhead = 16;
  const int64_t cols = (channels + 256 * E - 1) / (256 * E);
  const int64_t segs = (tokens + seg_tokens - 1) / seg_tokens;
  for (int64_t w = blockIdx.x; w < segs * cols; w += gridDim.x) {
    int64_t col;
    const int64_t seg = divide(w, cols, &col), s0 = seg * seg_tokens, end = s0 + seg_tokens;
    if (end >= tokens) continue;                          // nothing follows the last segment
    const uint32_t k = keys[end - 1];
    if (k >= (uint32_t)rows || keys[end] != k) continue;  // no run continues past this segment
    if (s0 > 0 && keys[s0 - 1] == k) continue;            // it began in an earlier one
    const int64_t ch = (col * 256 + threadIdx.x) * E;
    // pieces after the first: up to the first segment that does not go on
    int64_t pieces = 0;
    for (bool more = true; more;) {
      const int64_t e = (seg + 2 + pieces + lane_id()) * seg_tokens;
      const bool on = e < tokens && keys[e < tokens ? e - 1 : 0] == k && keys[e < tokens ? e : 0] == k;
      const uint64_t stop = __ballot(!on);
      more = stop == 0;
      pieces += more ? kWave : __ffsll((unsigned long long)stop);
    }
    if (ch >= channels) continue;
    float sum[E];
    IO::unpack(IO::template get<ALIGNED>(part + (seg * 2 + 1) * channels + ch, channels - ch), sum);
    const float* from = part + (seg + 1) * 2 * channels + ch;
    typename IO::Raw next[kAhead];
    auto fetch = [&](int64_t p0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        next[j] = p0 + j < pieces ? IO::template get<ALIGNED>(from + (p0 + j) * 2 * channels,
                                                              channels - ch)
                                  : typename IO::Raw{};
    };
    fetch(0);
    for (int64_t p0 = 0; p0 < pieces; p0 += kAhead) {
      typename IO::Raw v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) v[j] = next[j];
      fetch(p0 + kAhead);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        float x[E];
        IO::unpack(v[j], x);
#pragma unroll
        for (int c = 0; c < E; ++c) sum[c] += x[c];       // past the pieces: + 0
      }
    }
#pragma unroll
    for (int c = 0; c < E; ++c)
      if (ALIGNED || c < channels - ch)
        ((typename G::S*)dweight)[(int64_t)k * channels + ch + c] = narrow<G>(sum[c] * scale);
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

constexpr int64_t kGridMost = 1 << 20;     // workgroups; kernels loop beyond it

hipError_t launch_embedding(const void* weight, const void* ids, bool wide_ids, void* out,
                            int64_t tokens, int64_t rows, int64_t channels, int64_t row_stride,
                            Fmt fmt, float scale, hipStream_t stream) {
  return by_format(fmt, [&](auto f) {
    using F = decltype(f);
    constexpr int E = kVecElems<F>;
    const bool vec = channels % E == 0 && row_stride % E == 0 && (uintptr_t)weight % 16 == 0 &&
                     (uintptr_t)out % 16 == 0;
    const int64_t blocks = (tokens * ((channels + E - 1) / E) + 255) / 256;
    const dim3 grid((unsigned)(blocks < kGridMost ? blocks : kGridMost));
    auto go = [&](auto* id) {
      auto run = [&](auto aligned, auto past) {
        embedding_kernel<F, E, decltype(aligned)::value, decltype(past)::value>
            <<<grid, dim3(256), 0, stream>>>(weight, id, out, tokens, rows, channels, row_stride,
                                             scale);
      };
      if (!vec) {
        run(std::false_type{}, std::false_type{});
      } else if (past_caches(tokens * channels * (int64_t)sizeof(typename F::S))) {
        run(std::true_type{}, std::true_type{});
      } else {
        run(std::true_type{}, std::false_type{});
      }
    };
    if (wide_ids) {
      go((const int64_t*)ids);
    } else {
      go((const int32_t*)ids);
    }
    return hipGetLastError();
  });
}

// Sorted tokens per wave: short segments leave more waves to a short list, long
// ones fewer runs that cross a border.
static int embedding_seg(int64_t tokens, int64_t channels) {
  const int64_t cols = (channels + 511) / 512;
  return tokens * cols >= 4096 * 32 ? 32 : tokens * cols >= 4096 * 16 ? 16 : 8;
}
static bool embedding_few(int64_t tokens) { return tokens <= kFewTokens; }
static bool embedding_short(int64_t tokens, int64_t rows) {
  return tokens <= kBucketTokens && rows <= 512 * kBucketRows;
}

// Scratch: keys, positions and their sort temporaries; the sort's own scratch;
// two float32 rows per segment.
namespace {
struct GradScratch {
  size_t keys, pos, tmp_keys, tmp_pos, sort, part, bytes;
};
GradScratch grad_scratch(int64_t tokens, int64_t rows, int64_t channels) {
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  GradScratch s;
  const size_t list = up((size_t)tokens * 4);
  const int seg = embedding_seg(tokens, channels);
  s.keys = 0;
  s.pos = list;
  s.tmp_keys = 2 * list;
  s.tmp_pos = 3 * list;
  s.sort = 4 * list;
  s.part = embedding_short(tokens, rows) ? s.tmp_keys : s.sort + up(radix_sort_scratch(tokens, 4));
  s.bytes = s.part + up((size_t)((tokens + seg - 1) / seg) * 2 * (size_t)channels * 4);
  return s;
}
}  // namespace
size_t embedding_grad_scratch(int64_t tokens, int64_t rows, int64_t channels) {
  return tokens == 0 ? 0 : grad_scratch(tokens, rows, channels).bytes;
}

static hipError_t few_go(const void* dout, const void* ids, bool wide_ids, void* dweight,
                         int64_t tokens, int64_t rows, int64_t channels, int64_t row_stride, Fmt fmt,
                         Fmt out_fmt, float scale, hipStream_t stream) {
  return by_format(fmt, [&](auto f) {
    using F = decltype(f);
    auto go = [&](auto o, auto aligned, auto* id) {
      using G = decltype(o);
      constexpr int E = kVecElems<F>;
      const int64_t cols = (channels + 64 * E - 1) / (64 * E);
      // 16 waves a CU, or every row and column block its own
      const int64_t most = 4096 / cols < 1 ? 1 : 4096 / cols, step = rows < most ? rows : most;
      embedding_few_kernel<F, G, E, decltype(aligned)::value>
          <<<dim3((unsigned)((step * cols + 3) / 4)), dim3(256), 0, stream>>>(
          dout, id, dweight, (int)tokens, rows, channels, row_stride, scale, (uint32_t)cols,
          (uint32_t)step);
    };
    auto by_ids = [&](auto o, auto e) {
      if (wide_ids) {
        go(o, e, (const int64_t*)ids);
      } else {
        go(o, e, (const int32_t*)ids);
      }
    };
    auto by_vec = [&](auto o) {
      constexpr int E = kVecElems<F>;
      if (channels % E == 0 && row_stride % E == 0 && (uintptr_t)dout % 16 == 0 &&
          (uintptr_t)dweight % 16 == 0) {
        by_ids(o, std::true_type{});
      } else {
        by_ids(o, std::false_type{});
      }
    };
    if (out_fmt == Fmt::F32) {
      by_vec(FmtF32{});
    } else {
      by_vec(F{});
    }
    return hipGetLastError();
  });
}

hipError_t launch_embedding_grad(const void* dout, const void* ids, bool wide_ids, void* dweight,
                                 int64_t tokens, int64_t rows, int64_t channels,
                                 int64_t row_stride, Fmt fmt, Fmt out_fmt, float scale,
                                 void* scratch, hipStream_t stream) {
  if (embedding_few(tokens))
    return few_go(dout, ids, wide_ids, dweight, tokens, rows, channels, row_stride, fmt, out_fmt,
                  scale, stream);
  const int out_bytes = out_fmt == Fmt::F32 ? 4 : 2;
  const bool one_launch = embedding_short(tokens, rows);
  if (!one_launch) {
    // rows without a token are zero; the others are overwritten below
    const uintptr_t a = (uintptr_t)dweight, e = a + (uintptr_t)(rows * channels * out_bytes);
    const uintptr_t a16 = (a + 15) & ~(uintptr_t)15;
    const uintptr_t lo = a16 < e ? a16 : e, hi = lo + ((e - lo) & ~(uintptr_t)15);
    const int64_t vecs = (int64_t)(hi - lo) / 16, blocks = (vecs + 1023) / 1024;
    if (lo > a) {
      embedding_zero_kernel<<<dim3(1), dim3(256), 0, stream>>>((uint4*)lo, 0, (uint8_t*)a,
                                                               (int)(lo - a));
    }
    embedding_zero_kernel<<<dim3((unsigned)(blocks < 1 ? 1 : blocks < 8192 ? blocks : 8192)),
                            dim3(256), 0, stream>>>((uint4*)lo, vecs, (uint8_t*)hi, (int)(e - hi));
  }
  const GradScratch g = grad_scratch(tokens, rows, channels);
  char* base = (char*)scratch;
  uint32_t* keys = (uint32_t*)(base + g.keys);
  uint32_t* pos = (uint32_t*)(base + g.pos);
  auto with_ids = [&](auto&& fn) {
    if (wide_ids) {
      fn((const int64_t*)ids);
    } else {
      fn((const int32_t*)ids);
    }
  };
  if (one_launch) {
    // two workgroups per CU as long as a workgroup's rows fit its counters
    const int64_t even = (rows + 511) / 512;
    const int bucket = (int)(even < kBucketRows ? even : kBucketRows);
    with_ids([&](auto* id) {
      embedding_bucket_kernel<<<dim3((unsigned)((rows + bucket - 1) / bucket)),
                                dim3(64 * kBucketWaves), 0, stream>>>(
          id, (int)tokens, rows, bucket, keys, pos, (char*)dweight, channels * out_bytes, out_bytes);
    });
  } else {
    with_ids([&](auto* id) {
      embedding_keys_kernel<<<dim3((unsigned)((tokens + 255) / 256)), dim3(256), 0, stream>>>(
          id, tokens, rows, keys, pos);
    });
    int bits = 8;                       // keys go up to `rows`
    while (bits < 32 && ((uint64_t)rows >> bits) != 0) bits += 8;
    const hipError_t e = launch_radix_sort(keys, base + g.tmp_keys, pos, base + g.tmp_pos, tokens,
                                           Fmt::U32, 4, bits, base + g.sort, stream);
    if (e != hipSuccess) return e;
  }
  float* part = (float*)(base + g.part);
  const int seg = embedding_seg(tokens, channels);
  const int64_t segs = (tokens + seg - 1) / seg;
  return by_format(fmt, [&](auto f) {
    using F = decltype(f);
    auto go = [&](auto o) {
      using G = decltype(o);
      constexpr int E = kVecElems<F>;
      const bool vec = channels % E == 0 && row_stride % E == 0 && (uintptr_t)dout % 16 == 0 &&
                       (uintptr_t)dweight % 16 == 0;
      auto segment = [&](auto e, auto aligned) {
        constexpr int SE = decltype(e)::value;
        const int64_t b = (segs * ((channels + 64 * SE - 1) / (64 * SE)) + 3) / 4;
        embedding_segment_kernel<F, G, SE, decltype(aligned)::value>
            <<<dim3((unsigned)(b < kGridMost ? b : kGridMost)), dim3(256), 0, stream>>>(
                dout, keys, pos, dweight, part, tokens, rows, channels, row_stride, scale, seg);
      };
      // rows off alignment: wide loose accesses, or one channel per lane where that
      // is what fills the card (1531 tokens x 333: 4.3 us against 6.4)
      const bool wide = segs * ((channels + 64 * E - 1) / (64 * E)) >= 1024;
      if (vec) {
        segment(std::integral_constant<int, E>{}, std::true_type{});
      } else if (wide) {
        segment(std::integral_constant<int, E>{}, std::false_type{});
      } else {
        segment(std::integral_constant<int, 1>{}, std::true_type{});
      }
      auto border = [&](auto e, auto aligned) {
        constexpr int BE = decltype(e)::value;
        const int64_t b = segs * ((channels + 256 * BE - 1) / (256 * BE));
        embedding_border_kernel<G, BE, decltype(aligned)::value>
            <<<dim3((unsigned)(b < kGridMost ? b : kGridMost)), dim3(256), 0, stream>>>(
                keys, dweight, part, tokens, rows, channels, scale, seg);
      };
      if (channels % 4 == 0) {
        border(std::integral_constant<int, 4>{}, std::true_type{});
      } else if (wide) {
        border(std::integral_constant<int, 4>{}, std::false_type{});
      } else {
        border(std::integral_constant<int, 1>{}, std::true_type{});
      }
      return hipGetLastError();
    };
    // the table's gradient in the activations' type or in float32
    if (out_fmt == Fmt::F32) return go(FmtF32{});
    return go(F{});
  });
}

}  // namespace sca
