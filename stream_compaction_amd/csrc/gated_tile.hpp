// What the gated scan's forward and gradient share: a workgroup's tile of tokens
// and channels, the maps that carry a state over a run of tokens, and their
// exchange between workgroups.
//
// A tile is 128 channels, two to a lane, and a run of consecutive tokens for each
// of the 8 waves, kept in registers: the inputs are read once.  A state crosses a
// run by h -> 2^l h + b, where l sums the tokens' log2 decays.  Waves exchange
// their maps through LDS, workgroups through memory: each writes its tile's map as
// soon as it has read its tokens, and reads those of the tiles before it (after it,
// in the gradient) in its group of 16, and one state at the group's border.  So no
// tile waits for more than its neighbours' reading and one link a group, and what
// is added in which order does not depend on timing.
#pragma once

#include "gated.hpp"

namespace sca {

constexpr int kTileWaves = 8;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kTileChannels = 128;           // two to a lane
constexpr int kTileGroup = 16;               // tiles from one passed-on state to the next
constexpr int64_t kTicketWords = 16;         // a column's ticket, on a cache line of its own

// A launch's tiles: columns (a sequence's 128 channels) of `chunks` runs.  Its grid is
// the parts of the channels, the sequences, and the chunks (those beyond the third
// axis beside the parts), so that no workgroup divides to find its column.
struct Tiles {
  int64_t parts, batch, chunks;              // of the launch
  int64_t b0;                                // its first sequence
  __host__ __device__ int64_t cols() const { return parts * batch; }
  int64_t words() const {                    // of scratch, 8 bytes each
    if (chunks <= 1) return 0;
    return cols() * (kTicketWords + (chunks + (chunks + kTileGroup - 1) / kTileGroup) * kTileChannels);
  }
};
constexpr int64_t kAxis = 65535;             // a grid's second and third axis
inline Tiles gated_tiles(const GatedProblem& p, int tokens) {
  Tiles t;
  t.parts = (p.channels + kTileChannels - 1) / kTileChannels;
  t.batch = p.batch < kAxis ? p.batch : kAxis;
  t.chunks = p.length <= tokens ? 1 : (p.length + tokens - 1) / tokens;
  t.b0 = 0;
  return t;
}
// Fills `tickets` words with zeros and the others with ones.
hipError_t launch_tile_clear(uint64_t* scratch, int64_t tickets, int64_t words, hipStream_t stream);

// Launches `kernel(grid, tiles)` over all tiles; a batch beyond the second axis goes
// out in parts, one after the other in the same scratch.
template <class Kernel>
hipError_t launch_tiles(Tiles t, int64_t batch, uint64_t* scratch, hipStream_t stream, Kernel&& kernel) {
  const int64_t z = t.chunks < kAxis ? t.chunks : kAxis, x = (t.chunks + z - 1) / z;
  for (; t.b0 < batch; t.b0 += kAxis) {
    if (batch - t.b0 < t.batch) t.batch = batch - t.b0;
    if (t.chunks > 1) {
      const hipError_t e = launch_tile_clear(scratch, t.cols() * kTicketWords, t.words(), stream);
      if (e != hipSuccess) return e;
    }
    kernel(dim3((unsigned)(t.parts * x), (unsigned)t.batch, (unsigned)z), t);
  }
  return hipGetLastError();
}

// The tokens of a sequence that exist.
__device__ __forceinline__ int64_t sequence_tokens(const GatedProblem& p, int64_t b) {
  return p.lengths == nullptr ? p.length : live_count(p.length, p.lengths + b);
}

// A sequence's rows, one token after the other, as wave-uniform addresses.
struct Rows {
  uintptr_t at, step;
  __device__ __forceinline__ Rows(uintptr_t base, int64_t batch, int64_t token, int64_t b, int64_t t, int eb)
      : at(base + (uintptr_t)((b * batch + t * token) * eb)), step((uintptr_t)(token * eb)) {}
  // on: all ones, or zero past the last token, which is read again
  __device__ __forceinline__ void next(uintptr_t on) { at += step & on; }
};

// Two neighbouring channels of a row as one access, or, where the number of
// channels is odd, as one access each (a pair may then lie across a row's end).  An odd
// width costs as much again: 8 x 2048 bfloat16 tokens of 2303 channels 131 us and in the
// gradient 236, of 2304 65 and 129; 4 x 2048 in float32 87 and 177, 58 and 110.
// Pairs are stored past the caches where the outputs are large (past_caches):
// forward and gradient of 4 x 2048 x 2048 bf16, 34 MB an output, 108 to 102 us.  Once:
// loaded so, too, by the gradient and by a forward that keeps no states for one (after
// which nobody is known to read the inputs again): forward of 4 x 4096 x 4096 bf16 114.3
// to 111.9 us, of 4 x 2048 x 2304 f32 73.7 to 70.6; forward and gradient of 4 x 2048 x 4096
// 175 to 172; with the keeping forward's loads, too, 2 x 4096 x 2048 f32 159.5 to 166.
enum class Rows2 { Pairs, PairsPast, PairsOnce, Singles };
template <class F, Rows2 ROWS> struct PairIO {
  static constexpr bool ODD = ROWS == Rows2::Singles;
  using S = typename F::S;
  using IO = RowIO<F, 2>;
  using Raw = typename IO::Raw;
  typedef Raw Loose __attribute__((aligned(sizeof(S))));
  // o0, o1: byte offsets of the two channels, inside the row
  static __device__ __forceinline__ Raw load(uintptr_t row, uint32_t o0, uint32_t o1) {
    if constexpr (ODD) {
      typename IO::Elems e;
      e.e[0] = *(const __attribute__((address_space(1))) S*)(gptr<const char>(row) + o0);
      e.e[1] = *(const __attribute__((address_space(1))) S*)(gptr<const char>(row) + o1);
      return __builtin_bit_cast(Raw, e);
    } else {
      const auto at = (const __attribute__((address_space(1))) Loose*)(gptr<const char>(row) + o0);
      if constexpr (ROWS == Rows2::PairsOnce) {
        return __builtin_nontemporal_load(at);
      } else {
        return *at;
      }
    }
  }
  static __device__ __forceinline__ void put(uintptr_t row, uint32_t o0, Raw r) {
    auto at = (__attribute__((address_space(1))) Loose*)(gptr<char>(row) + o0);
    if constexpr (ROWS == Rows2::PairsPast || ROWS == Rows2::PairsOnce) {
      __builtin_nontemporal_store(r, at);
    } else {
      *at = r;
    }
  }
  template <class E> static __device__ __forceinline__ void put_one(uintptr_t at, uint32_t o, E e) {
    *(__attribute__((address_space(1))) E*)(gptr<char>(at) + o) = e;
  }
  // `room` of T rows, `step` bytes apart; n: how many of the two channels exist.  (One
  // decision for all rows of a whole run: one for each cost a tenth of the kernel.)
  template <int T>
  static __device__ __forceinline__ void store_rows(uintptr_t row, uintptr_t step, uint32_t o0, const Raw (&r)[T],
                                                    int room, int n) {
    if constexpr (ODD) {
#pragma unroll
      for (int k = 0; k < T; ++k, row += step) {
        const typename IO::Elems e = __builtin_bit_cast(typename IO::Elems, r[k]);
        if (k < room && n > 0) put_one(row, o0, e.e[0]);
        if (k < room && n > 1) put_one(row, o0 + (uint32_t)sizeof(S), e.e[1]);
      }
    } else if (n > 0) {
      if (room == T) {
#pragma unroll
        for (int k = 0; k < T; ++k, row += step) put(row, o0, r[k]);
      } else {
#pragma unroll
        for (int k = 0; k < T; ++k, row += step)
          if (k < room) put(row, o0, r[k]);
      }
    }
  }
  // The same bits, of which the compiler knows nothing any more: what is computed
  // from them is computed again, not kept in registers since the first time.
  static __device__ __forceinline__ Raw again(Raw r) {
    if constexpr (sizeof(Raw) == 4) {
      uint32_t w = __builtin_bit_cast(uint32_t, r);
      materialize(w);
      return __builtin_bit_cast(Raw, w);
    } else {
      u32x2 w = __builtin_bit_cast(u32x2, r);
      uint32_t lo = w.x, hi = w.y;
      materialize(lo);
      materialize(hi);
      return __builtin_bit_cast(Raw, u32x2{lo, hi});
    }
  }
  static __device__ __forceinline__ Raw splat(float v) {
    const float x[2] = {v, v};
    return IO::pack(x);
  }
};

// sqrt(2^l) of a run's decay, by which a state is multiplied twice: 2^l itself may
// leave float32's range where its product with a large state does not.  What is
// below 2^-252 counts as that, which leaves less than 2^-124 of any finite state, and an
// infinite one stays so; l = -inf (a decay of 0) gives 0.
__device__ __forceinline__ float half_decay(float l) {
  const float m = at_least(exp2_hw(0.5f * l), 1.17549435e-38f);
  return l == -__builtin_huge_valf() ? 0.0f : m;
}
__device__ __forceinline__ float carry_over(float m, float b, float h) {
  return __builtin_fmaf(h * m, m, b);
}

// Slots: a map or a state as one 64-bit word, written and read whole, whose upper
// half is never all ones; the launch before fills them with ones.
constexpr uint32_t kNoWord = 0xffffffffu;
__device__ __forceinline__ uint64_t map_word(float l, float b) {
  uint32_t hi = __builtin_bit_cast(uint32_t, l);
  if (hi == kNoWord) hi = 0x7fc00000u;       // that one NaN becomes another
  return ((uint64_t)hi << 32) | __builtin_bit_cast(uint32_t, b);
}
__device__ __forceinline__ float word_l(uint64_t w) { return __builtin_bit_cast(float, (uint32_t)(w >> 32)); }
__device__ __forceinline__ float word_b(uint64_t w) { return __builtin_bit_cast(float, (uint32_t)w); }
__device__ __forceinline__ uint64_t state_word(float h) { return __builtin_bit_cast(uint32_t, h); }

// Two channels' words, once they are there.  Every wait ends: a word that is not
// there after some seconds of asking never comes (two calls in flight have shared
// their scratch, which is not allowed), and stands for a state that is no number.
#ifndef SCA_TILE_POLLS
#define SCA_TILE_POLLS (1u << 22)
#endif
constexpr uint64_t kLostWord = 0x7fc000007fc00000ull;
// Whether a column's word is written: the library's always; of a test build, not the map of
// step 3 in every second column, nor the state at the first border in the others.
__device__ __forceinline__ bool map_comes(int64_t col, int64_t step) {
#ifdef SCA_TILE_MUTE
  return col % 2 != 0 || step != 3;
#else
  return true;
#endif
}
__device__ __forceinline__ bool border_comes(int64_t col, int64_t group) {
#ifdef SCA_TILE_MUTE
  return col % 2 == 0 || group != 1;
#else
  return true;
#endif
}
struct Words { uint64_t w[2]; };
__device__ __forceinline__ Words peek_words(const uint64_t* at) {
  return Words{{ld_relaxed(at), ld_relaxed(at + 1)}};
}
__device__ __forceinline__ bool no_word(uint64_t w) { return (uint32_t)(w >> 32) == kNoWord; }
__device__ __forceinline__ Words await_words(const uint64_t* at, Words w) {
  for (uint32_t polls = 0; __ballot(no_word(w.w[0]) || no_word(w.w[1])); ++polls) {
    if (polls >= SCA_TILE_POLLS) {
      for (uint64_t& v : w.w) v = no_word(v) ? kLostWord : v;
      break;
    }
    __builtin_amdgcn_s_sleep(4);
    w = peek_words(at);
  }
  return w;
}

// Which run of its column a workgroup takes: by the column's ticket, so that the
// tiles it will wait for are with workgroups that run already, whatever order the
// hardware starts them in.  (The column's first unfinished tile waits for none.)  One
// ticket for all tiles would cost 12 ns a tile, 25 us of the 72 of 8192 x 4096.
__device__ __forceinline__ int64_t draw_chunk(uint64_t* scratch, int64_t col, uint64_t* shared) {
  if (threadIdx.x == 0)
    *shared = __hip_atomic_fetch_add(scratch + col * kTicketWords, 1ull, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return (int64_t)readlane(*shared, 0);
}
// A workgroup's place: its part of the channels, its sequence and their column, and
// which of the column's runs it takes (-1: none is left).
struct Place { int part; int64_t col, b, run; };
// Workgroups go to the 8 XCDs in turn; with `near` one XCD takes four neighbouring parts of
// 32, 1 KB of a 16-bit row, where the parts are a multiple of 32.  (The forward of 4 x 4096 x
// 4096 77.0 to 74.6 us, 8192 x 8192 114.6 to 111.6; in float32 8192 x 8192 143 to 140, 2 x 4096 x
// 4096 and 4 x 4096 x 4096 the same; with both gates 4 x 2048 x 8192 lost, 148 to 151.  Two of
// 16 parts gained nothing at 2048 channels, nor did the gradient.)
template <bool near>
__device__ __forceinline__ Place draw_place(const Tiles& t, uint64_t* scratch, uint64_t* shared) {
  Place p;
  const uint32_t parts = (uint32_t)t.parts;
  p.part = (int)(gridDim.x == parts ? blockIdx.x : blockIdx.x % parts);
  if (near && parts % 32 == 0) p.part = (p.part & ~31) + (p.part & 7) * 4 + ((p.part >> 3) & 3);
  p.b = t.b0 + blockIdx.y;
  p.col = (int64_t)blockIdx.y * parts + p.part;
  p.run = 0;
  if (t.chunks > 1) {
    p.run = draw_chunk(scratch, p.col, shared);
    if (p.run >= t.chunks) p.run = -1;
  }
  return p;
}

struct TileMaps {                            // a workgroup's exchange
  float l[kTileWaves][kTileChannels], m[kTileWaves][kTileChannels], b[kTileWaves][kTileChannels];
  float fm[kTileWaves][kTileChannels], fb[kTileWaves][kTileChannels];   // tiles looked back to
  float base[kTileChannels];
  uint64_t tile;
};

__device__ __forceinline__ void put2(float* row, float a, float b) {
  *(f32x2*)(row + 2 * lane_id()) = f32x2{a, b};
}
__device__ __forceinline__ void get2(const float* row, float (&v)[2]) {
  const f32x2 r = *(const f32x2*)(row + 2 * lane_id());
  v[0] = r.x;
  v[1] = r.y;
}

// The state that enters tile `step` of its column's `steps` (both counted in the
// direction of the walk), and what the tile leaves to others: called by every wave
// when all maps are in LDS (before a barrier), with the state `first` that enters
// the column (of which the last wave asks in a column's first group).
__device__ __forceinline__ void tile_entry(TileMaps& s, int wave, int64_t step, int64_t steps,
                                           int64_t col, int64_t cols, uint64_t* scratch,
                                           int64_t chunks, const float (&first)[2], float (&h)[2]) {
  const int lane2 = 2 * lane_id();
  uint64_t* slots = scratch + cols * kTicketWords;
  uint64_t* borders = slots + chunks * cols * kTileChannels;
  auto slot = [&](int64_t i) { return slots + (i * cols + col) * kTileChannels + lane2; };
  auto border = [&](int64_t g) { return borders + (g * cols + col) * kTileChannels + lane2; };
  const int64_t group = step / kTileGroup, begin = group * kTileGroup;
  const int before = (int)(step - begin);
  constexpr int kEach = (kTileGroup - 1 + kTileWaves - 1) / kTileWaves;
  static_assert(kEach == 2, "each wave looks at two tiles");
  const int i0 = wave * kEach;
  const bool on0 = i0 < before, on1 = i0 + 1 < before;
  Words w0 = {}, w1 = {}, wb = {};
  if (on0) w0 = peek_words(slot(begin + i0));
  if (on1) w1 = peek_words(slot(begin + i0 + 1));
  const bool passes = wave == kTileWaves - 1 && group > 0;
  if (passes) wb = peek_words(border(group));
  if (wave == 0 && step + 1 < steps && map_comes(col, step)) {   // this tile's own map
    float l[2] = {0.0f, 0.0f}, b[2] = {0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) {
      float wl[2], wm[2], wb2[2];
      get2(s.l[w], wl);
      get2(s.m[w], wm);
      get2(s.b[w], wb2);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[c] += wl[c];
        b[c] = carry_over(wm[c], wb2[c], b[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) st_relaxed(slot(step) + c, map_word(l[c], b[c]));
  }
  float m[2] = {1.0f, 1.0f}, b[2] = {0.0f, 0.0f};
  if (on0) {
    w0 = await_words(slot(begin + i0), w0);
    float l[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      l[c] = word_l(w0.w[c]);
      b[c] = word_b(w0.w[c]);
    }
    if (on1) {
      w1 = await_words(slot(begin + i0 + 1), w1);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        b[c] = carry_over(half_decay(word_l(w1.w[c])), word_b(w1.w[c]), b[c]);
        l[c] += word_l(w1.w[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) m[c] = half_decay(l[c]);
  }
  put2(s.fm[wave], m[0], m[1]);
  put2(s.fb[wave], b[0], b[1]);
  if (wave == kTileWaves - 1) {
    float v[2] = {first[0], first[1]};
    if (passes) {
      wb = await_words(border(group), wb);
      v[0] = word_b(wb.w[0]);
      v[1] = word_b(wb.w[1]);
    }
    put2(s.base, v[0], v[1]);
  }
  lds_barrier();
  get2(s.base, h);
  const int used = (before + kEach - 1) / kEach;
  for (int w = 0; w < used; ++w) {
    get2(s.fm[w], m);
    get2(s.fb[w], b);
#pragma unroll
    for (int c = 0; c < 2; ++c) h[c] = carry_over(m[c], b[c], h[c]);
  }
  // the group's last tile passes the state on
  if (wave == kTileWaves - 1 && before == kTileGroup - 1 && step + 1 < steps && border_comes(col, group + 1)) {
    float v[2] = {h[0], h[1]};
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) {
      get2(s.m[w], m);
      get2(s.b[w], b);
#pragma unroll
      for (int c = 0; c < 2; ++c) v[c] = carry_over(m[c], b[c], v[c]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) st_relaxed(border(group + 1) + c, state_word(v[c]));
  }
}

// The state that enters this wave's run, from the one that enters the tile.
__device__ __forceinline__ void wave_entry(const TileMaps& s, int wave, float (&h)[2]) {
  for (int w = 0; w < wave; ++w) {
    float m[2], b[2];
    get2(s.m[w], m);
    get2(s.b[w], b);
#pragma unroll
    for (int c = 0; c < 2; ++c) h[c] = carry_over(m[c], b[c], h[c]);
  }
}

}  // namespace sca
