// Building blocks of the selective scan's forward and gradient kernels, which
// share their mapping: a lane owns one channel and one state (or NS of them, 16
// apart) and walks the tokens in order.  Lanes 16 r .. 16 r + 15 of wave w hold
// 16 channels' state 4 w + r, so that B and C are the same for a row of 16
// lanes: a lane holds them for one of 16 tokens, and products take them by DPP
// row broadcast.  Sums over states go over the rows of a wave by register swaps
// and over the four waves through LDS.
#pragma once

#include <utility>

#include "sequence.hpp"

namespace sca {

constexpr int kScanTile = 16;                  // channels per row of lanes
constexpr int kKeep = kScanKeepTokens;         // tokens between kept states

// v = the row's lane T of `from`, for all its lanes (folds into the product)
template <int T> __device__ __forceinline__ float row_bcast(float from) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, from), 0x150 + T,
                                                            0xf, 0xf, true));
}

// Sums over the four rows of 16 lanes of 16 values: row r gets values 4 r .. 4 r
// + 3.  The swaps exchange halves (then rows) of a pair of registers, so that one
// addition serves two values.
__device__ __forceinline__ float swapped_sum32(float a, float b) {
  const auto q = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a),
                                                  __builtin_bit_cast(uint32_t, b), false, false);
  const uint32_t x = q[0], y = q[1];
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
__device__ __forceinline__ float swapped_sum16(float a, float b) {
  const auto q = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a),
                                                  __builtin_bit_cast(uint32_t, b), false, false);
  const uint32_t x = q[0], y = q[1];
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
__device__ __forceinline__ void rows_sum(const float (&v)[16], float (&out)[4]) {
  float s[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) s[t] = swapped_sum32(v[t], v[t + 8]);
#pragma unroll
  for (int t = 0; t < 4; ++t) out[t] = swapped_sum16(s[t], s[t + 4]);
}

// A lane whose state does not exist walks with the others, and C = 0 times its
// state is added to their outputs, so that state must stay 0 whatever the inputs:
// its A takes an infinite step to a decay of 0 (and any other to 1), and it reads
// zeros for the products and gradients, as an infinite one times its B or C of 0
// would be no number.  With more than 16 states these are then read for each of a
// lane's states.  Where all 16 NS states exist that is left out: 4 x 2048 channels
// of 2048 tokens with 32 states take 155 us instead of 161, 4 x 1024 with 64 167
// instead of 188.
constexpr float kNoState = -1e-30f;
template <int NS> bool scan_all_states(const ScanProblem& p) { return NS > 1 && p.states == 16 * NS; }

template <class Fn, int... T>
__device__ __forceinline__ void for_tokens(Fn&& fn, std::integer_sequence<int, T...>) {
  (fn(std::integral_constant<int, T>{}), ...);
}

// An array of activations [.., token, channels] as a workgroup reads it: a
// thread's pair (thread % 8) of its token (thread / 8) of a block, block after
// block.  Loads are never skipped: a thread whose token or pair does not exist
// reads one that does (the caller drops it), because behind a load that may not
// have happened the compiler can only wait for all of them.  VEC: the pair is
// loaded as one.
template <class F, bool VEC> struct Pair {
  using S = typename F::S;
  using Raw = std::conditional_t<VEC, typename RowIO<F, 2>::Raw, S>;
  Raw r[VEC ? 1 : 2];
  __device__ __forceinline__ void unpack(float (&v)[2]) const {
    if constexpr (VEC) {
      RowIO<F, 2>::unpack(r[0], v);
    } else {
      v[0] = widen<F>(r[0]);
      v[1] = widen<F>(r[1]);
    }
  }
  // zero for an element that is not `on`, without a branch
  __device__ __forceinline__ void unpack_if(bool on0, bool on1, float (&v)[2]) const {
    unpack(v);
    v[0] = on0 ? v[0] : 0.0f;
    v[1] = on1 ? v[1] : 0.0f;
    asm volatile("" : "+v"(v[0]), "+v"(v[1]));
  }
};
template <class F, bool VEC> struct PairSrc {
  using S = typename F::S;
  const S *base, *p;         // of the workgroup; of this thread
  int64_t token;             // stride
  int first, second;         // this thread's elements (the second relative to the first)
  // `n` elements of a row exist, n > 0
  PairSrc() = default;
  __device__ __forceinline__ PairSrc(const void* at, int64_t batch_stride, int64_t token_stride,
                                     int64_t b, int64_t off, int n) {
    base = (const S*)at + b * batch_stride + off;
    token = token_stride;
    const int e = (int)(threadIdx.x % 8) * 2;
    first = e < n ? e : 0;
    second = first + 1 < n ? 1 : 0;
    p = base;
  }
  // to the thread's token of block t0, the last that exists at the latest
  __device__ __forceinline__ void seek(int64_t t0, int64_t len) {
    const int64_t t = t0 + (int)(threadIdx.x / 8);
    p = base + (t < len ? t : len - 1) * token + first;
  }
  __device__ __forceinline__ void advance(int tokens) { p += tokens * token; }
  __device__ __forceinline__ Pair<F, VEC> load() const {
    Pair<F, VEC> v;
    if constexpr (VEC) {
      v.r[0] = *gptr<const typename Pair<F, VEC>::Raw>((uintptr_t)p);
    } else {
      v.r[0] = *gptr<const S>((uintptr_t)p);
      v.r[1] = *gptr<const S>((uintptr_t)(p + second));
    }
    return v;
  }
};

// Whether every pair of channels and of states lies on its size's alignment.
template <class F> bool scan_pairs(const ScanProblem& p, const void* y) {
  auto even = [](const void* a, int64_t s0, int64_t s1, int64_t s2) {
    return (uintptr_t)a % (2 * sizeof(typename F::S)) == 0 && ((s0 | s1 | s2) & 1) == 0;
  };
  return even(y, 0, 0, 0) && (p.channels / p.groups) % 2 == 0 && p.states % 2 == 0 &&
         even(p.x, p.x_batch, p.x_token, 0) && even(p.dt, p.dt_batch, p.dt_token, 0) &&
         (p.z == nullptr || even(p.z, p.z_batch, p.z_token, 0)) &&
         even(p.B, p.B_batch, p.B_token, p.B_group) && even(p.C, p.C_batch, p.C_token, p.C_group);
}

// A scan with too few workgroups is split over its length: `chunks` of `tokens`
// tokens each.  A first kernel finds every chunk's state from a zero start
// (`ends`) and the sum of its steps (`spans`): a chunk's start is then exp(A sum)
// of the chunk before's times that one's start, plus that one's end.  One chunk:
// not split.
struct ScanSplit {
  int64_t tokens;
  uint32_t chunks;
  float* ends;          // [batch][chunks][channels][states]
  float* spans;         // [batch][chunks][channels]
};
// What becomes of h over a chunk: 2^p h, p = A log2(e) times the chunk's steps.
// The factor may leave float32's range where the product does not, so it is
// applied in two halves; and 0 and infinity stay what they are, as they do token by
// token, where a half that is infinite or 0 would make them no number.
__device__ __forceinline__ float carried(float p, float h) {
  const float half = exp2_hw(0.5f * p), v = h * half * half;
  const bool stays = h == 0.0f || __builtin_isinf(h);
  return stays && __builtin_isfinite(p) ? h : v;
}

// Where a workgroup stands in the problem: sequence, group of B and C, first
// channel, and how many of its channels exist.
struct ScanPlace {
  int64_t b, g, ch, nch, tile;
};
// `width` channels per workgroup, `tiles` workgroups per group.
__device__ __forceinline__ ScanPlace scan_place(const ScanProblem& p, int64_t b0, int64_t tiles,
                                                uint32_t id, int width) {
  ScanPlace s;
  const int64_t per = p.channels / p.groups;
  const int64_t w = id / (uint32_t)tiles;
  s.tile = id % (uint32_t)tiles;
  s.g = w % p.groups;
  s.b = b0 + w / p.groups;
  s.ch = s.g * per + s.tile * width;
  const int64_t left = per - s.tile * width;
  s.nch = left < width ? left : width;
  return s;
}
__device__ __forceinline__ int64_t scan_length(const ScanProblem& p, int64_t b) {
  if (p.lengths == nullptr) return p.length;
  const int64_t v = p.lengths[b];
  return v < 0 ? 0 : (v > p.length ? p.length : v);
}

}  // namespace sca
