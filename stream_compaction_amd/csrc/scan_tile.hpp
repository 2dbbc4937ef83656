// Building blocks of the selective scan's forward and gradient kernels.
//
// Mapping shared by both: the recurrence h[t] = a[t] h[t-1] + b[t] is an
// affine map per token, and affine maps compose, so it is scanned like a sum:
// each lane of a wave64 owns K consecutive tokens, folds them into one map
// (P, H), the 64 maps are scanned across the wave with DPP, and the lane then
// walks its K tokens from the state it got.  Lanes along time (instead of
// along channels) keep every sum over states and, in the gradient, every sum
// over channels inside a lane, and a sequence of one batch needs no split of
// its length to fill the chip: a wave owns one pair of channels.
//
// A workgroup of 8 waves owns 16 channels of one sequence and walks it in
// blocks of TB = 64 K tokens, whose activations and B, C rows it stages in LDS.
#pragma once

#include "sequence.hpp"

namespace sca {

constexpr int kRowRor1 = 0x121;                // DPP: rotate each row of 16 lanes right by one
constexpr int kScanWaves = 8;
constexpr int kScanThreads = 64 * kScanWaves;
constexpr int kScanTile = 2 * kScanWaves;      // channels per workgroup

// LDS planes hold one value (or one pair of 16-bit channels) per token of the
// block, ordered so that each lane's K tokens are read 16 bytes at a time with
// consecutive lanes 16 bytes apart (no bank conflicts).
template <int K> __device__ __forceinline__ int plane_index(int t) {
  constexpr int V = K < 4 ? K : 4;
  const int lane = t / K, k = t % K;
  return (k / V) * (64 * V) + lane * V + k % V;
}
template <int K> __device__ __forceinline__ int plane_token(int i) {
  constexpr int V = K < 4 ? K : 4;
  return ((i / V) % 64) * K + (i / (64 * V)) * V + i % V;
}

// This lane's K words of a plane.
template <int K, class T>
__device__ __forceinline__ void plane_read(const T* plane, int lane, T (&v)[K]) {
  static_assert(sizeof(T) == 4, "a plane holds 32-bit words");
  constexpr int V = K < 4 ? K : 4;
  typedef T vec __attribute__((ext_vector_type(V)));
#pragma unroll
  for (int j = 0; j < K / V; ++j) {
    if constexpr (V == 1) {
      v[j] = plane[lane];
    } else {
      const vec w = *(const vec*)(plane + j * 64 * V + lane * V);
#pragma unroll
      for (int k = 0; k < V; ++k) v[j * V + k] = w[k];
    }
  }
}
template <int K, class T>
__device__ __forceinline__ void plane_write(T* plane, int lane, const T (&v)[K]) {
  constexpr int V = K < 4 ? K : 4;
  typedef T vec __attribute__((ext_vector_type(V)));
#pragma unroll
  for (int j = 0; j < K / V; ++j) {
    if constexpr (V == 1) {
      plane[lane] = v[j];
    } else {
      vec w;
#pragma unroll
      for (int k = 0; k < V; ++k) w[k] = v[j * V + k];
      *(vec*)(plane + j * 64 * V + lane * V) = w;
    }
  }
}

// Inclusive scan across the 64 lanes of two independent sequences of affine
// maps h -> P h + H (an earlier lane's map applies first).  Written in asm so
// that each step is one instruction per register: lanes whose DPP source does
// not exist keep their value (their writes are disabled), which is the
// identity.  The leading s_nop and the order of the four instructions keep at
// least two issue slots between a write and the DPP read of the same register.
#define SCA_AFFINE_STEP(MODE)                                  \
  "v_fmac_f32_dpp %0, %0, %2 " MODE "\n\t"                     \
  "v_fmac_f32_dpp %1, %1, %3 " MODE "\n\t"                     \
  "v_mul_f32_dpp %2, %2, %2 " MODE "\n\t"                      \
  "v_mul_f32_dpp %3, %3, %3 " MODE "\n\t"
__device__ __forceinline__ void affine_scan2(float& H0, float& H1, float& P0, float& P1) {
  asm volatile(
      "s_nop 1\n\t"
      SCA_AFFINE_STEP("row_shr:1 row_mask:0xf bank_mask:0xf")
      SCA_AFFINE_STEP("row_shr:2 row_mask:0xf bank_mask:0xf")
      SCA_AFFINE_STEP("row_shr:4 row_mask:0xf bank_mask:0xf")
      SCA_AFFINE_STEP("row_shr:8 row_mask:0xf bank_mask:0xf")
      SCA_AFFINE_STEP("row_bcast:15 row_mask:0xa bank_mask:0xf")
      SCA_AFFINE_STEP("row_bcast:31 row_mask:0xc bank_mask:0xf")
      "s_nop 1"
      : "+v"(H0), "+v"(H1), "+v"(P0), "+v"(P1));
}
#undef SCA_AFFINE_STEP

// The same within each row of 16 lanes, one sequence per row.  P is left
// undefined.  An instruction and a wait state lie between a write and the DPP
// read of the same register.
#define SCA_ROW_STEP(SHIFT)                                                    \
  "v_fmac_f32_dpp %0, %0, %1 row_shr:" SHIFT " row_mask:0xf bank_mask:0xf\n\t"  \
  "v_mul_f32_dpp %1, %1, %1 row_shr:" SHIFT " row_mask:0xf bank_mask:0xf\n\t"   \
  "s_nop 0\n\t"
__device__ __forceinline__ void row_affine_scan(float& H, float& P) {
  asm volatile(
      "s_nop 1\n\t"
      SCA_ROW_STEP("1")
      SCA_ROW_STEP("2")
      SCA_ROW_STEP("4")
      "v_fmac_f32_dpp %0, %0, %1 row_shr:8 row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1"
      : "+v"(H), "+v"(P));
}
#undef SCA_ROW_STEP

// One array of activations [batch, length, channels] as a workgroup sees it:
// its sequence and first channel.
template <class F> struct TileSrc {
  const typename F::S* p;
  int64_t token;        // stride between tokens
  bool vec;             // every vector of the tile is 16-byte aligned
};
template <class F>
__device__ __forceinline__ TileSrc<F> tile_src(const void* base, int64_t batch_stride,
                                               int64_t token_stride, int64_t b, int64_t ch) {
  using S = typename F::S;
  TileSrc<F> s;
  s.p = (const S*)base + b * batch_stride + ch;
  s.token = token_stride;
  s.vec = ((uintptr_t)s.p % 16 == 0) && ((token_stride * (int64_t)sizeof(S)) % 16 == 0);
  return s;
}

// The same by pairs of neighbours: a thread's pair (thread % 8) of its token
// (thread / 8) of a block, block after block.  Loads are never skipped: a
// thread whose token or pair does not exist reads one that does (the caller
// drops it), because behind a load that may not have happened the compiler can
// only wait for all of them.  VEC: the pair is loaded as one.
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

// Global -> registers -> LDS staging of one activation array's block
// ([TB tokens, 16 channels]).  Planes: 16-bit types hold one channel pair per
// word (8 planes), float32 one channel (16 planes).
template <class F, int K> struct TileStage {
  using S = typename F::S;
  static constexpr int E = kVecElems<F>;
  static constexpr int TB = 64 * K;
  static constexpr int VT = kScanTile / E;                    // vectors per token
  static constexpr int NV = (TB * VT + kScanThreads - 1) / kScanThreads;
  static constexpr int PLANES = kScanTile * (int)sizeof(S) / 4;
  static constexpr int WORDS = PLANES * TB;
  uint4 r[NV];

  // tokens [t0, t0 + TB) of which those before `len` exist; nch channels exist
  __device__ __forceinline__ void load(const TileSrc<F>& s, int64_t t0, int64_t len, int64_t nch) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = (int)threadIdx.x + j * kScanThreads;
      const int64_t t = t0 + v / VT;
      const int c = (v % VT) * E;
      r[j] = uint4{0, 0, 0, 0};
      if (v < TB * VT && t < len && c < nch) r[j] = load_vec<F>(s.p + t * s.token + c, nch - c, s.vec);
    }
  }
  __device__ __forceinline__ void put(uint32_t* lds) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = (int)threadIdx.x + j * kScanThreads;
      if (TB * VT % kScanThreads == 0 || v < TB * VT) {
        uint32_t* p = lds + (v % VT) * 4 * TB + plane_index<K>(v / VT);
        p[0] = r[j].x;
        p[TB] = r[j].y;
        p[2 * TB] = r[j].z;
        p[3 * TB] = r[j].w;
      }
    }
  }
  // LDS -> global (contiguous [.., channels] output at `out`, row stride `token`)
  static __device__ __forceinline__ void store(const uint32_t* lds, S* out, int64_t token, bool vec,
                                               int64_t t0, int64_t end, int64_t nch) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = (int)threadIdx.x + j * kScanThreads;
      const int64_t t = t0 + v / VT;
      const int c = (v % VT) * E;
      if (v < TB * VT && t < end && c < nch) {
        const uint32_t* p = lds + (v % VT) * 4 * TB + plane_index<K>(v / VT);
        store_vec<F>(out + t * token + c, uint4{p[0], p[TB], p[2 * TB], p[3 * TB]}, nch - c, vec);
      }
    }
  }
  // this lane's K tokens of the two channels of `wave` (channel innermost, as
  // the 16-bit formats pack them)
  static __device__ __forceinline__ void get(const uint32_t* lds, int wave, int lane,
                                             float (&v)[K][2]) {
    if constexpr (sizeof(S) == 2) {
      uint32_t w[K];
      plane_read<K>(lds + wave * TB, lane, w);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k][0] = widen<F>((S)(w[k] & 0xffffu));
        v[k][1] = widen<F>((S)(w[k] >> 16));
      }
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[K];
        plane_read<K>(lds + (2 * wave + c) * TB, lane, w);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k][c] = __builtin_bit_cast(float, w[k]);
      }
    }
  }
  static __device__ __forceinline__ void set(uint32_t* lds, int wave, int lane,
                                             const float (&v)[K][2]) {
    if constexpr (sizeof(S) == 2) {
      uint32_t w[K];
#pragma unroll
      for (int k = 0; k < K; ++k) w[k] = narrow2<F>(v[k][0], v[k][1]);
      plane_write<K>(lds + wave * TB, lane, w);
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[K];
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = __builtin_bit_cast(uint32_t, v[k][c]);
        plane_write<K>(lds + (2 * wave + c) * TB, lane, w);
      }
    }
  }
};

// Staging of a block's rows of B or C: NG states per token, widened to float
// planes [NG][TB].
template <class F, int K, int NG> struct RowStage {
  using S = typename F::S;
  static constexpr int E = kVecElems<F>;
  static constexpr int TB = 64 * K;
  static constexpr int VT = NG / E;
  static constexpr int NV = (TB * VT + kScanThreads - 1) / kScanThreads;
  uint4 r[NV];

  // states [n0, n0 + NG) of which those below `states` exist
  __device__ __forceinline__ void load(const TileSrc<F>& s, int64_t t0, int64_t len, int n0,
                                       int states) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = (int)threadIdx.x + j * kScanThreads;
      const int64_t t = t0 + v / VT;
      const int n = n0 + (v % VT) * E;
      r[j] = uint4{0, 0, 0, 0};
      if (v < TB * VT && t < len && n < states)
        r[j] = load_vec<F>(s.p + t * s.token + n, states - n, s.vec);
    }
  }
  __device__ __forceinline__ void put(float* lds) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = (int)threadIdx.x + j * kScanThreads;
      if (TB * VT % kScanThreads == 0 || v < TB * VT) {
        float x[E];
        VecIO<S, E>::template unpack<F>(r[j], x);
        float* p = lds + (v % VT) * E * TB + plane_index<K>(v / VT);
#pragma unroll
        for (int e = 0; e < E; ++e) p[e * TB] = x[e];
      }
    }
  }
};

// Whether every pair of channels and of states lies on its size's alignment.
template <class F> bool scan_pairs(const ScanProblem& p, const void* y) {
  auto even = [](const void* a, int64_t s0, int64_t s1, int64_t s2) {
    return (uintptr_t)a % (2 * sizeof(typename F::S)) == 0 && ((s0 | s1 | s2) & 1) == 0;
  };
  return even(y, 0, 0, 0) && (p.channels / p.groups) % 2 == 0 && p.states % 2 == 0 && even(p.x, p.x_batch, p.x_token, 0) &&
         even(p.dt, p.dt_batch, p.dt_token, 0) &&
         (p.z == nullptr || even(p.z, p.z_batch, p.z_token, 0)) &&
         even(p.B, p.B_batch, p.B_token, p.B_group) && even(p.C, p.C_batch, p.C_token, p.C_group);
}

// Where a workgroup stands in the problem: sequence, group of B and C, first
// channel, and how many of its 16 channels exist.
struct ScanPlace {
  int64_t b, g, ch, nch, tile;
};
__device__ __forceinline__ ScanPlace scan_place(const ScanProblem& p, int64_t b0, int64_t tiles,
                                                uint32_t id) {
  ScanPlace s;
  const int64_t per = p.channels / p.groups;
  const int64_t w = id / (uint32_t)tiles;
  s.tile = id % (uint32_t)tiles;
  s.g = w % p.groups;
  s.b = b0 + w / p.groups;
  s.ch = s.g * per + s.tile * kScanTile;
  const int64_t left = per - s.tile * kScanTile;
  s.nch = left < kScanTile ? left : kScanTile;
  return s;
}
__device__ __forceinline__ int64_t scan_length(const ScanProblem& p, int64_t b) {
  if (p.lengths == nullptr) return p.length;
  const int64_t v = p.lengths[b];
  return v < 0 ? 0 : (v > p.length ? p.length : v);
}

}  // namespace sca
