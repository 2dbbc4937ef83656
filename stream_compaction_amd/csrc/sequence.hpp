// Shared by the sequence kernels (causal convolution, selective scan,
// embedding): vector loads and stores of activations, and the elementwise
// functions of a gated state space layer.
#pragma once

#include "device.hpp"
#include "launch.hpp"

namespace sca {

// The combine type is float everywhere here: activations widen exactly,
// parameters and states are float32, and each output is rounded once.
template <class F> constexpr int kVecElems = 16 / (int)sizeof(typename F::S);

// Outputs that the L2 caches (8 of 4 MB) cannot hold are stored past them where
// that gains (PAST below).  With inputs that no cache holds a convolution with 134
// MB of output, half of it padding, takes 47.5 us against 49.3, without padding 57.7
// against 60.7, a lookup of 67 MB (4 outputs in turn) 16.6 against 25.  With inputs
// in the 256 MB last-level cache, which such stores leave there, the convolution
// takes 34 us against 49.  With a kernel that reads the output behind it the two
// together take the same to within 4% either way, over 32 to 256 MB (a product
// behind 128 MB 110 against 114 us, behind 256 MB 183 against 180).  The one loss:
// an output that is written over and over unread (47.5 us against 39).
inline bool past_caches(int64_t bytes) { return bytes >= (32ll << 20); }

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// 2^v with the hardware instruction (1 ulp; results below 2^-126 flush to 0,
// which a decay factor that small may do).
__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float rcp_hw(float v) { return __builtin_amdgcn_rcpf(v); }

// sigmoid(v); v -> -inf gives rcp(inf) = 0, v -> inf gives 1.
__device__ __forceinline__ float sigmoid(float v) { return rcp_hw(1.0f + exp2_hw(-v * kLog2e)); }
// The greater and the lesser of two, a NaN if either is one.
__device__ __forceinline__ float at_least(float v, float low) {
  return __builtin_elementwise_maximum(v, low);
}
__device__ __forceinline__ float at_most(float v, float high) {
  return __builtin_elementwise_minimum(v, high);
}
// silu(v) = v sigmoid(v); v is kept finite, as -inf * 0 would be no number.
__device__ __forceinline__ float silu(float v) {
  v = at_least(v, -1e30f);
  return v * sigmoid(v);
}
// d silu / dv = s (1 + v (1 - s)), with 0 and 1 at the two ends.
__device__ __forceinline__ float silu_slope(float v) {
  v = at_most(at_least(v, -1e30f), 1e30f);
  const float s = sigmoid(v);
  return s * __builtin_fmaf(v, 1.0f - s, 1.0f);
}

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1].  The steps of
// a state space layer are small (1e-3 to 1e-1), where rounding 1 + e to w loses
// digits of e; c = e - (w - 1) is exactly what was lost (w - 1 is exact), and
// log(1 + e) = log(w) + c / w up to c^2, where c / w is c to within float32's
// half step (c is at most 2^-24, and w is 1 to within e where it matters).
__device__ __forceinline__ float softplus(float v) {
  const float e = exp2_hw(-__builtin_fabsf(v) * kLog2e);
  const float w = 1.0f + e, c = e - (w - 1.0f);
  return __builtin_fmaxf(v, 0.0f) + __builtin_fmaf(__builtin_amdgcn_logf(w), kLn2, c);
}

// E consecutive elements of a row as one load or store of 2 to 16 bytes.
template <class F, int E> struct RowIO {
  using S = typename F::S;
  struct Elems { S e[E]; };
  typedef uint32_t vec2 __attribute__((ext_vector_type(2)));
  using Raw = std::conditional_t<sizeof(Elems) == 16, u32x4,
              std::conditional_t<sizeof(Elems) == 8, vec2,
              std::conditional_t<sizeof(Elems) == 4, uint32_t, uint16_t>>>;
  // At any element, n > 0 of them exist: one access for a whole vector (global
  // accesses need no alignment), one by one at a row's end, where elements that do
  // not exist read as zero.
  static __device__ __forceinline__ Raw load_any(const S* p, int64_t n) {
    typedef Raw Loose __attribute__((aligned(sizeof(S))));
    if (n >= E) return *gptr<const Loose>((uintptr_t)p);
    Elems s = {};
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k < n) s.e[k] = *gptr<const S>((uintptr_t)(p + k));
    return __builtin_bit_cast(Raw, s);
  }
  static __device__ __forceinline__ void store_any(S* p, Raw r, int64_t n) {
    typedef Raw Loose __attribute__((aligned(sizeof(S))));
    if (n >= E) {
      *gptr<Loose>((uintptr_t)p) = r;
      return;
    }
    const Elems s = __builtin_bit_cast(Elems, r);
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k < n) *gptr<S>((uintptr_t)(p + k)) = s.e[k];
  }
  // aligned and whole (ALIGNED), or any
  template <bool ALIGNED> static __device__ __forceinline__ Raw get(const S* p, int64_t n) {
    if constexpr (ALIGNED) return load(p);
    return load_any(p, n);
  }
  template <bool ALIGNED> static __device__ __forceinline__ void put(S* p, Raw r, int64_t n) {
    if constexpr (ALIGNED) {
      store(p, r);
    } else {
      store_any(p, r, n);
    }
  }
  // all of them, aligned
  static __device__ __forceinline__ Raw load(const S* p) { return *gptr<const Raw>((uintptr_t)p); }
  static __device__ __forceinline__ void store(S* p, Raw r) { *gptr<Raw>((uintptr_t)p) = r; }
  template <bool PAST> static __device__ __forceinline__ void store_past(S* p, Raw r) {
    if constexpr (PAST) {
      __builtin_nontemporal_store(r, gptr<Raw>((uintptr_t)p));
    } else {
      store(p, r);
    }
  }
  static __device__ __forceinline__ void unpack(Raw r, float (&x)[E]) {
    const Elems s = __builtin_bit_cast(Elems, r);
#pragma unroll
    for (int k = 0; k < E; ++k) x[k] = widen<F>(s.e[k]);
  }
  static __device__ __forceinline__ Raw pack(const float (&x)[E]) {
    if constexpr (sizeof(S) == 2 && E > 1) {
      struct Words { uint32_t w[E / 2]; } s;
#pragma unroll
      for (int k = 0; k < E / 2; ++k) s.w[k] = narrow2<F>(x[2 * k], x[2 * k + 1]);
      return __builtin_bit_cast(Raw, s);
    } else {
      Elems s;
#pragma unroll
      for (int k = 0; k < E; ++k) s.e[k] = narrow<F>(x[k]);
      return __builtin_bit_cast(Raw, s);
    }
  }
};

// Stores v at `off` bytes (below 2^31) past the wave-uniform base, if `on`: a
// buffer store drops what lies outside the resource, so there is no branch.
template <class T>
__device__ __forceinline__ void store_if(const void* base, uint32_t off, bool on, T v) {
  const Buf b((uintptr_t)base, 0x7fffffff);
  const uint32_t at = on ? off : ~0u;
  if constexpr (sizeof(T) == 2) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), b.r, at, 0, 0);
  } else if constexpr (sizeof(T) == 4) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), b.r, at, 0, 0);
  } else {
    typedef uint32_t vec2 __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(vec2, v), b.r, at, 0, 0);
  }
}

// i = q d + r.  A 64-bit division costs some 150 instructions, a 32-bit one 25.
__device__ __forceinline__ int64_t divide(int64_t i, int64_t d, int64_t* r) {
  int64_t q;
  if (((uint64_t)(i | d) >> 32) == 0) {
    q = (int64_t)((uint32_t)i / (uint32_t)d);
  } else {
    q = i / d;
  }
  *r = i - q * d;
  return q;
}

// A barrier for data that waves exchange through LDS: unlike __syncthreads() it
// does not wait for the wave's global loads and stores.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Logical workgroup index: hardware deals consecutive workgroups to the 8
// XCDs in turn, each with its own L2.  Runs of 4 logical neighbours (which share
// the 128-byte lines of the activations) are put on one XCD and the runs dealt
// in turn, so that every XCD gets its part of each sequence, however long.  The
// grid is a multiple of 32 workgroups; logical indices may pass the last one.
__device__ __forceinline__ uint32_t xcd_order(uint32_t bid) {
  const uint32_t x = bid % 8, i = bid / 8;
  return (i / 4 * 8 + x) * 4 + i % 4;
}
inline unsigned xcd_grid(int64_t count) { return (unsigned)((count + 31) / 32 * 32); }

}  // namespace sca
