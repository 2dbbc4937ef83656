// Token embedding, out[i] = scale * weight[ids[i]], and the gradient of its
// table, dweight[v] = scale * sum over the tokens i with ids[i] = v of dout[i].
// Ids outside [0, rows) stand for masked tokens: their output is zero and they
// add to no row.
//
// The gradient sorts the tokens by id (the library's radix sort, stable), so
// that each table row is the sum of one run of sorted tokens, taken in token
// order: no float atomics, the same bits every time.  The sorted tokens are cut
// into segments of kSeg; a wave sums the runs of its segment (one table column
// block), writes the rows whose run lies inside, and leaves the sums of runs
// that cross a border to a second kernel.
#include "sequence.hpp"

namespace sca {

namespace {

template <class I>
__device__ __forceinline__ int64_t token_row(const I* ids, int64_t i, int64_t rows) {
  const int64_t v = (int64_t)ids[i];
  return v >= 0 && v < rows ? v : -1;
}

}  // namespace

template <class F, int E, class I>
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
      IO::unpack(IO::load((const S*)weight + row * row_stride + ch, channels - ch, E > 1), v);
#pragma unroll
      for (int c = 0; c < E; ++c) v[c] *= scale;
      r = IO::pack(v);
    }
    IO::store((S*)out + t * channels + ch, r, channels - ch, E > 1);
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

constexpr int kSeg = 32;          // sorted tokens per wave
constexpr int kSegAhead = 8;      // gradient rows loaded together

// A wave sums segment `seg` of the sorted tokens over one block of 64 E
// channels.  part[seg][0] gets the sum of the run that began before the
// segment, part[seg][1] that of the run that continues past it (both float32);
// a run that covers the whole segment and goes on at both ends is in [0].
template <class F, class G, int E>
__global__ __launch_bounds__(256) void embedding_segment_kernel(
    const void* dout, const uint32_t* keys, const uint32_t* pos, void* dweight, float* part,
    int64_t tokens, int64_t rows, int64_t channels, int64_t row_stride, float scale) {
  using S = typename F::S;
  using IO = RowIO<F, E>;
  constexpr int OE = E < kVecElems<G> ? E : kVecElems<G>;   // outputs per store
  using OIO = RowIO<G, OE>;
  const int lane = lane_id();
  const int64_t blocks = (channels + 64 * E - 1) / (64 * E);
  const int64_t total = (tokens + kSeg - 1) / kSeg * blocks;
  for (int64_t w = (int64_t)blockIdx.x * 4 + wave_id(); w < total; w += (int64_t)gridDim.x * 4) {
    const int64_t seg = w / blocks, s0 = seg * kSeg;
    const int64_t ch = (w % blocks * 64 + lane) * E, n = channels - ch;
    const int cnt = (int)(tokens - s0 < kSeg ? tokens - s0 : kSeg);
    // lane l holds the key and position of token s0 + l, lane kSeg the next
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
        if (j0 + j < cnt && n > 0) raw[j] = IO::load((const S*)dout + i * row_stride + ch, n, E > 1);
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
              OIO::store(to + h, OIO::pack(o), n - h, E > 1);
            }
          } else {
            float* to = out_part + (whole ? channels : 0);
#pragma unroll
            for (int c = 0; c < E; ++c)
              if (c < n) to[c] = sum[c];
          }
        }
#pragma unroll
        for (int c = 0; c < E; ++c) sum[c] = 0.0f;
        whole = true;
      }
    }
  }
}

// Runs that cross segments: the wave of the segment in which such a run begins
// adds its pieces in order and writes the row.
template <class G>
__global__ __launch_bounds__(256) void embedding_border_kernel(const uint32_t* keys, void* dweight,
                                                              const float* part, int64_t tokens,
                                                              int64_t rows, int64_t channels,
                                                              float scale) {
  const int64_t blocks = (channels + 63) / 64;
  const int64_t total = (tokens + kSeg - 1) / kSeg * blocks;
  for (int64_t w = (int64_t)blockIdx.x * 4 + wave_id(); w < total; w += (int64_t)gridDim.x * 4) {
    const int64_t seg = w / blocks, s0 = seg * kSeg, end = s0 + kSeg;
    if (end >= tokens) continue;                          // nothing follows the last segment
    const uint32_t k = keys[end - 1];
    if (k >= (uint32_t)rows || keys[end] != k) continue;  // no run continues past this segment
    if (s0 > 0 && keys[s0 - 1] == k) continue;            // it began in an earlier one
    const int64_t ch = w % blocks * 64 + lane_id();
    if (ch >= channels) continue;
    float sum = part[(seg * 2 + 1) * channels + ch];
    for (int64_t s = seg + 1;; ++s) {
      sum += part[s * 2 * channels + ch];
      const int64_t e = (s + 1) * kSeg;
      if (e >= tokens || keys[e - 1] != k || keys[e] != k) break;
    }
    ((typename G::S*)dweight)[(int64_t)k * channels + ch] = narrow<G>(sum * scale);
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
    const int64_t blocks = (tokens * (vec ? channels / E : channels) + 255) / 256;
    const dim3 grid((unsigned)(blocks < kGridMost ? blocks : kGridMost));
    auto go = [&](auto* id) {
      if (vec) {
        embedding_kernel<F, E><<<grid, dim3(256), 0, stream>>>(weight, id, out, tokens, rows,
                                                               channels, row_stride, scale);
      } else {
        embedding_kernel<F, 1><<<grid, dim3(256), 0, stream>>>(weight, id, out, tokens, rows,
                                                               channels, row_stride, scale);
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

// Scratch: keys, positions and their sort temporaries; the sort's own scratch;
// two float32 rows per segment.
namespace {
struct GradScratch {
  size_t keys, pos, tmp_keys, tmp_pos, sort, part, bytes;
};
GradScratch grad_scratch(int64_t tokens, int64_t channels) {
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  GradScratch s;
  const size_t list = up((size_t)tokens * 4);
  s.keys = 0;
  s.pos = list;
  s.tmp_keys = 2 * list;
  s.tmp_pos = 3 * list;
  s.sort = 4 * list;
  s.part = s.sort + up(radix_sort_scratch(tokens, 4));
  s.bytes = s.part + up((size_t)((tokens + kSeg - 1) / kSeg) * 2 * (size_t)channels * 4);
  return s;
}
}  // namespace
size_t embedding_grad_scratch(int64_t tokens, int64_t rows, int64_t channels) {
  (void)rows;
  return tokens == 0 ? 0 : grad_scratch(tokens, channels).bytes;
}

hipError_t launch_embedding_grad(const void* dout, const void* ids, bool wide_ids, void* dweight,
                                 int64_t tokens, int64_t rows, int64_t channels,
                                 int64_t row_stride, Fmt fmt, Fmt out_fmt, float scale,
                                 void* scratch, hipStream_t stream) {
  const int out_bytes = out_fmt == Fmt::F32 ? 4 : 2;
  {
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
  if (tokens == 0) return hipGetLastError();
  const GradScratch g = grad_scratch(tokens, channels);
  char* base = (char*)scratch;
  uint32_t* keys = (uint32_t*)(base + g.keys);
  uint32_t* pos = (uint32_t*)(base + g.pos);
  const dim3 tgrid((unsigned)((tokens + 255) / 256));
  if (wide_ids) {
    embedding_keys_kernel<<<tgrid, dim3(256), 0, stream>>>((const int64_t*)ids, tokens, rows, keys, pos);
  } else {
    embedding_keys_kernel<<<tgrid, dim3(256), 0, stream>>>((const int32_t*)ids, tokens, rows, keys, pos);
  }
  int bits = 8;                       // keys go up to `rows`
  while (bits < 32 && ((uint64_t)rows >> bits) != 0) bits += 8;
  hipError_t e = launch_radix_sort(keys, base + g.tmp_keys, pos, base + g.tmp_pos, tokens, Fmt::U32,
                                   4, bits, base + g.sort, stream);
  if (e != hipSuccess) return e;
  float* part = (float*)(base + g.part);
  const int64_t segs = (tokens + kSeg - 1) / kSeg;
  return by_format(fmt, [&](auto f) {
    using F = decltype(f);
    auto go = [&](auto o) {
      using G = decltype(o);
      constexpr int E = kVecElems<F>;
      const bool vec = channels % E == 0 && row_stride % E == 0 && (uintptr_t)dout % 16 == 0 &&
                       (uintptr_t)dweight % 16 == 0;
      const int64_t waves = segs * ((channels + 64 * (vec ? E : 1) - 1) / (64 * (vec ? E : 1)));
      auto grid_of = [](int64_t w) {
        const int64_t b = (w + 3) / 4;
        return dim3((unsigned)(b < kGridMost ? b : kGridMost));
      };
      const dim3 grid = grid_of(waves);
      if (vec) {
        embedding_segment_kernel<F, G, E><<<grid, dim3(256), 0, stream>>>(
            dout, keys, pos, dweight, part, tokens, rows, channels, row_stride, scale);
      } else {
        embedding_segment_kernel<F, G, 1><<<grid, dim3(256), 0, stream>>>(
            dout, keys, pos, dweight, part, tokens, rows, channels, row_stride, scale);
      }
      const int64_t bw = segs * ((channels + 63) / 64);
      embedding_border_kernel<G><<<grid_of(bw), dim3(256), 0, stream>>>(
          keys, dweight, part, tokens, rows, channels, scale);
      return hipGetLastError();
    };
    // the table's gradient in the activations' type or in float32
    if (out_fmt == Fmt::F32) return go(FmtF32{});
    return go(F{});
  });
}

}  // namespace sca
