// The global norm of the ranks' gradients, and their clipping by it (see vc.h).
//
// Two passes over memory: squares are summed, then every gradient is scaled.
// The second walks the chunks in the opposite order, so that it begins on what
// the first left in L2.  Memory bounds both.  On a GB300 (copy rate 6.78 TB/s):
// 2.4 GB of bf16 gradients in 1536 tensors, 390 us for the norm (6.2 TB/s) and
// 740 us for the clipping (6.5 TB/s); 34 MB in 64 tensors 24 us together.
#include <iterator>
#include <memory>

#include "layer.cuh"

namespace vc {
namespace layer {
namespace {

constexpr int kClipThreads = 256, kClipUnits = 8;
// Blocks of a multiprocessor, by their registers.  24 layers' 2.4 GB, eight
// ranks: the norm 400 us with 4 and 419 with 3 (what its loads need), clipping
// 749 with 3 and 860 with 4 (which spills).
constexpr int kNormBlocks = 4, kClipBlocks = 3;
constexpr int64_t kChunkBytes = int64_t(kClipThreads) * kClipUnits * 16;  // of one tensor, at most, at a time

struct Tensor {
  const char* g;
  char* out;
  int64_t n;
};
// What both sizes of table have.
struct ClipCall {
  uint16_t first[VC_MAX_RANKS + 1];  // of a rank's tensors
  double* part;          // [rank][block], of the launches so far
  float* norm[VC_MAX_RANKS];
  float max_norm;
  uint32_t blocks;       // parts of a rank
  uint32_t at;           // launch
  bool across;
};
// The tensors of one launch.  A call of few copies a small table.
template <int N>
struct ClipParams : ClipCall {
  static constexpr int kTable = N;
  Tensor t[N];
  uint32_t end[N];  // chunks of the rank's tensors so far in this launch
  uint8_t dtype[N];
};
constexpr int kFew = 96, kMany = 768;
// Above this many bytes a clipping call's blocks do not come in before the launch
// ahead has ended.  Behind a clipping launch that costs more than the launch's
// latency that it hides: calls one after another, 8 ranks of 96 tensors, 131 us
// with blocks that come in early and 118 without for 128 MB, 199 and 175 for 256
// MB (8 tensors: 143 and 136), but 24.7 and 29.2 for 32 MB of 8 tensors.  The
// norm alone is faster with them at every size (43 and 50 us for 128 MB).
constexpr int64_t kLateBytes = 64 << 20;

// A chunk: `n` elements at g and out.
struct Chunk {
  const Tensor* t;
  const char* g;
  char* out;
  int64_t n;
  int dtype;
};
template <class P>
__device__ __forceinline__ Chunk chunk_at(const P& p, int rank, uint32_t c) {
  int lo = p.first[rank], hi = p.first[rank + 1] - 1;
  const int base = lo;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.end[mid] > c) hi = mid; else lo = mid + 1;
  }
  Chunk x;
  x.t = p.t + lo;
  x.dtype = p.dtype[lo];
  const int es = x.dtype == VC_FLOAT32 ? 4 : 2;
  const int64_t at = static_cast<int64_t>(c - (lo > base ? p.end[lo - 1] : 0)) * kChunkBytes;
  x.g = x.t->g + at;
  x.out = x.t->out + at;
  x.n = min(kChunkBytes / es, x.t->n - at / es);
  return x;
}
template <class P>
__device__ __forceinline__ uint32_t chunks_of(const P& p, int rank) {
  return p.first[rank + 1] > p.first[rank] ? p.end[p.first[rank + 1] - 1] : 0;
}

template <class F>
__device__ __forceinline__ void by_dtype(int dtype, F&& f) {
  if (dtype == VC_BFLOAT16) f(std::integral_constant<int, VC_BFLOAT16>{});
  else if (dtype == VC_FLOAT32) f(std::integral_constant<int, VC_FLOAT32>{});
  else f(std::integral_constant<int, VC_FLOAT16>{});
}

// Sum over the block of doubles, in a fixed order, the same in every thread.
__device__ __forceinline__ double block_sum(double x, double* part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  double all = 0;
#pragma unroll
  for (int i = 0; i < kClipThreads / 32; ++i) all += part[i];
  return all;
}

// A thread's units of a chunk, all loaded before `f` takes the first.  Off
// 16-byte boundaries a unit is cut out of two loads: half as many at a time.
// `between` runs once, while loads are on their way.
template <int DT, bool VEC, class B, class F>
__device__ __forceinline__ void units(const Chunk& x, B&& between, F&& f) {
  using E = El<DT>;
  constexpr int kN = VEC ? kClipUnits : kClipUnits / 2;
  const int units = static_cast<int>((x.n + E::kVec - 1) / E::kVec);
  const Row<E::kSize, VEC> row(x.g, units, Bytes{x.t->g, x.t->g + x.t->n * E::kSize});
#pragma unroll
  for (int i0 = 0; i0 < kClipUnits; i0 += kN) {
    typename Row<E::kSize, VEC>::Raw raw[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i0 + i) * kClipThreads + threadIdx.x;
      raw[i] = c < units ? row.load_plain(c) : row.zero();
    }
    if (i0 == 0) between();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i0 + i) * kClipThreads + threadIdx.x;
      if ((c & ~31) >= units) break;
      float v[E::kVec] = {};
      if (c < units) {
        E::widen(row.finish(raw[i], c, x.n), v);
        mask_unit<E::kSize, VEC>(c, x.n, v);
      }
      f(c, v);
    }
  }
}

// The sum of a thread's squares in a chunk.  Up to 64 are added in fp32, whose
// numbers end at 2^128 and lose bits below 2^-126: within [kLow, kHigh] what a
// sum has lost is below 2^-34 of it.  Elsewhere they are added again, of the
// elements times a power of two:
//   below 2^-110 every element is below 2^-55, and the squares of 2^100 times
//   them lie between 2^-98 (2^-149 is the smallest number) and 2^90;
//   above 2^100 (or infinite, or NaN) one element is above 2^46; the squares of
//   2^-76 times them lie below 2^104, and what is lost of those below 2^-126
//   is nothing next to the largest, above 2^-60.
// fp16's squares are within 2^-48 and 2^32.  The loaded units are kept for that,
// which is why this has a loop of its own.
constexpr float kLow = 0x1p-110f, kHigh = 0x1p100f;
template <int DT, bool VEC, class B>
__device__ __forceinline__ double squares(const Chunk& x, B&& between) {
  using E = El<DT>;
  constexpr int kN = VEC ? kClipUnits : kClipUnits / 2;  // as in units()
  const int units = static_cast<int>((x.n + E::kVec - 1) / E::kVec);
  const Row<E::kSize, VEC> row(x.g, units, Bytes{x.t->g, x.t->g + x.t->n * E::kSize});
  double sum = 0;
#pragma unroll
  for (int i0 = 0; i0 < kClipUnits; i0 += kN) {
    typename Row<E::kSize, VEC>::Raw raw[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = (i0 + i) * kClipThreads + threadIdx.x;
      raw[i] = c < units ? row.load_plain(c) : row.zero();
    }
    if (i0 == 0) between();
    const auto add = [&](float by) {
      float s[4] = {};
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int c = (i0 + i) * kClipThreads + threadIdx.x;
        if ((c & ~31) >= units) break;
        float v[E::kVec] = {};
        if (c < units) {
          E::widen(row.finish(raw[i], c, x.n), v);
          mask_unit<E::kSize, VEC>(c, x.n, v);
        }
#pragma unroll
        for (int k = 0; k < E::kVec; ++k) s[k % 4] = fmaf(v[k] * by, v[k] * by, s[k % 4]);
      }
      return (s[0] + s[1]) + (s[2] + s[3]);
    };
    const float all = add(1.f);
    if (DT == VC_FLOAT16 || (all >= kLow && all <= kHigh)) {
      sum += all;
      continue;
    }
    if constexpr (VEC) {  // zeros are common: 2.4 GB of them take 403 us so, 609 added again
      constexpr uint32_t kMagnitude = E::kSize == 4 ? 0x7fffffff : 0x7fff7fff;
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) any |= raw[i].x | raw[i].y | raw[i].z | raw[i].w;
      if ((any & kMagnitude) == 0) continue;
    }
    sum += add(all < kLow ? 0x1p100f : 0x1p-76f) * (all < kLow ? 0x1p-200 : 0x1p152);
  }
  return sum;
}

template <class P>
__global__ void __launch_bounds__(kClipThreads, kNormBlocks) grad_norm_kernel(const __grid_constant__ P p) {
  __shared__ double part[kClipThreads / 32];
  stream_order();
  const int rank = blockIdx.y;
  const uint32_t total = chunks_of(p, rank);
  double sum = 0;
  if (p.at != 0 && threadIdx.x == 0) sum = __ldcg(p.part + static_cast<int64_t>(rank) * p.blocks + blockIdx.x);  // the last launch's
  Chunk x, next{};
  if (blockIdx.x < total) next = chunk_at(p, rank, blockIdx.x);
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    x = next;
    by_dtype(x.dtype, [&](auto code) {
      constexpr int DT = decltype(code)::value;
      const auto go = [&](auto vec) {
        sum += squares<DT, decltype(vec)::value>(x, [&] { if (c + gridDim.x < total) next = chunk_at(p, rank, c + gridDim.x); });
      };
      const bool whole = reinterpret_cast<uintptr_t>(x.g) % 16 == 0 && x.n % El<DT>::kVec == 0;
      whole ? go(std::true_type{}) : go(std::false_type{});
    });
  }
  sum = block_sum(sum, part);
  if (threadIdx.x == 0) p.part[static_cast<int64_t>(rank) * p.blocks + blockIdx.x] = sum;
}

// The norm that rank `rank` goes by, from every block's part, however many
// launches there were: each block of each clipping launch adds them up.
__device__ __forceinline__ float norm_of(const ClipCall& p, int rank, int ranks, double* part) {
  double sum = 0;
  const uint32_t first = p.across ? 0 : rank * p.blocks, last = p.across ? ranks * p.blocks : first + p.blocks;
  for (uint32_t i = first + threadIdx.x; i < last; i += kClipThreads) sum += __ldcg(p.part + i);
  return static_cast<float>(sqrt(block_sum(sum, part)));
}

// In place too: a unit's bytes are written by its own warp alone, after it has
// loaded them, and of what else its loads bring nothing is used.
template <class P>
__global__ void __launch_bounds__(kClipThreads, kClipBlocks) clip_kernel(const __grid_constant__ P p) {
  __shared__ double part[kClipThreads / 32];
  __shared__ __align__(16) unsigned char rooms[kClipThreads / 32][Span<2, 16, false>::kRoom];
  stream_order();
  const int rank = blockIdx.y;
  unsigned char* room = rooms[threadIdx.x / 32];
  const float norm = norm_of(p, rank, gridDim.y, part);
  if (p.at == 0 && blockIdx.x == 0 && threadIdx.x == 0) *p.norm[rank] = norm;
  const float by = norm <= p.max_norm ? 1.f : __fdiv_rn(p.max_norm, norm);
  const uint32_t total = chunks_of(p, rank);
  Chunk x, next{};
  if (blockIdx.x < total) next = chunk_at(p, rank, total - 1 - blockIdx.x);
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    x = next;
    const auto ahead = [&] { if (c + gridDim.x < total) next = chunk_at(p, rank, total - 1 - c - gridDim.x); };
    if (by == 1.f && x.g == x.out) {
      ahead();
      continue;
    }
    by_dtype(x.dtype, [&](auto code) {
      constexpr int DT = decltype(code)::value;
      const auto go = [&](auto vec) {
        constexpr bool VEC = decltype(vec)::value;
        units<DT, VEC>(x, ahead, [&](int u, float* v) {
#pragma unroll
          for (int k = 0; k < El<DT>::kVec; ++k) v[k] *= by;
          Span<El<DT>::kSize, 16, VEC>(room, El<DT>::narrow(v)).template write<true>(x.out, u & ~31, x.n);
        });
      };
      const bool whole = (reinterpret_cast<uintptr_t>(x.g) | reinterpret_cast<uintptr_t>(x.out)) % 16 == 0 && x.n % El<DT>::kVec == 0;
      whole ? go(std::true_type{}) : go(std::false_type{});
    });
  }
}

__global__ void __launch_bounds__(kClipThreads) norm_kernel(const __grid_constant__ ClipCall p) {
  __shared__ double part[kClipThreads / 32];
  stream_order();
  const float norm = norm_of(p, blockIdx.x, gridDim.x, part);
  if (threadIdx.x == 0) *p.norm[blockIdx.x] = norm;
}

// No output over another buffer; an output may be its own gradient.
vc_status_t check_apart(const void* const* g, void* const* out, const size_t* counts, const vc_dtype_t* dtypes, size_t tensors,
                        int nranks, float* const* norm) {
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  // As a rule a rank's tensors lie one behind another, or a few runs of them
  // do: runs that do not interleave have no overlaps.
  std::vector<Range> ranges;
  const auto every = [&](auto&& add) {
    for (int pass = 0; pass < (out ? 2 : 1); ++pass)
      for (size_t i = 0; i < tensors * nranks; ++i) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(pass ? out[i] : g[i]);
        const uintptr_t bytes = counts[i] * static_cast<uintptr_t>(dtype_size(dtypes[i % tensors]));
        if (bytes && (pass || !out || out[i] != g[i])) add(Range{lo, lo + bytes, pass != 0});
      }
    for (int r = 0; r < nranks; ++r) add(Range{reinterpret_cast<uintptr_t>(norm[r]), reinterpret_cast<uintptr_t>(norm[r]) + 4, true});
  };
  const auto apart = [&] {
    std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t any = 0, outs = 0;
    for (const Range& x : ranges) {
      if (x.lo < outs || (x.out && x.lo < any)) return false;
      any = std::max(any, x.hi);
      if (x.out) outs = std::max(outs, x.hi);
    }
    return true;
  };
  every([&](const Range& x) {
    if (!ranges.empty() && ranges.back().out == x.out && x.lo >= ranges.back().hi) ranges.back().hi = x.hi;
    else ranges.push_back(x);
  });
  if (apart()) return VC_SUCCESS;
  ranges.clear();
  every([&](const Range& x) { ranges.push_back(x); });
  return apart() ? VC_SUCCESS : fail(VC_ERR_INVALID_ARG, "an output buffer overlaps another buffer");
}

// The call's launches, with tables of P's size.
template <class P>
vc_status_t clip_with(const void* const* g, void* const* out, const size_t* counts, const vc_dtype_t* dtypes, int nranks, size_t tensors,
                      float* const* norm, double max_norm, int across, int64_t bytes, cudaStream_t stream) {
  DeviceState* st = nullptr;
  int dev = 0;
  vc_status_t rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  // the tensors that hold something, cut into tables by rank
  std::vector<std::unique_ptr<P>> tables;
  uint32_t most = 0;  // chunks of the rank that has most, in any table
  int filled = P::kTable;
  const auto open = [&] {
    tables.emplace_back(new P);  // of the arrays, what is filled is looked at
    std::fill(std::begin(tables.back()->first), std::end(tables.back()->first), uint16_t(0));
    filled = 0;
  };
  for (int r = 0; r < nranks; ++r) {
    uint32_t end = 0;
    for (size_t i = 0; i < tensors; ++i) {
      const size_t at = r * tensors + i;
      if (counts[at] == 0) continue;
      if (filled == P::kTable) {
        if (!tables.empty())
          for (int q = r + 1; q <= nranks; ++q) tables.back()->first[q] = static_cast<uint16_t>(filled);
        open();
        end = 0;
      }
      P& p = *tables.back();
      const int64_t size = static_cast<int64_t>(counts[at]) * dtype_size(dtypes[i]);
      p.t[filled] = Tensor{static_cast<const char*>(g[at]), out ? static_cast<char*>(out[at]) : nullptr, static_cast<int64_t>(counts[at])};
      p.dtype[filled] = static_cast<uint8_t>(dtypes[i]);
      end += static_cast<uint32_t>((size + kChunkBytes - 1) / kChunkBytes);
      p.end[filled++] = end;
      most = std::max(most, end);
    }
    if (!tables.empty()) tables.back()->first[r + 1] = static_cast<uint16_t>(filled);
  }
  if (tables.empty()) open();
  const uint32_t launches = static_cast<uint32_t>(tables.size());
  const auto blocks_of = [&](int resident) {
    const int64_t fit = (int64_t(st->nsm) * resident + nranks - 1) / nranks;
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(fit, most)));
  };
  const unsigned blocks = blocks_of(resident_blocks<grad_norm_kernel<P>>(dev, kClipThreads, 0));
  const unsigned clip_blocks = blocks_of(resident_blocks<clip_kernel<P>>(dev, kClipThreads, 0));
  cudaMemPool_t pool;
  rc = scratch_pool(st, dev, &pool);
  if (rc != VC_SUCCESS) return rc;
  double* part = nullptr;
  const size_t need = sizeof(double) * nranks * blocks;
  cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void**>(&part), need, pool, stream);
  if (e == cudaErrorMemoryAllocation) {
    cudaGetLastError();
    return fail(VC_ERR_NOMEM, "scratch allocation of " + std::to_string(need) + " bytes failed");
  }
  if (e != cudaSuccess) return cuda_fail(e, "cudaMallocFromPoolAsync");
  const unsigned n = static_cast<unsigned>(nranks);
  const bool early = !out || bytes <= kLateBytes;
  int step = 0;
  for (uint32_t i = 0; i < launches && rc == VC_SUCCESS; ++i) {
    P& p = *tables[i];
    std::copy(norm, norm + nranks, p.norm);
    p.part = part;
    p.blocks = blocks;
    p.at = i;
    p.across = across != 0;
    p.max_norm = static_cast<float>(max_norm);
    rc = launch<grad_norm_kernel<P>>(dev, Shape{blocks, kClipThreads, 0, 1, n, early}, stream, p, kGradNorm, step++, i == 0 ? bytes : 0);
  }
  if (rc == VC_SUCCESS && !out)
    rc = launch<norm_kernel, ClipCall>(dev, Shape{n, kClipThreads}, stream, *tables[0], kGradNorm, step++, static_cast<int64_t>(need));
  // the last table first: its gradients are the ones left in L2
  for (uint32_t i = launches; out && i-- > 0 && rc == VC_SUCCESS;)
    rc = launch<clip_kernel<P>>(dev, Shape{clip_blocks, kClipThreads, 0, 1, n, early}, stream, *tables[i], kClip, step++, i == 0 ? 2 * bytes : 0);
  e = cudaFreeAsync(part, stream);
  if (e != cudaSuccess && rc == VC_SUCCESS) rc = cuda_fail(e, "cudaFreeAsync");
  return rc;
}

vc_status_t clip(const void* const* g, void* const* out, const size_t* counts, const vc_dtype_t* dtypes, int nranks, size_t tensors,
                 float* const* norm, double max_norm, int across, cudaStream_t stream) {
  vc_status_t rc = check_ranks(nranks);
  if (rc != VC_SUCCESS) return rc;
  if (tensors > (size_t(1) << 20)) return fail(VC_ERR_INVALID_ARG, "too many tensors");
  if (!norm || (tensors && (!g || !counts || !dtypes))) return fail(VC_ERR_INVALID_ARG, "null array");
  if (out && !(max_norm >= 0)) return fail(VC_ERR_INVALID_ARG, "max_norm must not be negative or NaN");
  for (size_t i = 0; i < tensors; ++i) {
    rc = check_float(dtypes[i]);
    if (rc != VC_SUCCESS) return rc;
  }
  int64_t bytes = 0;
  for (int r = 0; r < nranks; ++r) {
    if (!norm[r]) return fail(VC_ERR_INVALID_ARG, "null norm buffer");
    if (reinterpret_cast<uintptr_t>(norm[r]) % 4) return fail(VC_ERR_INVALID_ARG, "norm is not aligned to its element");
    for (size_t i = 0; i < tensors; ++i) {
      const size_t at = r * tensors + i;
      const int es = dtype_size(dtypes[i]);
      if (counts[at] > (uint64_t(1) << 40)) return fail(VC_ERR_INVALID_ARG, "a tensor of more than 2^40 elements");
      bytes += static_cast<int64_t>(counts[at]) * es;
      if (bytes > (int64_t(1) << 44)) return fail(VC_ERR_INVALID_ARG, "more than 2^44 bytes of gradients");
      if (counts[at] == 0) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(g[at]), b = out ? reinterpret_cast<uintptr_t>(out[at]) : a;
      if (!a || !b) return fail(VC_ERR_INVALID_ARG, "null gradient buffer");
      if ((a | b) % es) return fail(VC_ERR_INVALID_ARG, "a gradient is not aligned to its element");
    }
  }
  rc = check_apart(g, out, counts, dtypes, tensors, nranks, norm);
  if (rc != VC_SUCCESS) return rc;
  if (tensors * nranks <= kFew)
    return clip_with<ClipParams<kFew>>(g, out, counts, dtypes, nranks, tensors, norm, max_norm, across, bytes, stream);
  return clip_with<ClipParams<kMany>>(g, out, counts, dtypes, nranks, tensors, norm, max_norm, across, bytes, stream);
}

}  // namespace
}  // namespace layer
}  // namespace vc

using namespace vc;

VC_EXPORT vc_status_t vc_clip_grad_norm(const void* const* grads, void* const* out, const size_t* counts,
                                        const vc_dtype_t* dtypes, int nranks, size_t ntensors, float* const* norm,
                                        double max_norm, int across, vc_stream_t stream) {
  return entry([&] {
    return layer::clip(grads, out, counts, dtypes, nranks, ntensors, norm, max_norm, across,
                       reinterpret_cast<cudaStream_t>(stream));
  });
}
