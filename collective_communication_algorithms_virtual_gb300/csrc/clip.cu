// The global norm of the ranks' gradients, and their clipping by it (see vc.h).
//
// Two passes over memory: squares are summed, then every gradient is scaled.
// The second walks the chunks in the opposite order, so that it begins on what
// the first left in L2.
#include "layer.cuh"

namespace vc {
namespace layer {
namespace {

constexpr int kClipThreads = 256, kClipUnits = 8;
constexpr int64_t kChunkBytes = int64_t(kClipThreads) * kClipUnits * 16;  // of one tensor, at most, at a time
constexpr int kTable = 768;  // tensors of one launch

struct Tensor {
  const char* g;
  char* out;
  int64_t n;
};
struct ClipParams {
  Tensor t[kTable];
  uint32_t end[kTable];  // chunks of the rank's tensors so far in this launch
  uint8_t dtype[kTable];
  uint16_t first[VC_MAX_RANKS + 1];  // of a rank's tensors
  double* part;          // [launch][rank][block]
  float* norm[VC_MAX_RANKS];
  float max_norm;
  uint32_t blocks;       // parts of a rank and launch
  uint32_t launches, at;
  bool across;
};

// A chunk: `n` elements at g and out.
struct Chunk {
  const Tensor* t;
  const char* g;
  char* out;
  int64_t n;
  int dtype;
};
__device__ __forceinline__ Chunk chunk_at(const ClipParams& p, int rank, uint32_t c) {
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

template <int DT, bool VEC>
__device__ __forceinline__ float squares(const Chunk& x) {
  using E = El<DT>;
  const int units = static_cast<int>((x.n + E::kVec - 1) / E::kVec);
  const Row<E::kSize, VEC> row(x.g, units, Bytes{x.t->g, x.t->g + x.t->n * E::kSize});
  typename Row<E::kSize, VEC>::Raw raw[kClipUnits];
#pragma unroll
  for (int i = 0; i < kClipUnits; ++i) {
    const int c = i * kClipThreads + threadIdx.x;
    raw[i] = c < units ? row.load(c) : row.zero();
  }
  float sum[4] = {};
#pragma unroll
  for (int i = 0; i < kClipUnits; ++i) {
    const int c = i * kClipThreads + threadIdx.x;
    if (c >= units) break;
    float f[E::kVec];
    E::widen(row.finish(raw[i], c, x.n), f);
    mask_unit<E::kSize, VEC>(c, x.n, f);
#pragma unroll
    for (int k = 0; k < E::kVec; ++k) sum[k % 4] = fmaf(f[k], f[k], sum[k % 4]);
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_kernel(const __grid_constant__ ClipParams p) {
  __shared__ double part[kClipThreads / 32];
  stream_order();
  const int rank = blockIdx.y;
  const uint32_t total = p.first[rank + 1] > p.first[rank] ? p.end[p.first[rank + 1] - 1] : 0;
  double sum = 0;
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    const Chunk x = chunk_at(p, rank, c);
    by_dtype(x.dtype, [&](auto code) {
      constexpr int DT = decltype(code)::value;
      const bool whole = reinterpret_cast<uintptr_t>(x.g) % 16 == 0 && x.n % El<DT>::kVec == 0;
      sum += whole ? squares<DT, true>(x) : squares<DT, false>(x);
    });
  }
  sum = block_sum(sum, part);
  if (threadIdx.x == 0) p.part[(static_cast<int64_t>(p.at) * gridDim.y + rank) * p.blocks + blockIdx.x] = sum;
}

// The norm that rank `rank` goes by, from every block's part.
__device__ __forceinline__ float norm_of(const ClipParams& p, int rank, int ranks, double* part) {
  double sum = 0;
  const int64_t all = static_cast<int64_t>(p.launches) * ranks * p.blocks;
  for (int64_t i = threadIdx.x; i < all; i += kClipThreads)
    if (p.across || static_cast<int>(i / p.blocks % ranks) == rank) sum += __ldcg(p.part + i);
  return static_cast<float>(sqrt(block_sum(sum, part)));
}

template <int DT, bool VEC>
__device__ __forceinline__ void scale_chunk(const Chunk& x, float by, unsigned char* room) {
  using E = El<DT>;
  const int units = static_cast<int>((x.n + E::kVec - 1) / E::kVec);
  const Row<E::kSize, VEC> row(x.g, units, Bytes{x.t->g, x.t->g + x.t->n * E::kSize});
  typename Row<E::kSize, VEC>::Raw raw[kClipUnits];
#pragma unroll
  for (int i = 0; i < kClipUnits; ++i) {
    const int c = i * kClipThreads + threadIdx.x;
    raw[i] = c < units ? row.load_plain(c) : row.zero();
  }
  if constexpr (!VEC) __syncthreads();  // in place: a unit is cut out of a neighbour's bytes too
#pragma unroll
  for (int i = 0; i < kClipUnits; ++i) {
    const int c = i * kClipThreads + threadIdx.x, c0 = c & ~31;
    if (c0 >= units) break;
    float f[E::kVec];
    E::widen(row.finish(raw[i], c, x.n), f);
#pragma unroll
    for (int k = 0; k < E::kVec; ++k) f[k] *= by;
    Span<E::kSize, 16, VEC>(room, E::narrow(f)).template write<true>(x.out, c0, x.n);
  }
}

__global__ void __launch_bounds__(kClipThreads) clip_kernel(const __grid_constant__ ClipParams p) {
  __shared__ double part[kClipThreads / 32];
  __shared__ __align__(16) unsigned char room[kClipThreads / 32][Span<2, 16, false>::kRoom];
  stream_order();
  const int rank = blockIdx.y;
  const float norm = norm_of(p, rank, gridDim.y, part);
  if (p.at == 0 && blockIdx.x == 0 && threadIdx.x == 0) *p.norm[rank] = norm;
  const float by = norm <= p.max_norm ? 1.f : __fdiv_rn(p.max_norm, norm);
  const uint32_t total = p.first[rank + 1] > p.first[rank] ? p.end[p.first[rank + 1] - 1] : 0;
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    const Chunk x = chunk_at(p, rank, total - 1 - i);
    if (by == 1.f && x.g == x.out) continue;
    by_dtype(x.dtype, [&](auto code) {
      constexpr int DT = decltype(code)::value;
      const bool whole = (reinterpret_cast<uintptr_t>(x.g) | reinterpret_cast<uintptr_t>(x.out)) % 16 == 0 && x.n % El<DT>::kVec == 0;
      whole ? scale_chunk<DT, true>(x, by, room[threadIdx.x / 32]) : scale_chunk<DT, false>(x, by, room[threadIdx.x / 32]);
    });
  }
}

__global__ void __launch_bounds__(kClipThreads) norm_kernel(const __grid_constant__ ClipParams p) {
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
  std::vector<Range> ranges;
  ranges.reserve(tensors * nranks * 2 + nranks);
  const auto add = [&](const void* p, int64_t bytes, bool o) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (bytes) ranges.push_back(Range{lo, lo + static_cast<uintptr_t>(bytes), o});
  };
  for (size_t i = 0; i < tensors * nranks; ++i) {
    const int64_t bytes = static_cast<int64_t>(counts[i]) * dtype_size(dtypes[i % tensors]);
    if (!out || out[i] != g[i]) add(g[i], bytes, false);
    if (out) add(out[i], bytes, true);
  }
  for (int r = 0; r < nranks; ++r) add(norm[r], 4, true);
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t any = 0, outs = 0;
  for (const Range& x : ranges) {
    if (x.lo < outs || (x.out && x.lo < any)) return fail(VC_ERR_INVALID_ARG, "an output buffer overlaps another buffer");
    any = std::max(any, x.hi);
    if (x.out) outs = std::max(outs, x.hi);
  }
  return VC_SUCCESS;
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
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;

  // the tensors that hold something, cut into tables by rank
  std::vector<ClipParams> tables;
  std::vector<uint32_t> most;  // chunks of the rank that has most, of each table
  int64_t chunks = 0;
  int filled = kTable;
  for (int r = 0; r < nranks; ++r) {
    uint32_t end = 0;
    for (size_t i = 0; i < tensors; ++i) {
      const size_t at = r * tensors + i;
      if (counts[at] == 0) continue;
      if (filled == kTable) {
        if (!tables.empty())
          for (int q = r + 1; q <= nranks; ++q) tables.back().first[q] = static_cast<uint16_t>(filled);
        tables.emplace_back();
        most.push_back(0);
        for (int q = 0; q <= nranks; ++q) tables.back().first[q] = 0;
        filled = 0;
        end = 0;
      }
      ClipParams& p = tables.back();
      const int64_t bytes = static_cast<int64_t>(counts[at]) * dtype_size(dtypes[i]), n = (bytes + kChunkBytes - 1) / kChunkBytes;
      p.t[filled] = Tensor{static_cast<const char*>(g[at]), out ? static_cast<char*>(out[at]) : nullptr, static_cast<int64_t>(counts[at])};
      p.dtype[filled] = static_cast<uint8_t>(dtypes[i]);
      end += static_cast<uint32_t>(n);
      chunks += n;
      p.end[filled++] = end;
      most.back() = std::max(most.back(), end);
    }
    if (!tables.empty()) tables.back().first[r + 1] = static_cast<uint16_t>(filled);
  }
  if (tables.empty()) {
    tables.emplace_back();
    most.push_back(0);
    for (int q = 0; q <= nranks; ++q) tables.back().first[q] = 0;
  }
  const uint32_t launches = static_cast<uint32_t>(tables.size());
  const auto blocks_of = [&](int resident) {
    const int64_t fit = (int64_t(st->nsm) * resident + nranks - 1) / nranks;
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(fit, *std::max_element(most.begin(), most.end()))));
  };
  const unsigned blocks = blocks_of(resident_blocks<grad_norm_kernel>(dev, kClipThreads, 0));
  const unsigned clip_blocks = blocks_of(resident_blocks<clip_kernel>(dev, kClipThreads, 0));
  cudaMemPool_t pool;
  rc = scratch_pool(st, dev, &pool);
  if (rc != VC_SUCCESS) return rc;
  double* part = nullptr;
  const size_t need = sizeof(double) * launches * nranks * blocks;
  cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void**>(&part), need, pool, stream);
  if (e == cudaErrorMemoryAllocation) {
    cudaGetLastError();
    return fail(VC_ERR_NOMEM, "scratch allocation of " + std::to_string(need) + " bytes failed");
  }
  if (e != cudaSuccess) return cuda_fail(e, "cudaMallocFromPoolAsync");
  const unsigned n = static_cast<unsigned>(nranks);
  int step = 0;
  for (uint32_t i = 0; i < launches; ++i) {
    ClipParams& p = tables[i];
    for (int r = 0; r < nranks; ++r) p.norm[r] = norm[r];
    p.part = part;
    p.blocks = blocks;
    p.launches = launches;
    p.at = i;
    p.across = across != 0;
    p.max_norm = static_cast<float>(max_norm);
    if (rc == VC_SUCCESS)
      rc = launch<grad_norm_kernel>(dev, Shape{blocks, kClipThreads, 0, 1, n}, stream, p, kGradNorm, step++, i == 0 ? bytes : 0);
  }
  if (rc == VC_SUCCESS && !out)
    rc = launch<norm_kernel>(dev, Shape{n, kClipThreads}, stream, tables[0], kGradNorm, step++, static_cast<int64_t>(need));
  for (uint32_t i = 0; out && i < launches && rc == VC_SUCCESS; ++i)
    rc = launch<clip_kernel>(dev, Shape{clip_blocks, kClipThreads, 0, 1, n}, stream, tables[i], kClip, step++, i == 0 ? 2 * bytes : 0);
  e = cudaFreeAsync(part, stream);
  if (e != cudaSuccess && rc == VC_SUCCESS) rc = cuda_fail(e, "cudaFreeAsync");
  return rc;
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
