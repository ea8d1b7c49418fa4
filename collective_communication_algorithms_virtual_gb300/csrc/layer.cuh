// What the layer operators' translation units (norm.cu, route.cu,
// exchange.cu) share: argument checks and launches on the host, element
// formats and small reductions on the device.
#pragma once

#include <atomic>
#include <cmath>
#include <cstdint>

#include "host.h"
#include "kernels.cuh"

namespace vc {
namespace layer {

// ---------------------------------------------------------------------------
// host: arguments
// ---------------------------------------------------------------------------

// Kernel index of the launch trace (vc.h).
enum Kernel : int {
  kNorm = 0, kNormBackward = 1, kNormWeight = 2, kRoute = 3, kRouteBackward = 4, kPlan = 5, kDispatch = 6,
  kCombine = 7, kCombineBackward = 8
};
constexpr int kTraceLayer = 1 << 9;

inline int dtype_size(vc_dtype_t d) {
  switch (d) {
    case VC_FLOAT32: case VC_INT32: return 4;
    case VC_BFLOAT16: case VC_FLOAT16: return 2;
    case VC_INT8: return 1;
  }
  return 0;
}

// The device buffers of one call: no null pointer, element alignment, and no
// output that overlaps another buffer of the call.
class Buffers {
 public:
  Buffers() { v_.reserve(256); }
  // One buffer of `bytes` per rank.  `in_place`: an array whose entries an
  // output may equal (the entry is then the same buffer, not an overlap).
  vc_status_t add(const void* const* a, int n, int64_t bytes, int align, bool out, const char* what,
                  const void* const* in_place = nullptr) {
    if (!a) return fail(VC_ERR_INVALID_ARG, std::string("null ") + what + " array");
    if (bytes == 0) return VC_SUCCESS;  // an empty tensor's pointer is not looked at
    for (int r = 0; r < n; ++r) {
      if (!a[r]) return fail(VC_ERR_INVALID_ARG, std::string("null ") + what + " buffer");
      const uintptr_t p = reinterpret_cast<uintptr_t>(a[r]);
      if (p % static_cast<uintptr_t>(align)) return fail(VC_ERR_INVALID_ARG, std::string(what) + " is not aligned to its element");
      all_ |= p;
      if (in_place && in_place[r] == a[r]) continue;
      v_.push_back({p, p + static_cast<uintptr_t>(bytes), out});
    }
    return VC_SUCCESS;
  }
  vc_status_t disjoint() {
    std::sort(v_.begin(), v_.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
    uintptr_t any = 0, outs = 0;  // where the buffers, the outputs so far end
    for (const Range& x : v_) {
      if (x.lo == x.hi) continue;
      if (x.lo < outs || (x.out && x.lo < any)) return fail(VC_ERR_INVALID_ARG, "an output buffer overlaps another buffer");
      any = std::max(any, x.hi);
      if (x.out) outs = std::max(outs, x.hi);
    }
    return VC_SUCCESS;
  }
  // Whether every buffer added so far starts on a 16-byte boundary.
  bool aligned16() const { return (all_ & 15) == 0; }

 private:
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  std::vector<Range> v_;
  uintptr_t all_ = 0;
};

inline vc_status_t check_ranks(int nranks) {
  if (nranks < 1 || nranks > VC_MAX_RANKS) return fail(VC_ERR_INVALID_ARG, "nranks must be in [1, 64]");
  return VC_SUCCESS;
}
inline vc_status_t check_float(vc_dtype_t d) {
  if (d == VC_FLOAT32 || d == VC_BFLOAT16 || d == VC_FLOAT16) return VC_SUCCESS;
  if (d == VC_INT32 || d == VC_INT8) return fail(VC_ERR_UNSUPPORTED, "the layer operators compute on fp32, bf16 and fp16");
  return fail(VC_ERR_INVALID_ARG, "unknown dtype");
}
// nranks * rows tokens of `width` elements: the token count fits int32, and
// nranks times all their bytes fits int64 with room to spare.
inline vc_status_t check_tokens(int nranks, size_t rows, size_t width) {
  constexpr uint64_t kMax = uint64_t(1) << 31;
  if (rows >= kMax || width >= (uint64_t(1) << 40) || rows * static_cast<uint64_t>(nranks) >= kMax)
    return fail(VC_ERR_INVALID_ARG, "too many tokens");
  const uint64_t tokens = rows * static_cast<uint64_t>(nranks);
  if (width != 0 && tokens > (uint64_t(1) << 52) / width) return fail(VC_ERR_INVALID_ARG, "tokens times width too large");
  return VC_SUCCESS;
}

// ---------------------------------------------------------------------------
// host: launches
// ---------------------------------------------------------------------------

// Blocks of kernel K (with `threads` threads and `smem` dynamic bytes)
// resident per SM; queried once per device and shape.
template <auto K>
int resident_blocks(int dev, int threads, size_t smem) {
  static std::atomic<uint64_t> cache[64];  // threads << 40 | smem << 8 | blocks
  const uint64_t key = (static_cast<uint64_t>(threads) << 40) | (static_cast<uint64_t>(smem) << 8);
  const uint64_t seen = cache[dev].load(std::memory_order_relaxed);
  if (seen != 0 && (seen & ~uint64_t(255)) == key) return static_cast<int>(seen & 255);
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, K, threads, smem) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 1;
  }
  cache[dev].store(key | static_cast<uint64_t>(n), std::memory_order_relaxed);
  return n;
}

// Lets kernel K take `smem` dynamic bytes and, where asked, a cluster above
// the portable 8 blocks; once per device and size reached.
template <auto K>
vc_status_t allow(int dev, size_t smem, bool big_cluster) {
  static std::atomic<size_t> most[64];
  static std::atomic<bool> wide[64];
  if (smem > (48u << 10) && smem > most[dev].load(std::memory_order_relaxed)) {
    cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    most[dev].store(smem, std::memory_order_relaxed);
  }
  if (big_cluster && !wide[dev].load(std::memory_order_relaxed)) {
    cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    wide[dev].store(true, std::memory_order_relaxed);
  }
  return VC_SUCCESS;
}

struct Shape {
  unsigned grid, block;
  size_t smem = 0;
  unsigned cluster = 1;
};

// One launch of kernel K with its parameter block; `what`, `step` and `bytes`
// for the trace.
template <auto K, class P>
vc_status_t launch(int dev, const Shape& s, cudaStream_t stream, const P& p, Kernel what, int step, int64_t bytes) {
  vc_status_t rc = allow<K>(dev, s.smem, s.cluster > 8);
  if (rc != VC_SUCCESS) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.grid);
  cfg.blockDim = dim3(s.block);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  if (pdl_enabled()) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (s.cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs++].val.clusterDim = {s.cluster, 1, 1};
  }
  struct Arg {
    cudaLaunchConfig_t* cfg;
    const P* p;
  } arg{&cfg, &p};
  vc_trace_record_t rec{};
  rec.coll = rec.algo = -1;
  rec.step = step;
  rec.kernel = kTraceLayer | what;
  rec.bytes = bytes;
  rec.nops = 1;
  return launch_traced(
      stream, rec,
      [](void* a) {
        Arg* x = static_cast<Arg*>(a);
        return cudaLaunchKernelEx(x->cfg, K, *x->p);
      },
      &arg);
}

// Runs f with the dtype's code as a compile-time constant.
template <class F>
vc_status_t for_dtype(vc_dtype_t d, F&& f) {
  switch (d) {
    case VC_FLOAT32: return f(std::integral_constant<int, VC_FLOAT32>{});
    case VC_BFLOAT16: return f(std::integral_constant<int, VC_BFLOAT16>{});
    default: return f(std::integral_constant<int, VC_FLOAT16>{});
  }
}

// ---------------------------------------------------------------------------
// device
// ---------------------------------------------------------------------------

// A kernel may start before its predecessor in the stream has ended; it
// touches memory only after the wait.  The next grid is let in right after
// (its blocks take only room that this grid leaves), and waits likewise.
__device__ __forceinline__ void stream_order() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Element formats: 16-byte vectors and single elements to and from fp32.
template <int DT>
struct El {
  static constexpr int kSize = DT == VC_FLOAT32 ? 4 : 2;
  static constexpr int kVec = 16 / kSize;  // elements of a 16-byte vector
  static constexpr bool kF16 = DT == VC_FLOAT16;

  static __device__ __forceinline__ void widen(uint4 v, float* f) {
    if constexpr (DT == VC_FLOAT32) {
      f[0] = __uint_as_float(v.x);
      f[1] = __uint_as_float(v.y);
      f[2] = __uint_as_float(v.z);
      f[3] = __uint_as_float(v.w);
    } else {
      dev::widen8<kF16>(v, f);
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float* f) {
    if constexpr (DT == VC_FLOAT32)
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else
      return make_uint4(dev::pack2<kF16>(f[0], f[1]), dev::pack2<kF16>(f[2], f[3]), dev::pack2<kF16>(f[4], f[5]),
                        dev::pack2<kF16>(f[6], f[7]));
  }
  static __device__ __forceinline__ float load(const void* p, int64_t i) {
    if constexpr (DT == VC_FLOAT32) return static_cast<const float*>(p)[i];
    else return dev::widen1<kF16>(static_cast<const uint16_t*>(p)[i]);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, float x) {
    if constexpr (DT == VC_FLOAT32) static_cast<float*>(p)[i] = x;
    else static_cast<uint16_t*>(p)[i] = dev::narrow1<kF16>(x);
  }
};

__device__ __forceinline__ uint4 ld16_plain(const void* p) { return *static_cast<const uint4*>(p); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// Sum over the block, the same in every thread.  `part` is 32 floats of
// shared memory that no thread reads or writes between this call and the
// barrier of the one after the next (callers alternate two).
__device__ __forceinline__ float block_sum(float x, float* part) {
  x = warp_sum(x);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  const int l = threadIdx.x & 31;
  return warp_sum(l < warps ? part[l] : 0.f);
}
// Largest over the block of values that compare as their bits do (>= 0, NaN
// above infinity).
__device__ __forceinline__ uint32_t block_max_bits(uint32_t x, uint32_t* part) {
  x = __reduce_max_sync(0xffffffffu, x);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  const int l = threadIdx.x & 31;
  return __reduce_max_sync(0xffffffffu, l < warps ? part[l] : 0u);
}

}  // namespace layer
}  // namespace vc
