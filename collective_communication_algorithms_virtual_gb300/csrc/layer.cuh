// What the layer operators' translation units (norm.cu, route.cu,
// exchange.cu, expert.cu, quantize.cu, clip.cu) share: argument checks and launches on the host, element
// formats and small reductions on the device.
#pragma once

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <type_traits>

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
  kCombine = 7, kCombineBackward = 8, kExpertProduct = 9, kExpertWeight = 10, kExpertProduct8 = 11, kQuantize = 12,
  kGradNorm = 13, kClip = 14, kPad = 15
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
  // One buffer of `bytes` per rank.  `in_place`: an array whose entries an
  // output may equal (the entry is then the same buffer, not an overlap).
  vc_status_t add(const void* const* a, int n, int64_t bytes, int align, bool out, const char* what,
                  const void* const* in_place = nullptr) {
    if (!a) return fail(VC_ERR_INVALID_ARG, std::string("null ") + what + " array");
    if (bytes == 0) return VC_SUCCESS;  // an empty tensor's pointer is not looked at
    Span s{UINTPTR_MAX, 0, count_, count_, out, true};
    for (int r = 0; r < n; ++r) {
      const uintptr_t p = reinterpret_cast<uintptr_t>(a[r]);
      if (!p) return fail(VC_ERR_INVALID_ARG, std::string("null ") + what + " buffer");
      if (p % static_cast<uintptr_t>(align)) return fail(VC_ERR_INVALID_ARG, std::string(what) + " is not aligned to its element");
      all_ |= p;
      if (in_place && in_place[r] == a[r]) continue;
      const Range x{p, p + static_cast<uintptr_t>(bytes), out};
      s.apart = s.apart && x.lo >= s.hi;
      s.lo = std::min(s.lo, x.lo);
      s.hi = std::max(s.hi, x.hi);
      range_[count_++] = x;
    }
    s.end = count_;
    if (s.end > s.begin) span_[spans_++] = s;
    return VC_SUCCESS;
  }
  vc_status_t disjoint() {
    // as a rule each argument's buffers ascend and no two arguments' interleave
    bool plain = true;
    for (int i = 0; i < spans_ && plain; ++i) {
      plain = span_[i].apart || !span_[i].out;
      for (int j = 0; j < i && plain; ++j)
        plain = !(span_[i].out || span_[j].out) || span_[i].lo >= span_[j].hi || span_[j].lo >= span_[i].hi;
    }
    if (plain) return VC_SUCCESS;
    std::sort(range_, range_ + count_, [](const Range& x, const Range& y) { return x.lo < y.lo; });
    uintptr_t any = 0, outs = 0;  // where the buffers, the outputs so far end
    for (int i = 0; i < count_; ++i) {
      const Range& x = range_[i];
      if (x.lo < outs || (x.out && x.lo < any)) return fail(VC_ERR_INVALID_ARG, "an output buffer overlaps another buffer");
      any = std::max(any, x.hi);
      if (x.out) outs = std::max(outs, x.hi);
    }
    return VC_SUCCESS;
  }
  // Whether every buffer added so far starts on a 16-byte boundary.
  bool aligned16() const { return (all_ & 15) == 0; }

 private:
  static constexpr int kMost = 8;  // arguments of a call
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  struct Span {  // one argument's buffers
    uintptr_t lo, hi;
    int begin, end;
    bool out, apart;  // apart: ascending, none into the next
  };
  Range range_[kMost * VC_MAX_RANKS];
  Span span_[kMost];
  int count_ = 0, spans_ = 0;
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

// Lets kernel K take all the dynamic shared memory that a block can have,
// where a call wants more than 32 KB (with its static bytes that may pass the
// 48 KB that need no leave), and, where asked, a cluster above the portable 8
// blocks; once per device.  Every thread sets the same values, so first calls
// that race agree whatever sizes they are for.
template <auto K>
vc_status_t allow(int dev, size_t smem, bool big_cluster) {
  static std::atomic<bool> raised[64], wide[64];
  if (smem > (32u << 10) && !raised[dev].load(std::memory_order_acquire)) {
    int block = 0;
    cudaFuncAttributes own;
    cudaError_t e = cudaDeviceGetAttribute(&block, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&own, K);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, block - static_cast<int>(own.sharedSizeBytes));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    raised[dev].store(true, std::memory_order_release);
  }
  if (big_cluster && !wide[dev].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    wide[dev].store(true, std::memory_order_release);
  }
  return VC_SUCCESS;
}

// Blocks of kernel K (with `threads` threads and `smem` dynamic bytes)
// resident per SM; queried once per device and shape.
template <auto K>
int resident_blocks(int dev, int threads, size_t smem) {
  static std::atomic<uint64_t> cache[64];  // threads << 40 | smem << 8 | blocks
  const uint64_t key = (static_cast<uint64_t>(threads) << 40) | (static_cast<uint64_t>(smem) << 8);
  const uint64_t seen = cache[dev].load(std::memory_order_relaxed);
  if (seen != 0 && (seen & ~uint64_t(255)) == key) return static_cast<int>(seen & 255);
  int n = 0;
  if (allow<K>(dev, smem, false) != VC_SUCCESS) return 1;  // the launch will say why
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, K, threads, smem) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 1;
  }
  cache[dev].store(key | static_cast<uint64_t>(n), std::memory_order_relaxed);
  return n;
}

struct Shape {
  unsigned grid, block;
  size_t smem = 0;
  unsigned cluster = 1;
  unsigned ranks = 1;  // the grid's second dimension, where blocks belong to ranks
  bool early = true;   // its blocks may come in before the launch ahead has ended (stream_order)
};

// One launch of kernel K with its parameter block; `what`, `step` and `bytes`
// for the trace.
template <auto K, class P>
vc_status_t launch(int dev, const Shape& s, cudaStream_t stream, const P& p, Kernel what, int step, int64_t bytes) {
  vc_status_t rc = allow<K>(dev, s.smem, s.cluster > 8);
  if (rc != VC_SUCCESS) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.grid, s.ranks);
  cfg.blockDim = dim3(s.block);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  if (s.early && pdl_enabled()) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (s.cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs++].val.clusterDim = {s.cluster, 1, 1};
  }
  if (log_enabled())
    std::fprintf(stderr, "[vc] layer kernel=%d grid=%ux%u block=%u cluster=%u smem=%zu bytes=%lld\n", static_cast<int>(what), s.grid,
                 s.ranks, s.block, s.cluster, s.smem, static_cast<long long>(bytes));
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

// -- rows ----------------------------------------------------------------------
// A row is worked in units of 16 bytes, a warp on 32 neighbouring ones.  VEC:
// every row starts on a 16-byte boundary and is whole units.  Otherwise rows
// lie at any element: a unit is cut out of two aligned loads, and a warp's
// units go through shared memory, where aligned stores are cut out of them
// (only the bytes before the first boundary and after the last one are stored
// by element).  A last unit that the row does not fill ends in elements that
// are not the row's: whoever sums over it masks them.  No access passes the
// ends of a buffer.  A load may bring bytes of the neighbouring rows along,
// which are dropped (in an in-place call another block may be writing them);
// a store never touches them.  (A combine of 4096 tokens, 8 choices and 4099 bf16: 166
// us with an access per element, 94 us so, against 48 us for 4096 elements; an
// 8-rank norm of 2048 x 8191: 107 us, against 54 us for 8192.)
//
// Units are loaded raw and finished when they are used, so that a thread's
// loads are all in flight before the first is waited for.
struct Bytes {  // a buffer, for its ends
  const char* lo;
  const char* hi;
};

// 16 bytes from byte m (0 .. 15) of two neighbouring vectors.
__device__ __forceinline__ uint4 cut(uint4 x, uint4 y, uint32_t m) {
  const bool two = m & 8, one = m & 4;
  const uint32_t a0 = two ? x.z : x.x, a1 = two ? x.w : x.y, a2 = two ? y.x : x.z, a3 = two ? y.y : x.w,
                 a4 = two ? y.z : y.x, a5 = two ? y.w : y.y;
  const uint32_t b0 = one ? a1 : a0, b1 = one ? a2 : a1, b2 = one ? a3 : a2, b3 = one ? a4 : a3, b4 = one ? a5 : a4;
  const uint32_t s = (m & 3) * 8;
  return make_uint4(__funnelshift_r(b0, b1, s), __funnelshift_r(b1, b2, s), __funnelshift_r(b2, b3, s),
                    __funnelshift_r(b3, b4, s));
}

// The 16 / ES elements at `at`, of which the first `n` are the row's, by
// element (the others 0).  Kept out of line: few get here.
template <int ES>
__device__ __noinline__ uint4 load_elements(const char* at, int64_t n) {
  uint32_t out[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16 / ES; ++i)
    if (i < n) {
      uint32_t e;
      if constexpr (ES == 4) e = *reinterpret_cast<const uint32_t*>(at + i * 4);
      else if constexpr (ES == 2) e = *reinterpret_cast<const uint16_t*>(at + i * 2);
      else e = static_cast<uint8_t>(at[i]);
      out[i * ES / 4] |= e << (i * ES % 4 * 8);
    }
  return make_uint4(out[0], out[1], out[2], out[3]);
}
struct Two {
  uint4 x, y;
};

// A row of n elements of ES bytes that is read, by units.
template <int ES, bool VEC>
struct Row {
  static constexpr int kN = 16 / ES;
  using Raw = std::conditional_t<VEC, uint4, Two>;
  const char* base;  // unit 0, or the boundary before it
  uint32_t m;        // bytes from there to unit 0
  int lo, hi;        // the units whose vectors are all the buffer's

  // A row of `units` units.
  __device__ __forceinline__ Row(const void* row, int units, Bytes in) {
    base = static_cast<const char*>(row);
    if constexpr (!VEC) {
      m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(base)) & 15;
      base -= m;
      lo = 0;
      hi = units;
      if (base < in.lo || base + (static_cast<int64_t>(units) + 1) * 16 > in.hi) {  // the buffer's first or last row
        lo = base < in.lo;
        hi = min(static_cast<int64_t>(units), (in.hi - base) / 16 - (m != 0));
      }
    }
  }
  static __device__ __forceinline__ Raw zero() { return Raw{}; }
  // Data that nothing writes during the kernel.
  __device__ __forceinline__ Raw load(int c) const {
    if constexpr (VEC) return dev::ld16(base + static_cast<int64_t>(c) * 16);
    else return two<false>(c);
  }
  // What every block reads: kept in L1.
  __device__ __forceinline__ Raw load_kept(int c) const {
    if constexpr (VEC) return __ldg(reinterpret_cast<const uint4*>(base) + c);
    else return two<false>(c);
  }
  // What this thread may overwrite later.
  __device__ __forceinline__ Raw load_plain(int c) const {
    if constexpr (VEC) return reinterpret_cast<const uint4*>(base)[c];
    else return two<true>(c);
  }
  // Unit c of the row, whose vectors were loaded.
  __device__ __forceinline__ uint4 finish(const Raw& v, int c, int64_t n) const {
    if constexpr (VEC) {
      return v;
    } else {
      if (c >= lo && c < hi) return m ? cut(v.x, v.y, m) : v.x;
      return load_elements<ES>(base + m + static_cast<int64_t>(c) * 16, n - static_cast<int64_t>(c) * kN);
    }
  }

 private:
  template <bool PLAIN>
  __device__ __forceinline__ Two two(int c) const {
    const uint4* w = reinterpret_cast<const uint4*>(base) + c;
    Two v{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    const bool in = c >= lo && c < hi;
    if (in) v.x = PLAIN ? w[0] : __ldg(w);
    if (in && m) v.y = PLAIN ? w[1] : __ldg(w + 1);
    return v;
  }
};

// 0 for the elements of unit c that a row of n does not have.
template <int ES, bool VEC>
__device__ __forceinline__ void mask_unit(int c, int64_t n, float* f) {
  if constexpr (!VEC) {
    const int64_t left = n - static_cast<int64_t>(c) * (16 / ES);
    if (left < 16 / ES) {
#pragma unroll
      for (int i = 0; i < 16 / ES; ++i)
        if (i >= left) f[i] = 0.f;
    }
  }
}

// What a warp writes of a row: B bytes of each lane, one behind another, of
// ES-byte elements.  Without VEC all lanes call both functions together.
template <int ES, int B, bool VEC>
struct Span {
  using V = std::conditional_t<B == 16, uint4, std::conditional_t<B == 8, uint2, uint32_t>>;
  static constexpr int kRoom = VEC ? 16 : 32 * B + 16;  // shared memory of a warp
  unsigned char* sm;
  V v;

  // Lane's bytes (any, past the row's end), which go to the same place of one
  // row or several.
  __device__ __forceinline__ Span(unsigned char* room, V value) : sm(room), v(value) {
    if constexpr (!VEC) {
      __syncwarp();  // the last span has been read
      reinterpret_cast<V*>(sm)[threadIdx.x & 31] = v;
      __syncwarp();
    }
  }
  // To a row of `n` elements, lane 0's bytes being the row's unit c0.  STREAM:
  // results that nothing here reads again.
  template <bool STREAM = false>
  __device__ __forceinline__ void write(void* row, int c0, int64_t n) const {
    const int lane = threadIdx.x & 31;
    if constexpr (VEC) {
      const int64_t c = static_cast<int64_t>(c0) + lane;
      if (c * B >= n * ES) return;
      if constexpr (STREAM && B == 16) dev::st16(static_cast<V*>(row) + c, v);
      else static_cast<V*>(row)[c] = v;
    } else {
      const int64_t left = n * ES - static_cast<int64_t>(c0) * B;
      if (left <= 0) return;
      const int bytes = left < 32 * B ? static_cast<int>(left) : 32 * B;
      char* a = static_cast<char*>(row) + static_cast<int64_t>(c0) * B;
      const int head = min(bytes, static_cast<int>(-reinterpret_cast<uintptr_t>(a) & 15));
      const int words = (bytes - head) >> 4, tail = head + words * 16;
      if (lane < words) {
        const uint4* w = reinterpret_cast<const uint4*>(sm) + lane;
        *reinterpret_cast<uint4*>(a + head + lane * 16) = head ? cut(w[0], w[1], head) : w[0];
      }
      // lanes 0 .. 15: the elements before the first boundary; 16 .. 31: those after the last
      const int at = lane < 16 ? lane * ES : tail + (lane - 16) * ES;
      if (at < (lane < 16 ? head : bytes)) {
        if constexpr (ES == 4) *reinterpret_cast<uint32_t*>(a + at) = *reinterpret_cast<const uint32_t*>(sm + at);
        else if constexpr (ES == 2) *reinterpret_cast<uint16_t*>(a + at) = *reinterpret_cast<const uint16_t*>(sm + at);
        else a[at] = static_cast<char>(sm[at]);
      }
    }
  }
};
// Units of a row of n elements of ES bytes.
inline int64_t units_of(int64_t n, int es) { return (n * es + 15) / 16; }

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
