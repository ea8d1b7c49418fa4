// Rounding to 8-bit floating point (e4m3) with a scale for each block of a row's
// 128 elements, or of 128 rows by 128 (see vc.h).
//
// Memory bounds it: every element is read once, held in registers while its
// block's largest magnitude is found, and written once.  On a GB300 (copy rate
// 6.78 TB/s): 32768 rows of 4096 bf16, 66 us, 6.2 TB/s; 64 matrices of 2048 by
// 4096 by tiles, 257 us, 6.3 TB/s; one to eight rows are a launch, 1.7 us.
#include <cuda_fp8.h>

#include "layer.cuh"

namespace vc {
namespace layer {
namespace {

constexpr int kBlock = VC_FP8_BLOCK;
constexpr float kMost8 = 448.f;          // the largest e4m3 number
constexpr float kLeastScale = 0x1p-126f;  // the smallest normal number
constexpr int kThreads8 = 256, kWarps8 = kThreads8 / 32;

struct QuantizeParams {
  const void* x[VC_MAX_RANKS];
  void* out[VC_MAX_RANKS];
  float* scale[VC_MAX_RANKS];
  const int32_t* count[VC_MAX_RANKS];
  int64_t rows;    // of each rank (by rows), of each matrix (by tiles)
  int64_t width;
  int64_t blocks;  // of a row
  int64_t down;    // tiles of a matrix, one below another
  int64_t matrices;
  uint32_t pieces;  // of a row
  bool counted;
};

// A block's scale, and what its elements are multiplied by.  `bits`: its
// largest magnitude's (a NaN's are above infinity's).
struct Scale {
  float scale, by;  // by: NaN for a block with a NaN or an infinity
  __device__ __forceinline__ explicit Scale(uint32_t bits) {
    const float most = __uint_as_float(bits);
    const bool fine = bits < 0x7f800000u;
    scale = !fine ? most : bits == 0 ? 0.f : fmaxf(__fdiv_rn(most, kMost8), kLeastScale);
    by = fine ? fminf(__fdiv_rn(kMost8, most), 1.f / kLeastScale) : __uint_as_float(0x7fffffffu);
  }
};
// Four elements, rounded once each to the nearest e4m3 number (ties to even);
// zeros where `by` is NaN.
__device__ __forceinline__ uint32_t round4(const float* f, float by) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0] * by, f[1] * by), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2] * by, f[3] * by), __NV_SATFINITE, __NV_E4M3);
  return by == by ? lo | hi << 16 : 0u;
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// The largest magnitude of a 16-byte unit, as the type's own bits (the two
// halves of a word each have one for 16-bit types: their order is their bits').
template <int DT>
__device__ __forceinline__ uint32_t largest_of(uint4 v) {
  if constexpr (DT == VC_FLOAT32) {
    constexpr uint32_t m = 0x7fffffffu;
    return max(max(v.x & m, v.y & m), max(v.z & m, v.w & m));
  } else {
    constexpr uint32_t m = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  }
}
template <int DT>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  if constexpr (DT == VC_FLOAT32) return max(a, b);
  else return __vmaxu2(a, b);
}
// As fp32 bits.
template <int DT>
__device__ __forceinline__ uint32_t magnitude_of(uint32_t x) {
  if constexpr (DT == VC_FLOAT32) return x;
  else return __float_as_uint(dev::widen1<DT == VC_FLOAT16>(static_cast<uint16_t>(max(x & 0xffffu, x >> 16))));
}

// -- a scale for each row's 128 ---------------------------------------------------
// A warp works four spans of 32 units (16 bytes) of one row, all loaded first;
// 128 elements are 16 lanes (fp32: 32) of one span.  Of those lanes, lane i
// divides for span i: with every lane dividing for its own span the kernel is
// bound by its instructions (80 us for 268 MB of rows, where memory takes 60).
constexpr int kSpans = 4;

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads8, 4) quantize_rows_kernel(const __grid_constant__ QuantizeParams p) {
  using E = El<DT>;
  constexpr int kLanes = kBlock / E::kVec;
  __shared__ __align__(16) unsigned char room[kWarps8][Span<1, E::kVec, VEC>::kRoom];
  stream_order();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, d = blockIdx.y;
  const int64_t rows = p.counted ? min(max(static_cast<int64_t>(__ldg(p.count[d])), int64_t(0)), p.rows) : p.rows;
  const char* x = static_cast<const char*>(p.x[d]);
  const Bytes ends{x, x + p.rows * p.width * E::kSize};
  const int units = static_cast<int>((p.width + E::kVec - 1) / E::kVec);
  // rows and pieces of a rank: neither they nor the rows' warps pass 32 bits
  const uint32_t warps = gridDim.x * kWarps8;
  uint32_t r = (blockIdx.x * kWarps8 + warp) / p.pieces, piece = (blockIdx.x * kWarps8 + warp) % p.pieces;
  const uint32_t step_r = warps / p.pieces, step_piece = warps % p.pieces;
  while (r < rows) {
    const int c0 = static_cast<int>(piece) * (kSpans * 32);
    const Row<E::kSize, VEC> row(x + r * p.width * E::kSize, units, ends);
    typename Row<E::kSize, VEC>::Raw raw[kSpans];
#pragma unroll
    for (int s = 0; s < kSpans; ++s) {
      const int c = c0 + s * 32 + lane;
      raw[s] = c < units ? row.load(c) : row.zero();
    }
    uint4 unit[kSpans];
    uint32_t mine = 0;
#pragma unroll
    for (int s = 0; s < kSpans; ++s) {
      const int c = c0 + s * 32 + lane;
      unit[s] = make_uint4(0, 0, 0, 0);
      if constexpr (VEC) {
        unit[s] = raw[s];
      } else if (c < units) {
        float f[E::kVec];
        E::widen(row.finish(raw[s], c, p.width), f);
        mask_unit<E::kSize, VEC>(c, p.width, f);
        unit[s] = E::narrow(f);  // exact
      }
      uint32_t most = largest_of<DT>(unit[s]);
#pragma unroll
      for (int k = kLanes / 2; k > 0; k >>= 1) most = larger<DT>(most, __shfl_xor_sync(0xffffffffu, most, k));
      if (lane % kSpans == s) mine = most;
    }
    const Scale own(magnitude_of<DT>(mine));
    const int first = lane & ~(kLanes - 1), block = c0 / kLanes + (lane % kSpans) * (32 / kLanes) + first / kLanes;
    if (lane - first < kSpans && block < p.blocks) p.scale[d][r * p.blocks + block] = own.scale;
    char* out = static_cast<char*>(p.out[d]) + r * p.width;
#pragma unroll
    for (int s = 0; s < kSpans; ++s) {
      if (c0 + s * 32 >= units) break;
      const float by = __shfl_sync(0xffffffffu, own.by, first + s);
      float f[E::kVec];
      E::widen(unit[s], f);
      if constexpr (E::kVec == 8)
        Span<1, 8, VEC>(room[warp], make_uint2(round4(f, by), round4(f + 4, by))).write(out, c0 + s * 32, p.width);
      else
        Span<1, 4, VEC>(room[warp], round4(f, by)).write(out, c0 + s * 32, p.width);
    }
    r += step_r;
    if ((piece += step_piece) >= p.pieces) piece -= p.pieces, ++r;
  }
}

// -- a scale for each 128 rows by 128 ---------------------------------------------
// A block of threads holds a tile in registers.  VEC: a row's 128 elements are
// 16 lanes (fp32: 32); otherwise a thread takes one column, element by element.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads8, 2) quantize_tiles_kernel(const __grid_constant__ QuantizeParams p) {
  using E = El<DT>;
  __shared__ uint32_t part[2][32];
  stream_order();
  const int d = blockIdx.y;
  const int64_t total = p.matrices * p.down * p.blocks;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x, turn ^= 1) {
    const int64_t across = t % p.blocks, below = t / p.blocks % p.down, matrix = t / p.blocks / p.down;
    const int64_t first = matrix * p.rows + below * kBlock, col0 = across * kBlock;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kBlock), p.rows - below * kBlock));
    const int cols = static_cast<int>(min(static_cast<int64_t>(kBlock), p.width - col0));
    uint32_t most = 0;
    if constexpr (VEC) {
      constexpr int kLanes = kBlock / E::kVec, kPass = kThreads8 / kLanes, kHeld = kBlock / kPass;
      const int u = threadIdx.x % kLanes * E::kVec, r0 = threadIdx.x / kLanes;
      const char* x = static_cast<const char*>(p.x[d]) + ((first + r0) * p.width + col0 + u) * E::kSize;
      uint4 held[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        held[i] = r0 + i * kPass < rows && u < cols ? dev::ld16(x + i * kPass * p.width * E::kSize) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) most = larger<DT>(most, largest_of<DT>(held[i]));
      const Scale by(block_max_bits(magnitude_of<DT>(most), part[turn]));
      if (threadIdx.x == 0) p.scale[d][t] = by.scale;
      char* out = static_cast<char*>(p.out[d]) + (first + r0) * p.width + col0 + u;
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (r0 + i * kPass < rows && u < cols) {
          float f[E::kVec];
          E::widen(held[i], f);
          if constexpr (E::kVec == 8) *reinterpret_cast<uint2*>(out + i * kPass * p.width) = make_uint2(round4(f, by.by), round4(f + 4, by.by));
          else *reinterpret_cast<uint32_t*>(out + i * kPass * p.width) = round4(f, by.by);
        }
    } else {
      constexpr int kPass = kThreads8 / kBlock, kHeld = kBlock / kPass;
      const int c = threadIdx.x % kBlock, r0 = threadIdx.x / kBlock;
      const int64_t at = (first + r0) * p.width + col0 + c;
      float f[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        f[i] = r0 + i * kPass < rows && c < cols ? E::load(p.x[d], at + i * kPass * p.width) : 0.f;
        most = max(most, magnitude(f[i]));
      }
      const Scale by(block_max_bits(most, part[turn]));
      if (threadIdx.x == 0) p.scale[d][t] = by.scale;
      uint8_t* out = static_cast<uint8_t*>(p.out[d]) + at;
#pragma unroll
      for (int i = 0; i < kHeld; i += 4) {
        const uint32_t q = round4(f + i, by.by);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r0 + (i + k) * kPass < rows && c < cols) out[(i + k) * kPass * p.width] = static_cast<uint8_t>(q >> (8 * k));
      }
    }
  }
}

vc_status_t quantize(const void* const* x, void* const* out, float* const* scale, const int32_t* const* count, int nranks,
                     size_t matrices, size_t rows, size_t width, int block_rows, vc_dtype_t dtype, cudaStream_t stream) {
  vc_status_t rc = check_ranks(nranks);
  if (rc == VC_SUCCESS) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  if (block_rows != 1 && block_rows != kBlock) return fail(VC_ERR_UNSUPPORTED, "block_rows is 1 or VC_FP8_BLOCK");
  if (count && (matrices != 1 || block_rows != 1)) return fail(VC_ERR_INVALID_ARG, "a count of rows wants one matrix and block_rows 1");
  if (matrices >= (uint64_t(1) << 31) || rows >= (uint64_t(1) << 31)) return fail(VC_ERR_INVALID_ARG, "too many rows");
  if (width > VC_EXPERT_MAX_WIDTH) return fail(VC_ERR_UNSUPPORTED, "width above VC_EXPERT_MAX_WIDTH");
  rc = check_tokens(nranks, matrices * rows, width);
  if (rc != VC_SUCCESS) return rc;
  const int es = dtype_size(dtype);
  const int64_t n = static_cast<int64_t>(matrices * rows), w = static_cast<int64_t>(width), blocks = (w + kBlock - 1) / kBlock;
  const int64_t down = block_rows == 1 ? static_cast<int64_t>(rows) : (static_cast<int64_t>(rows) + kBlock - 1) / kBlock;
  const int64_t scales = static_cast<int64_t>(matrices) * down * blocks;
  Buffers b;
  rc = b.add(x, nranks, n * w * es, es, false, "x");
  const bool whole = b.aligned16();
  if (rc == VC_SUCCESS) rc = b.add(out, nranks, n * w, 1, true, "out");
  uintptr_t outs = 0;
  for (int r = 0; rc == VC_SUCCESS && n * w != 0 && r < nranks; ++r) outs |= reinterpret_cast<uintptr_t>(out[r]);
  if (rc == VC_SUCCESS) rc = b.add(reinterpret_cast<const void* const*>(scale), nranks, scales * 4, 4, true, "scale");
  if (rc == VC_SUCCESS && count) rc = b.add(reinterpret_cast<const void* const*>(count), nranks, 4, 4, false, "count");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || n == 0 || w == 0) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  QuantizeParams p = {};
  for (int r = 0; r < nranks; ++r) {
    p.x[r] = x[r];
    p.out[r] = out[r];
    p.scale[r] = scale[r];
    if (count) p.count[r] = count[r];
  }
  p.counted = count != nullptr;
  p.width = w;
  p.blocks = blocks;
  p.matrices = static_cast<int64_t>(matrices);
  p.down = down;
  p.rows = block_rows == 1 ? n : static_cast<int64_t>(rows);
  const int64_t bytes = nranks * (n * w * (es + 1) + scales * 4);
  return for_dtype(dtype, [&](auto code) {
    constexpr int DT = code();
    constexpr int kVec = El<DT>::kVec;
    const auto go = [&](auto vec) {
      constexpr bool VEC = vec();
      if (block_rows == 1) {
        constexpr auto K = quantize_rows_kernel<DT, VEC>;
        p.pieces = static_cast<uint32_t>((units_of(w, es) + kSpans * 32 - 1) / (kSpans * 32));
        const int64_t fit = (int64_t(st->nsm) * resident_blocks<K>(dev, kThreads8, 0) + nranks - 1) / nranks;
        const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((n * p.pieces + kWarps8 - 1) / kWarps8, fit));
        return launch<K>(dev, Shape{blocks, kThreads8, 0, 1, static_cast<unsigned>(nranks)}, stream, p, kQuantize, 0, bytes);
      }
      constexpr auto K = quantize_tiles_kernel<DT, VEC>;
      const int64_t fit = (int64_t(st->nsm) * resident_blocks<K>(dev, kThreads8, 0) + nranks - 1) / nranks;
      const unsigned grid = static_cast<unsigned>(std::min<int64_t>(scales, fit));
      return launch<K>(dev, Shape{grid, kThreads8, 0, 1, static_cast<unsigned>(nranks)}, stream, p, kQuantize, 0, bytes);
    };
    return whole && w % kVec == 0 && outs % kVec == 0 ? go(std::true_type{}) : go(std::false_type{});
  });
}

}  // namespace
}  // namespace layer
}  // namespace vc

using namespace vc;

VC_EXPORT vc_status_t vc_quantize_fp8(const void* const* x, void* const* out, float* const* scale,
                                      const int32_t* const* count, int nranks, size_t matrices, size_t rows,
                                      size_t width, int block_rows, vc_dtype_t dtype, vc_stream_t stream) {
  return entry([&] {
    return layer::quantize(x, out, scale, count, nranks, matrices, rows, width, block_rows, dtype,
                           reinterpret_cast<cudaStream_t>(stream));
  });
}
