// The products of an expert-parallel layer: the rows that each rank's experts
// have received with the experts' weights, and their gradients (see vc.h).
//
// How many rows an expert has is known on the device alone, so every kernel
// here makes its list of tiles from the offsets and walks it with as many
// blocks as the GPU holds.
#include "tc.cuh"

namespace vc {
namespace layer {
namespace {

using tc::Rows;

constexpr int kMaxExperts = VC_ROUTE_MAX_EXPERTS;

// ---------------------------------------------------------------------------
// products in fp32
// ---------------------------------------------------------------------------
// out(n, m) = sum over k of b(n, k) * a(m, k) in tiles of 64 n by 128 m, 16 of
// k at a time; 256 threads with 4 n by 8 m each.
//   rows' products: n is a row of the expert, m of its outputs, a its weights.
//   weights' gradients: k is a row, n and m run over the weights.
constexpr int kSimpleM = 128, kSimpleN = 64, kSimpleK = 16, kSimpleThreads = 256;

struct SimpleParams {
  const void* a[VC_MAX_RANKS];
  const void* b[VC_MAX_RANKS];
  void* out[VC_MAX_RANKS];
  const int32_t* offsets[VC_MAX_RANKS];
  int64_t am, ak, ae, bn, bk;  // elements between neighbours in m, k; of experts; in n, k
  int32_t capacity;
  int M, N, K;  // N: of weights' gradients; K: of rows' products
  int experts, each;
};

// One operand's 16 by W tile of k by m (or n) to shared memory, in fp32.
// Neighbouring threads take neighbouring elements in memory.
template <int DT, int W>
struct SimpleTile {
  static constexpr int kEach = kSimpleK * W / kSimpleThreads;
  float v[kEach];
  static __device__ __forceinline__ void place(int i, bool k_runs, int* k, int* w) {
    const int at = i * kSimpleThreads + threadIdx.x;
    *k = k_runs ? at % kSimpleK : at / W;
    *w = k_runs ? at / kSimpleK : at % W;
  }
  __device__ __forceinline__ void load(const void* p, int64_t sw, int64_t sk, int ws, int ks) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      int k, w;
      place(i, sk == 1, &k, &w);
      v[i] = w < ws && k < ks ? El<DT>::load(p, w * sw + k * sk) : 0.f;
    }
  }
  __device__ __forceinline__ void store(float (*to)[W + 4], bool k_runs) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      int k, w;
      place(i, k_runs, &k, &w);
      to[k][w] = v[i];
    }
  }
};

template <int DT, int OUT, bool WEIGHT>
__global__ void __launch_bounds__(kSimpleThreads, 2) product_simple_kernel(const __grid_constant__ SimpleParams p) {
  __shared__ uint32_t ends[kMaxExperts];
  __shared__ int longest;
  __shared__ __align__(16) float sa[2][kSimpleK][kSimpleM + 4], sb[2][kSimpleK][kSimpleN + 4];
  stream_order();
  const uint32_t across = (p.M + kSimpleM - 1) / kSimpleM, down = (p.N + kSimpleN - 1) / kSimpleN;
  uint32_t total = p.experts * across * down;
  if constexpr (!WEIGHT) {
    if (threadIdx.x < 32) tc::list_tiles(p.offsets, p.experts, p.each, p.capacity, kSimpleN, across, ends, &longest);
    __syncthreads();
    total = ends[p.experts - 1];
  }
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  int e = 0;
  for (uint32_t t = blockIdx.x; t < total; t += gridDim.x) {
    uint32_t at = t;
    if constexpr (WEIGHT) {
      e = t / (across * down);
      at -= e * (across * down);
    } else {
      while (ends[e] <= t) ++e;
      if (e) at -= ends[e - 1];
    }
    const int d = e / p.each, i = e % p.each;
    const Rows r = tc::rows_of(p.offsets[d], i, p.capacity);
    const int n0 = static_cast<int>(at / across) * kSimpleN, m0 = static_cast<int>(at % across) * kSimpleM;
    const int ns = min(kSimpleN, (WEIGHT ? p.N : r.count) - n0), ms = min(kSimpleM, p.M - m0), K = WEIGHT ? r.count : p.K;
    const int es = El<DT>::kSize;
    const char* a = static_cast<const char*>(p.a[d]) + ((WEIGHT ? r.first * p.ak : i * p.ae) + m0 * p.am) * es;
    const char* b = static_cast<const char*>(p.b[d]) + (r.first * (WEIGHT ? p.bk : p.bn) + n0 * p.bn) * es;
    const bool ka = p.ak == 1, kb = p.bk == 1;
    float acc[4][8] = {};
    SimpleTile<DT, kSimpleM> ta;
    SimpleTile<DT, kSimpleN> tb;
    const int steps = (K + kSimpleK - 1) / kSimpleK;
    __syncthreads();  // the last tile's products have read shared memory
    for (int s = 0; s <= steps; ++s) {
      if (s < steps) {
        const int k0 = s * kSimpleK;
        ta.load(a + static_cast<int64_t>(k0) * p.ak * es, p.am, p.ak, ms, K - k0);
        tb.load(b + static_cast<int64_t>(k0) * p.bk * es, p.bn, p.bk, ns, K - k0);
      }
      if (s > 0) {
        const int w = (s - 1) & 1;
#pragma unroll
        for (int k = 0; k < kSimpleK; ++k) {
          float x[8], y[4];
          *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(&sa[w][k][tx * 4]);
          *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(&sa[w][k][64 + tx * 4]);
          *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(&sb[w][k][ty * 4]);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int l = 0; l < 8; ++l) acc[j][l] = fmaf(y[j], x[l], acc[j][l]);
        }
      }
      if (s < steps) {
        ta.store(sa[s & 1], ka);
        tb.store(sb[s & 1], kb);
        __syncthreads();
      }
    }
    void* out = p.out[d];
    const int64_t row = WEIGHT ? static_cast<int64_t>(i) * p.N + n0 : static_cast<int64_t>(r.first) + n0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = ty * 4 + j;
      if (n >= ns) continue;
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        const int m = (l / 4) * 64 + tx * 4 + l % 4;
        if (m < ms) El<OUT>::store(out, (row + n) * p.M + m0 + m, acc[j][l]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
const void* const* untyped(const int32_t* const* a) { return reinterpret_cast<const void* const*>(a); }

struct Sizes {
  int nranks, nexperts, each;
  int64_t capacity, in, out;
};

vc_status_t check_sizes(Sizes* z, int nranks, int nexperts, size_t capacity, size_t in, size_t out) {
  vc_status_t rc = check_ranks(nranks);
  if (rc != VC_SUCCESS) return rc;
  if (nexperts < 1 || nexperts > VC_ROUTE_MAX_EXPERTS || nexperts % nranks != 0)
    return fail(VC_ERR_INVALID_ARG, "nexperts must be in [1, VC_ROUTE_MAX_EXPERTS] and a multiple of nranks");
  if (in > VC_EXPERT_MAX_WIDTH || out > VC_EXPERT_MAX_WIDTH) return fail(VC_ERR_UNSUPPORTED, "a width above VC_EXPERT_MAX_WIDTH");
  rc = check_tokens(nranks, capacity, std::max(in, out));
  if (rc != VC_SUCCESS) return rc;
  *z = Sizes{nranks, nexperts, nexperts / nranks, static_cast<int64_t>(capacity), static_cast<int64_t>(in), static_cast<int64_t>(out)};
  return VC_SUCCESS;
}

// Blocks of a simple kernel, for `tiles` of them at most.
template <auto K>
unsigned simple_blocks(DeviceState* st, int dev, int64_t tiles) {
  const int64_t fit = int64_t(st->nsm) * resident_blocks<K>(dev, kSimpleThreads, 0);
  return static_cast<unsigned>(std::max<int64_t>(1, std::min(tiles, fit)));
}
// Tiles of at most `most` rows that the ranks' experts can make.
int64_t row_tiles(const Sizes& z, int most) {
  return z.nranks * (std::min<int64_t>(z.each, z.capacity) + z.capacity / most);
}

// rows (capacity, in) times weights, in by out or out by in, to out (capacity, out).
vc_status_t rows_product(DeviceState* st, int dev, const Sizes& z, const void* const* rows, const void* const* weight,
                         const int32_t* const* offsets, void* const* out, int64_t in, int64_t width, bool transposed,
                         vc_dtype_t dtype, int step, cudaStream_t stream) {
  SimpleParams p = {};
  for (int r = 0; r < z.nranks; ++r) {
    p.a[r] = weight[r];
    p.b[r] = rows[r];
    p.out[r] = out[r];
    p.offsets[r] = offsets[r];
  }
  p.am = transposed ? in : 1;
  p.ak = transposed ? 1 : width;
  p.ae = in * width;
  p.bn = in;
  p.bk = 1;
  p.capacity = static_cast<int32_t>(z.capacity);
  p.M = static_cast<int>(width);
  p.K = static_cast<int>(in);
  p.experts = z.nexperts;
  p.each = z.each;
  const int64_t bytes = (z.nranks * z.capacity * (in + width) + z.nexperts * in * width) * dtype_size(dtype);
  const int64_t tiles = row_tiles(z, kSimpleN) * ((width + kSimpleM - 1) / kSimpleM);
  return for_dtype(dtype, [&](auto code) {
    constexpr auto K = product_simple_kernel<code(), code(), false>;
    return launch<K>(dev, Shape{simple_blocks<K>(st, dev, tiles), kSimpleThreads}, stream, p, kExpertProduct, step, bytes);
  });
}

// dweight(n, m) = sum over the expert's rows of left(row, n) * right(row, m).
vc_status_t weights_gradient(DeviceState* st, int dev, const Sizes& z, const void* const* left, const void* const* right,
                             const int32_t* const* offsets, void* const* dweight, int64_t N, int64_t M, vc_dtype_t dtype,
                             vc_dtype_t out_dtype, int step, cudaStream_t stream) {
  SimpleParams p = {};
  for (int r = 0; r < z.nranks; ++r) {
    p.a[r] = right[r];
    p.b[r] = left[r];
    p.out[r] = dweight[r];
    p.offsets[r] = offsets[r];
  }
  p.am = p.bn = 1;
  p.ak = M;
  p.bk = N;
  p.capacity = static_cast<int32_t>(z.capacity);
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.experts = z.nexperts;
  p.each = z.each;
  const int64_t bytes = z.nranks * z.capacity * (N + M) * dtype_size(dtype) + z.nexperts * N * M * dtype_size(out_dtype);
  const int64_t tiles = z.nexperts * ((N + kSimpleN - 1) / kSimpleN) * ((M + kSimpleM - 1) / kSimpleM);
  const auto go = [&](auto code, auto out) {
    constexpr auto K = product_simple_kernel<code(), out(), true>;
    return launch<K>(dev, Shape{simple_blocks<K>(st, dev, tiles), kSimpleThreads}, stream, p, kExpertWeight, step, bytes);
  };
  return for_dtype(dtype, [&](auto code) {
    return out_dtype == VC_FLOAT32 ? go(code, std::integral_constant<int, VC_FLOAT32>{}) : go(code, code);
  });
}

vc_status_t product(const void* const* rows, const void* const* weight, const int32_t* const* offsets, void* const* out,
                    int nranks, int nexperts, size_t capacity, size_t in, size_t width, int transposed, vc_dtype_t dtype,
                    cudaStream_t stream) {
  Sizes z;
  vc_status_t rc = check_sizes(&z, nranks, nexperts, capacity, in, width);
  if (rc == VC_SUCCESS) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  const int es = dtype_size(dtype);
  Buffers b;
  rc = b.add(rows, nranks, z.capacity * z.in * es, es, false, "rows");
  if (rc == VC_SUCCESS) rc = b.add(weight, nranks, z.each * z.in * z.out * es, es, false, "weight");
  if (rc == VC_SUCCESS) rc = b.add(untyped(offsets), nranks, (z.each + 1) * 4, 4, false, "offsets");
  if (rc == VC_SUCCESS) rc = b.add(out, nranks, z.capacity * z.out * es, es, true, "out");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || z.capacity == 0 || z.out == 0) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  return rows_product(st, dev, z, rows, weight, offsets, out, z.in, z.out, transposed != 0, dtype, 0, stream);
}

vc_status_t product_grad(const void* const* dout, const void* const* rows, const void* const* weight,
                         const int32_t* const* offsets, void* const* drows, void* const* dweight, int nranks,
                         int nexperts, size_t capacity, size_t in, size_t width, int transposed, vc_dtype_t dtype,
                         vc_dtype_t dweight_dtype, cudaStream_t stream) {
  Sizes z;
  vc_status_t rc = check_sizes(&z, nranks, nexperts, capacity, in, width);
  if (rc == VC_SUCCESS) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  if (!drows && !dweight) return fail(VC_ERR_INVALID_ARG, "no gradient is asked for");
  if (dweight && dweight_dtype != dtype && dweight_dtype != VC_FLOAT32)
    return fail(VC_ERR_UNSUPPORTED, "dweight is of the data type or fp32");
  const int es = dtype_size(dtype), ws = dtype_size(dweight_dtype);
  Buffers b;
  rc = b.add(dout, nranks, z.capacity * z.out * es, es, false, "dout");
  if (rc == VC_SUCCESS && dweight) rc = b.add(rows, nranks, z.capacity * z.in * es, es, false, "rows");
  if (rc == VC_SUCCESS && drows) rc = b.add(weight, nranks, z.each * z.in * z.out * es, es, false, "weight");
  if (rc == VC_SUCCESS) rc = b.add(untyped(offsets), nranks, (z.each + 1) * 4, 4, false, "offsets");
  if (rc == VC_SUCCESS && drows) rc = b.add(drows, nranks, z.capacity * z.in * es, es, true, "drows");
  if (rc == VC_SUCCESS && dweight) rc = b.add(dweight, nranks, z.each * z.in * z.out * ws, ws, true, "dweight");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  if (drows && z.capacity != 0 && z.in != 0) {
    rc = device_state(&st, &dev);
    if (rc == VC_SUCCESS) rc = rows_product(st, dev, z, dout, weight, offsets, drows, z.out, z.in, !transposed, dtype, 0, stream);
    if (rc != VC_SUCCESS) return rc;
  }
  if (dweight && z.in != 0 && z.out != 0) {
    rc = device_state(&st, &dev);
    if (rc == VC_SUCCESS)
      rc = transposed ? weights_gradient(st, dev, z, dout, rows, offsets, dweight, z.out, z.in, dtype, dweight_dtype, drows != nullptr, stream)
                      : weights_gradient(st, dev, z, rows, dout, offsets, dweight, z.in, z.out, dtype, dweight_dtype, drows != nullptr, stream);
  }
  return rc;
}

}  // namespace
}  // namespace layer
}  // namespace vc

using namespace vc;

VC_EXPORT vc_status_t vc_expert_product(const void* const* rows, const void* const* weight,
                                        const int32_t* const* offsets, void* const* out, int nranks, int nexperts,
                                        size_t capacity, size_t in_width, size_t out_width, int transposed,
                                        vc_dtype_t dtype, vc_stream_t stream) {
  return entry([&] {
    return layer::product(rows, weight, offsets, out, nranks, nexperts, capacity, in_width, out_width, transposed, dtype,
                          reinterpret_cast<cudaStream_t>(stream));
  });
}

VC_EXPORT vc_status_t vc_expert_product_backward(const void* const* dout, const void* const* rows,
                                                 const void* const* weight, const int32_t* const* offsets,
                                                 void* const* drows, void* const* dweight, int nranks, int nexperts,
                                                 size_t capacity, size_t in_width, size_t out_width, int transposed,
                                                 vc_dtype_t dtype, vc_dtype_t dweight_dtype, vc_stream_t stream) {
  return entry([&] {
    return layer::product_grad(dout, rows, weight, offsets, drows, dweight, nranks, nexperts, capacity, in_width,
                               out_width, transposed, dtype, dweight_dtype, reinterpret_cast<cudaStream_t>(stream));
  });
}
