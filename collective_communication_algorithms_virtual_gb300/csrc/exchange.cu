// The exchange of tokens between the ranks that hold them and the ranks that
// hold their experts: the plan from the chosen experts, the rows there
// (dispatch), the answers back (combine), and combine's gradient (see vc.h).
//
// The plan is a stable counting sort by expert in one launch of one
// thread-block cluster; no atomics, so the order is the definition's.  The
// moves stream: each token's row is read once and written to all its places,
// or the other way round, 16 bytes a thread where rows allow it.
#include <cooperative_groups.h>

#include "layer.cuh"

namespace vc {
namespace layer {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

struct DispatchPlanParams {
  const int32_t* ids[VC_MAX_RANKS];
  int32_t* slots[VC_MAX_RANKS];
  int32_t* offsets[VC_MAX_RANKS];
  uint32_t per;       // choices of each rank
  uint32_t total;     // of all ranks
  uint32_t piece;     // of each warp, a multiple of 32
  int experts, each;  // experts, and of each rank
  uint32_t capacity;
};

size_t plan_smem(int experts) { return static_cast<size_t>(experts) * (kPlanWarps + 3) * sizeof(uint32_t); }

// The choices, in order of (source rank, token, choice), are cut into one
// contiguous piece per warp.  Each warp counts its piece by expert; the counts
// before each warp's (of the same expert), the experts before (on the same
// rank) and the equal choices before in the warp's own piece add up to a
// choice's row.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ DispatchPlanParams p) {
  extern __shared__ uint32_t sm[];
  __shared__ uint32_t part[32];
  cg::cluster_group cluster = cg::this_cluster();
  const int E = p.experts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* count = sm + warp * E;              // [warps][E]: this warp's row
  uint32_t* total = sm + kPlanWarps * E;        // [E]: this block's counts
  uint32_t* first = total + E;                  // [E]: where the expert begins, over all ranks
  uint32_t* base = first + E;                   // [E]: row of this block's first choice of the expert
  for (int i = tid; i < kPlanWarps * E; i += kPlanThreads) sm[i] = 0;
  __syncthreads();
  stream_order();
  const uint32_t lo = (cluster.block_rank() * kPlanWarps + warp) * p.piece;
  const uint32_t hi = min(p.total, lo + p.piece);
  const auto expert = [&](uint32_t a) {
    if (a >= hi) return -1;
    const uint32_t r = a / p.per;
    const int e = p.ids[r][a - r * p.per];
    return e >= 0 && e < E ? e : -1;
  };
  for (uint32_t a = lo; a < hi; a += 32) {
    const int e = expert(a + lane);
    const unsigned same = __match_any_sync(kAll, e);
    if (e >= 0 && lane == __ffs(same) - 1) count[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  uint32_t sum = 0;
  if (tid < E) {
    for (int w = 0; w < kPlanWarps; ++w) {
      const uint32_t n = sm[w * E + tid];
      sm[w * E + tid] = sum;
      sum += n;
    }
    total[tid] = sum;
  }
  cluster.sync();
  uint32_t before = 0, all = 0;
  if (tid < E)
    for (unsigned b = 0; b < cluster.num_blocks(); ++b) {
      const uint32_t n = *cluster.map_shared_rank(total + tid, b);
      if (b < cluster.block_rank()) before += n;
      all += n;
    }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // the others' counts are read
  uint32_t upto = all;  // inclusive scan over the experts
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t n = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += n;
  }
  if (lane == 31) part[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    uint32_t n = part[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t m = __shfl_up_sync(kAll, n, d);
      if (lane >= d) n += m;
    }
    part[lane] = n;
  }
  __syncthreads();
  if (warp > 0) upto += part[warp - 1];
  if (tid < E) first[tid] = upto - all;
  __syncthreads();
  if (tid < E) {
    const int d = tid / p.each, i = tid - d * p.each;
    const uint32_t here = first[tid] - first[tid - i];  // row on the expert's rank
    base[tid] = here + before;
    if (cluster.block_rank() == 0) {
      p.offsets[d][i] = static_cast<int32_t>(min(here, p.capacity));
      if (i == p.each - 1) p.offsets[d][p.each] = static_cast<int32_t>(min(here + all, p.capacity));
    }
  }
  __syncthreads();
  for (uint32_t a = lo; a < hi; a += 32) {
    const int e = expert(a + lane);
    const unsigned same = __match_any_sync(kAll, e);
    uint32_t row = 0;
    if (e >= 0) row = base[e] + count[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) count[e] += __popc(same);
    __syncwarp();
    if (a + lane < hi) {
      const uint32_t r = (a + lane) / p.per;
      p.slots[r][a + lane - r * p.per] =
          e >= 0 && row < p.capacity ? static_cast<int32_t>(static_cast<uint32_t>(e / p.each) * p.capacity + row) : -1;
    }
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no block ends while its counts are read
}

// ---------------------------------------------------------------------------
// moves
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kUnits = 4;  // units of a thread in one piece of a row

// A slot's rank and row; the address of `width` bytes per row, or null where
// the slot is skipped.
struct Slots {
  const int32_t* slots[VC_MAX_RANKS];
  uint32_t rows, capacity, limit;  // limit: nranks * capacity
  int topk;
};
__device__ __forceinline__ bool locate(const Slots& p, int slot, uint32_t* rank, uint32_t* row) {
  if (slot < 0 || static_cast<uint32_t>(slot) >= p.limit) return false;
  *rank = static_cast<uint32_t>(slot) / p.capacity;
  *row = static_cast<uint32_t>(slot) - *rank * p.capacity;
  return true;
}

struct DispatchParams {
  const void* send[VC_MAX_RANKS];
  const float* scale[VC_MAX_RANKS];
  void* recv[VC_MAX_RANKS];
  float* recv_scale[VC_MAX_RANKS];
  Slots s;
  int64_t units;  // of a row
  uint32_t pieces;
  int64_t tiles;  // tokens * pieces
  int has_scale;
};

// One warp moves one piece (kUnits units a lane) of one token's row to all its
// places.  U: the unit, 16 bytes or an element.
template <class U>
__global__ void __launch_bounds__(kMoveThreads) dispatch_kernel(const __grid_constant__ DispatchParams p) {
  stream_order();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMoveWarps;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5); tile < p.tiles; tile += step) {
    const uint32_t token = static_cast<uint32_t>(tile / p.pieces);
    const uint32_t piece = static_cast<uint32_t>(tile - static_cast<int64_t>(token) * p.pieces);
    const uint32_t r = token / p.s.rows, t = token - r * p.s.rows;
    const int64_t at = static_cast<int64_t>(piece) * 32 * kUnits + lane;
    const U* from = static_cast<const U*>(p.send[r]) + static_cast<int64_t>(t) * p.units;
    U v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (at + u * 32 < p.units) v[u] = from[at + u * 32];
    char* to = nullptr;  // lane j: where choice j goes
    if (lane < p.s.topk) {
      uint32_t rank, row;
      if (locate(p.s, p.s.slots[r][static_cast<int64_t>(t) * p.s.topk + lane], &rank, &row)) {
        to = reinterpret_cast<char*>(static_cast<U*>(p.recv[rank]) + static_cast<int64_t>(row) * p.units);
        if (p.has_scale && piece == 0) p.recv_scale[rank][row] = p.scale[r][t];
      }
    }
    for (int j = 0; j < p.s.topk; ++j) {
      U* d = reinterpret_cast<U*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(to), j));
      if (!d) continue;
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        if (at + u * 32 < p.units) d[at + u * 32] = v[u];
    }
  }
}

struct CombineParams {
  const void* recv[VC_MAX_RANKS];
  const float* weights[VC_MAX_RANKS];
  void* out[VC_MAX_RANKS];
  Slots s;
  int64_t units;
  uint32_t pieces;
  int64_t tiles;
  int has_weights;
};

// One unit of a row in fp32: a 16-byte vector, or an element.
template <int DT, bool VEC>
struct Unit {
  static constexpr int kN = VEC ? El<DT>::kVec : 1;
  static constexpr int kBytes = VEC ? 16 : El<DT>::kSize;
  static __device__ __forceinline__ void load(const char* row, int64_t i, float* f) {
    if constexpr (VEC) El<DT>::widen(dev::ld16(row + i * 16), f);
    else f[0] = El<DT>::load(row, i);
  }
  static __device__ __forceinline__ void store(char* row, int64_t i, const float* f) {
    if constexpr (VEC) dev::st16_wb(row + i * 16, El<DT>::narrow(f));
    else El<DT>::store(row, i, f[0]);
  }
};

constexpr int kCombineUnits = 2;  // units of a thread in one piece
constexpr int kCombineBatch = 4;  // choices whose loads are in flight together

template <int DT, bool VEC>
__global__ void __launch_bounds__(kMoveThreads) combine_kernel(const __grid_constant__ CombineParams p) {
  using X = Unit<DT, VEC>;
  stream_order();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMoveWarps;
  const int64_t width = p.units * X::kBytes;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5); tile < p.tiles; tile += step) {
    const uint32_t token = static_cast<uint32_t>(tile / p.pieces);
    const uint32_t piece = static_cast<uint32_t>(tile - static_cast<int64_t>(token) * p.pieces);
    const uint32_t r = token / p.s.rows, t = token - r * p.s.rows;
    const int64_t at = static_cast<int64_t>(piece) * 32 * kCombineUnits + lane;
    const char* from = nullptr;  // lane j: choice j's row and weight
    float weight = 0.f;
    if (lane < p.s.topk) {
      uint32_t rank, row;
      const int64_t j = static_cast<int64_t>(t) * p.s.topk + lane;
      if (locate(p.s, p.s.slots[r][j], &rank, &row)) {
        from = static_cast<const char*>(p.recv[rank]) + static_cast<int64_t>(row) * width;
        weight = p.has_weights ? p.weights[r][j] : 1.f;
      }
    }
    float sum[kCombineUnits][X::kN];
#pragma unroll
    for (int u = 0; u < kCombineUnits; ++u)
#pragma unroll
      for (int i = 0; i < X::kN; ++i) sum[u][i] = 0.f;
    for (int j0 = 0; j0 < p.s.topk; j0 += kCombineBatch) {
      float v[kCombineBatch][kCombineUnits][X::kN], w[kCombineBatch];
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b) {  // lanes past topk hold no row
        const int j = (j0 + b) & 31;
        const char* s = reinterpret_cast<const char*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(from), j));
        w[b] = __shfl_sync(kAll, weight, j);
        if (j0 + b >= p.s.topk) s = nullptr;
#pragma unroll
        for (int u = 0; u < kCombineUnits; ++u) {
          if (s && at + u * 32 < p.units) {
            X::load(s, at + u * 32, v[b][u]);
          } else {
            if (!s) w[b] = 0.f;
#pragma unroll
            for (int i = 0; i < X::kN; ++i) v[b][u][i] = 0.f;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b)
#pragma unroll
        for (int u = 0; u < kCombineUnits; ++u)
#pragma unroll
          for (int i = 0; i < X::kN; ++i) sum[u][i] += w[b] * v[b][u][i];
    }
    char* to = static_cast<char*>(p.out[r]) + static_cast<int64_t>(t) * width;
#pragma unroll
    for (int u = 0; u < kCombineUnits; ++u)
      if (at + u * 32 < p.units) X::store(to, at + u * 32, sum[u]);
  }
}

struct CombineGradParams {
  const void* dout[VC_MAX_RANKS];
  const void* recv[VC_MAX_RANKS];
  const float* weights[VC_MAX_RANKS];
  void* drecv[VC_MAX_RANKS];
  float* dweights[VC_MAX_RANKS];
  Slots s;
  int64_t units;
  int has_weights, has_drecv, has_dweights;
};
constexpr int kGradBatch = 8;  // choices whose dot products are in registers together

// One block takes one token.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kMoveThreads) combine_grad_kernel(const __grid_constant__ CombineGradParams p) {
  using X = Unit<DT, VEC>;
  __shared__ const char* from[VC_ROUTE_MAX_TOPK];
  __shared__ char* to[VC_ROUTE_MAX_TOPK];
  __shared__ float weight[VC_ROUTE_MAX_TOPK];
  __shared__ float dots[kMoveWarps][VC_ROUTE_MAX_TOPK];
  stream_order();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const uint32_t token = blockIdx.x;
  const uint32_t r = token / p.s.rows, t = token - r * p.s.rows;
  const int k = p.s.topk;
  const int64_t width = p.units * X::kBytes;
  if (warp == 0 && lane < k) {
    uint32_t rank, row;
    const int64_t j = static_cast<int64_t>(t) * k + lane;
    from[lane] = nullptr;
    to[lane] = nullptr;
    if (locate(p.s, p.s.slots[r][j], &rank, &row)) {
      if (p.has_dweights) from[lane] = static_cast<const char*>(p.recv[rank]) + static_cast<int64_t>(row) * width;
      if (p.has_drecv) to[lane] = static_cast<char*>(p.drecv[rank]) + static_cast<int64_t>(row) * width;
      weight[lane] = p.has_weights ? p.weights[r][j] : 1.f;
    }
  }
  __syncthreads();
  const char* dout = static_cast<const char*>(p.dout[r]) + static_cast<int64_t>(t) * width;
  for (int j0 = 0; j0 < k; j0 += kGradBatch) {
    float dot[kGradBatch];
#pragma unroll
    for (int b = 0; b < kGradBatch; ++b) dot[b] = 0.f;
    for (int64_t c = threadIdx.x; c < p.units; c += blockDim.x) {
      float g[X::kN];
      X::load(dout, c, g);
#pragma unroll
      for (int b = 0; b < kGradBatch; ++b) {
        if (j0 + b < k) {
          if (from[j0 + b]) {
            float y[X::kN];
            X::load(from[j0 + b], c, y);
#pragma unroll
            for (int i = 0; i < X::kN; ++i) dot[b] += g[i] * y[i];
          }
          if (to[j0 + b]) {
            float d[X::kN];
#pragma unroll
            for (int i = 0; i < X::kN; ++i) d[i] = weight[j0 + b] * g[i];
            X::store(to[j0 + b], c, d);
          }
        }
      }
    }
    if (p.has_dweights) {
#pragma unroll
      for (int b = 0; b < kGradBatch; ++b) {
        const float x = warp_sum(dot[b]);
        if (lane == 0 && j0 + b < k) dots[warp][j0 + b] = x;
      }
    }
  }
  if (p.has_dweights) {
    __syncthreads();
    if (warp == 0 && lane < k) {
      float x = 0.f;
      for (int w = 0; w < warps; ++w) x += dots[w][lane];
      p.dweights[r][static_cast<int64_t>(t) * k + lane] = x;  // a skipped choice's dot is 0
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
constexpr int64_t kMaxInt = 0x7fffffff;

vc_status_t check_slots(int nranks, size_t rows, int topk, size_t capacity) {
  vc_status_t rc = check_ranks(nranks);
  if (rc != VC_SUCCESS) return rc;
  if (topk < 1 || topk > VC_ROUTE_MAX_TOPK) return fail(VC_ERR_INVALID_ARG, "topk outside [1, 32]");
  if (capacity < 1 || capacity > static_cast<size_t>(kMaxInt / nranks))
    return fail(VC_ERR_INVALID_ARG, "nranks * capacity outside [1, 2^31 - 1]");
  if (rows > static_cast<size_t>(kMaxInt / nranks / topk)) return fail(VC_ERR_INVALID_ARG, "too many choices");
  return VC_SUCCESS;
}
template <class T>
const void* const* untyped(T* const* a) {
  return reinterpret_cast<const void* const*>(const_cast<const std::remove_const_t<T>* const*>(a));
}

// Warps of a cluster that sorts `total` choices.
unsigned plan_blocks(int64_t total) { return total <= 4096 ? 1 : total <= 32768 ? 8 : 16; }

vc_status_t dispatch_plan(const int32_t* const* ids, int32_t* const* slots, int32_t* const* offsets, int nranks,
                          size_t rows, int topk, int nexperts, size_t capacity, cudaStream_t stream) {
  vc_status_t rc = check_slots(nranks, rows, topk, capacity);
  if (rc != VC_SUCCESS) return rc;
  if (nexperts < 1 || nexperts > VC_ROUTE_MAX_EXPERTS || nexperts % nranks)
    return fail(VC_ERR_INVALID_ARG, "nexperts must be in [1, 1024] and a multiple of nranks");
  const int64_t per = static_cast<int64_t>(rows) * topk, each = nexperts / nranks;
  Buffers b;
  rc = b.add(untyped(ids), nranks, per * 4, 4, false, "ids");
  if (rc == VC_SUCCESS) rc = b.add(untyped(slots), nranks, per * 4, 4, true, "slots");
  if (rc == VC_SUCCESS) rc = b.add(untyped(offsets), nranks, (each + 1) * 4, 4, true, "offsets");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS) return rc;
  if (rows == 0) {
    for (int r = 0; r < nranks; ++r) {
      cudaError_t e = cudaMemsetAsync(offsets[r], 0, static_cast<size_t>(each + 1) * 4, stream);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    }
    return VC_SUCCESS;
  }
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  DispatchPlanParams p = {};
  for (int r = 0; r < nranks; ++r) {
    p.ids[r] = ids[r];
    p.slots[r] = slots[r];
    p.offsets[r] = offsets[r];
  }
  const int64_t total = per * nranks;
  const unsigned blocks = plan_blocks(total);
  const int64_t warps = static_cast<int64_t>(blocks) * kPlanWarps;
  p.per = static_cast<uint32_t>(per);
  p.total = static_cast<uint32_t>(total);
  p.piece = static_cast<uint32_t>(((total + warps - 1) / warps + 31) / 32 * 32);
  p.experts = nexperts;
  p.each = static_cast<int>(each);
  p.capacity = static_cast<uint32_t>(capacity);
  return launch<plan_kernel>(dev, Shape{blocks, kPlanThreads, plan_smem(nexperts), blocks}, stream, p, kPlan, 0,
                             total * 8 + (int64_t(nexperts) + nranks) * 4);
}

Slots slots_of(const int32_t* const* slots, int nranks, size_t rows, int topk, size_t capacity) {
  Slots s = {};
  for (int r = 0; r < nranks; ++r) s.slots[r] = slots[r];
  s.rows = static_cast<uint32_t>(rows);
  s.capacity = static_cast<uint32_t>(capacity);
  s.limit = s.capacity * static_cast<uint32_t>(nranks);
  s.topk = topk;
  return s;
}
// Checks the sizes of a move's rows of `hidden` elements.
vc_status_t check_move(int nranks, size_t rows, size_t hidden, int topk, size_t capacity) {
  vc_status_t rc = check_slots(nranks, rows, topk, capacity);
  if (rc == VC_SUCCESS) rc = check_tokens(nranks, rows, hidden);
  if (rc == VC_SUCCESS) rc = check_tokens(nranks, capacity, hidden);
  return rc;
}
// Blocks for `tiles` tiles of one warp: all of them, or as many as are resident.
template <auto K>
unsigned move_blocks(DeviceState* st, int dev, int64_t tiles) {
  const int64_t want = (tiles + kMoveWarps - 1) / kMoveWarps;
  return static_cast<unsigned>(std::min<int64_t>(want, int64_t(st->nsm) * resident_blocks<K>(dev, kMoveThreads, 0)));
}

template <class U>
vc_status_t launch_dispatch(DeviceState* st, int dev, DispatchParams& p, int64_t row_bytes, int64_t bytes, cudaStream_t s) {
  p.units = row_bytes / static_cast<int64_t>(sizeof(U));
  p.pieces = static_cast<uint32_t>((p.units + 32 * kUnits - 1) / (32 * kUnits));
  p.tiles = p.tiles * p.pieces;
  return launch<dispatch_kernel<U>>(dev, Shape{move_blocks<dispatch_kernel<U>>(st, dev, p.tiles), kMoveThreads}, s, p, kDispatch, 0, bytes);
}

vc_status_t dispatch(const void* const* send, const float* const* scale, const int32_t* const* slots,
                     void* const* recv, float* const* recv_scale, int nranks, size_t rows, size_t hidden, int topk,
                     size_t capacity, vc_dtype_t dtype, cudaStream_t stream) {
  vc_status_t rc = check_move(nranks, rows, hidden, topk, capacity);
  if (rc == VC_SUCCESS && dtype != VC_INT8) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  if (!scale != !recv_scale) return fail(VC_ERR_INVALID_ARG, "scale and recv_scale come together");
  const int es = dtype_size(dtype);
  const int64_t row = static_cast<int64_t>(hidden) * es, n = static_cast<int64_t>(rows), cap = static_cast<int64_t>(capacity);
  Buffers b;
  rc = b.add(send, nranks, n * row, es, false, "send");
  if (rc == VC_SUCCESS) rc = b.add(recv, nranks, cap * row, es, true, "recv");
  const bool whole = b.aligned16() && row % 16 == 0;
  if (rc == VC_SUCCESS) rc = b.add(untyped(slots), nranks, n * topk * 4, 4, false, "slots");
  if (rc == VC_SUCCESS && scale) rc = b.add(untyped(scale), nranks, n * 4, 4, false, "scale");
  if (rc == VC_SUCCESS && scale) rc = b.add(untyped(recv_scale), nranks, cap * 4, 4, true, "recv_scale");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || rows == 0 || hidden == 0) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  DispatchParams p = {};
  p.s = slots_of(slots, nranks, rows, topk, capacity);
  for (int r = 0; r < nranks; ++r) {
    p.send[r] = send[r];
    p.recv[r] = recv[r];
    if (scale) p.scale[r] = scale[r];
    if (scale) p.recv_scale[r] = recv_scale[r];
  }
  p.has_scale = scale != nullptr;
  p.tiles = n * nranks;
  const int64_t bytes = p.tiles * (row * (1 + topk) + topk * 4 + (scale ? 4 + 4 * topk : 0));
  if (whole) return launch_dispatch<uint4>(st, dev, p, row, bytes, stream);
  if (es == 4) return launch_dispatch<uint32_t>(st, dev, p, row, bytes, stream);
  if (es == 2) return launch_dispatch<uint16_t>(st, dev, p, row, bytes, stream);
  return launch_dispatch<uint8_t>(st, dev, p, row, bytes, stream);
}

vc_status_t combine(const void* const* recv, const int32_t* const* slots, const float* const* weights,
                    void* const* out, int nranks, size_t rows, size_t hidden, int topk, size_t capacity,
                    vc_dtype_t dtype, cudaStream_t stream) {
  vc_status_t rc = check_move(nranks, rows, hidden, topk, capacity);
  if (rc == VC_SUCCESS) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  const int es = dtype_size(dtype);
  const int64_t row = static_cast<int64_t>(hidden) * es, n = static_cast<int64_t>(rows), cap = static_cast<int64_t>(capacity);
  Buffers b;
  rc = b.add(recv, nranks, cap * row, es, false, "recv");
  if (rc == VC_SUCCESS) rc = b.add(out, nranks, n * row, es, true, "out");
  const bool whole = b.aligned16() && row % 16 == 0;
  if (rc == VC_SUCCESS) rc = b.add(untyped(slots), nranks, n * topk * 4, 4, false, "slots");
  if (rc == VC_SUCCESS && weights) rc = b.add(untyped(weights), nranks, n * topk * 4, 4, false, "weights");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || rows == 0 || hidden == 0) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  CombineParams p = {};
  p.s = slots_of(slots, nranks, rows, topk, capacity);
  for (int r = 0; r < nranks; ++r) {
    p.recv[r] = recv[r];
    p.out[r] = out[r];
    if (weights) p.weights[r] = weights[r];
  }
  p.has_weights = weights != nullptr;
  const int64_t bytes = n * nranks * (row * (1 + topk) + topk * (weights ? 8 : 4));
  return for_dtype(dtype, [&](auto code) {
    constexpr int DT = code();
    const auto go = [&](auto vec) {
      constexpr bool VEC = vec();
      p.units = row / Unit<DT, VEC>::kBytes;
      p.pieces = static_cast<uint32_t>((p.units + 32 * kCombineUnits - 1) / (32 * kCombineUnits));
      p.tiles = n * nranks * p.pieces;
      return launch<combine_kernel<DT, VEC>>(dev, Shape{move_blocks<combine_kernel<DT, VEC>>(st, dev, p.tiles), kMoveThreads}, stream, p,
                                             kCombine, 0, bytes);
    };
    return whole ? go(std::true_type{}) : go(std::false_type{});
  });
}

vc_status_t combine_grad(const void* const* dout, const void* const* recv, const int32_t* const* slots,
                         const float* const* weights, void* const* drecv, float* const* dweights, int nranks,
                         size_t rows, size_t hidden, int topk, size_t capacity, vc_dtype_t dtype, cudaStream_t stream) {
  vc_status_t rc = check_move(nranks, rows, hidden, topk, capacity);
  if (rc == VC_SUCCESS) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  if (!drecv && !dweights) return fail(VC_ERR_INVALID_ARG, "no gradient is asked for");
  const int es = dtype_size(dtype);
  const int64_t row = static_cast<int64_t>(hidden) * es, n = static_cast<int64_t>(rows), cap = static_cast<int64_t>(capacity);
  Buffers b;
  rc = b.add(dout, nranks, n * row, es, false, "dout");
  if (rc == VC_SUCCESS && dweights) rc = b.add(recv, nranks, cap * row, es, false, "recv");
  if (rc == VC_SUCCESS && drecv) rc = b.add(drecv, nranks, cap * row, es, true, "drecv");
  const bool whole = b.aligned16() && row % 16 == 0;
  if (rc == VC_SUCCESS) rc = b.add(untyped(slots), nranks, n * topk * 4, 4, false, "slots");
  if (rc == VC_SUCCESS && weights) rc = b.add(untyped(weights), nranks, n * topk * 4, 4, false, "weights");
  if (rc == VC_SUCCESS && dweights) rc = b.add(untyped(dweights), nranks, n * topk * 4, 4, true, "dweights");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || rows == 0) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  CombineGradParams p = {};
  p.s = slots_of(slots, nranks, rows, topk, capacity);
  for (int r = 0; r < nranks; ++r) {
    p.dout[r] = dout[r];
    if (dweights) p.recv[r] = recv[r];
    if (weights) p.weights[r] = weights[r];
    if (drecv) p.drecv[r] = drecv[r];
    if (dweights) p.dweights[r] = dweights[r];
  }
  p.has_weights = weights != nullptr;
  p.has_drecv = drecv != nullptr;
  p.has_dweights = dweights != nullptr;
  const int64_t bytes = n * nranks * (row * (1 + topk * (p.has_drecv + p.has_dweights)) + topk * 4 * (1 + p.has_weights + p.has_dweights));
  return for_dtype(dtype, [&](auto code) {
    constexpr int DT = code();
    const auto go = [&](auto vec) {
      constexpr bool VEC = vec();
      p.units = row / Unit<DT, VEC>::kBytes;
      const unsigned threads = static_cast<unsigned>(std::max<int64_t>(32, std::min<int64_t>(kMoveThreads, (p.units + 31) / 32 * 32)));
      return launch<combine_grad_kernel<DT, VEC>>(dev, Shape{static_cast<unsigned>(n * nranks), threads}, stream, p, kCombineBackward, 0, bytes);
    };
    return whole ? go(std::true_type{}) : go(std::false_type{});
  });
}

}  // namespace
}  // namespace layer
}  // namespace vc

using namespace vc;

VC_EXPORT vc_status_t vc_dispatch_plan(const int32_t* const* ids, int32_t* const* slots, int32_t* const* offsets,
                                       int nranks, size_t rows, int topk, int nexperts, size_t capacity,
                                       vc_stream_t stream) {
  return entry([&] {
    return layer::dispatch_plan(ids, slots, offsets, nranks, rows, topk, nexperts, capacity,
                                reinterpret_cast<cudaStream_t>(stream));
  });
}

VC_EXPORT vc_status_t vc_dispatch(const void* const* send, const float* const* scale, const int32_t* const* slots,
                                  void* const* recv, float* const* recv_scale, int nranks, size_t rows, size_t hidden,
                                  int topk, size_t capacity, vc_dtype_t dtype, vc_stream_t stream) {
  return entry([&] {
    return layer::dispatch(send, scale, slots, recv, recv_scale, nranks, rows, hidden, topk, capacity, dtype,
                           reinterpret_cast<cudaStream_t>(stream));
  });
}

VC_EXPORT vc_status_t vc_combine(const void* const* recv, const int32_t* const* slots, const float* const* weights,
                                 void* const* out, int nranks, size_t rows, size_t hidden, int topk, size_t capacity,
                                 vc_dtype_t dtype, vc_stream_t stream) {
  return entry([&] {
    return layer::combine(recv, slots, weights, out, nranks, rows, hidden, topk, capacity, dtype,
                          reinterpret_cast<cudaStream_t>(stream));
  });
}

VC_EXPORT vc_status_t vc_combine_backward(const void* const* dout, const void* const* recv,
                                          const int32_t* const* slots, const float* const* weights,
                                          void* const* drecv, float* const* dweights, int nranks, size_t rows,
                                          size_t hidden, int topk, size_t capacity, vc_dtype_t dtype,
                                          vc_stream_t stream) {
  return entry([&] {
    return layer::combine_grad(dout, recv, slots, weights, drecv, dweights, nranks, rows, hidden, topk, capacity,
                               dtype, reinterpret_cast<cudaStream_t>(stream));
  });
}
