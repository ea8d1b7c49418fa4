// The exchange of tokens between the ranks that hold them and the ranks that
// hold their experts: the plan from the chosen experts, the rows there
// (dispatch), the answers back (combine), and combine's gradient (see vc.h).
//
// The plan is a stable counting sort by expert in one launch of one
// thread-block cluster.  The moves stream: each token's row is read once and
// written to all its places, or the other way round, and memory bounds them;
// on a GB300, copy rate 6.69 TB/s, 4096 tokens of 4096 bf16 to 8 places each:
//   dispatch 302 MB, 48.1 us, 6.3 TB/s (its plan 7.1 us)
//   combine  302 MB, 48.3 us, 6.3 TB/s
//   combine's gradient 570 MB, 94.9 us, 6.0 TB/s
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
  int bits;           // of the largest expert
  uint32_t capacity;
};

constexpr int kPlanRow = kPlanWarps + 1;  // counts of one expert, a bank apart from the next expert's
constexpr int kPlanAhead = 4;             // choices of a lane whose loads are in flight together

size_t plan_smem(int experts) { return static_cast<size_t>(experts) * (kPlanRow + 3) * sizeof(uint32_t); }

// The choices, in order of (source rank, token, choice), are cut into one
// contiguous piece per warp.  Each warp counts its piece by expert; the counts
// before each warp's (of the same expert), the experts before (on the same
// rank) and the equal choices before in the warp's own piece add up to a
// choice's row.  Counting is additions of whole numbers in shared memory, in
// any order; equal choices of a step are found by a ballot for each bit of the
// expert (__match_any_sync: 13.0 us on 8 blocks where this takes 8.8).
// Latency bounds it: two walks over the ids, a cluster barrier, two scans.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ DispatchPlanParams p) {
  extern __shared__ uint32_t sm[];
  __shared__ uint32_t part[32];
  cg::cluster_group cluster = cg::this_cluster();
  const int E = p.experts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* count = sm + warp;                  // [E] of stride kPlanRow: this warp's counts
  uint32_t* total = sm + kPlanRow * E;          // [E]: this block's counts
  uint32_t* first = total + E;                  // [E]: where the expert begins, over all ranks
  uint32_t* base = first + E;                   // [E]: row of this block's first choice of the expert
  for (int i = tid; i < kPlanRow * E; i += kPlanThreads) sm[i] = 0;
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
  for (uint32_t a = lo; a < hi; a += 32 * kPlanAhead) {
    int e[kPlanAhead];
#pragma unroll
    for (int i = 0; i < kPlanAhead; ++i) e[i] = expert(a + i * 32 + lane);
#pragma unroll
    for (int i = 0; i < kPlanAhead; ++i)
      if (e[i] >= 0) atomicAdd(count + e[i] * kPlanRow, 1u);  // this warp's own count: whole numbers, in any order
  }
  __syncthreads();
  for (int e = warp; e < E; e += kPlanWarps) {  // lane w: what the warps before w counted
    const uint32_t n = sm[e * kPlanRow + lane];
    uint32_t upto = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t m = __shfl_up_sync(kAll, upto, d);
      if (lane >= d) upto += m;
    }
    sm[e * kPlanRow + lane] = upto - n;
    if (lane == 31) total[e] = upto;
  }
  cluster.sync();
  uint32_t before = 0, all = 0;
  if (tid < E)
    for (unsigned b = 0; b < cluster.num_blocks(); ++b) {
      const uint32_t n = *cluster.map_shared_rank(total + tid, b);
      if (b < cluster.block_rank()) before += n;
      all += n;
    }
  __syncwarp();
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
  for (uint32_t a = lo; a < hi; a += 32 * kPlanAhead) {
    int e[kPlanAhead];
#pragma unroll
    for (int i = 0; i < kPlanAhead; ++i) e[i] = expert(a + i * 32 + lane);
#pragma unroll
    for (int i = 0; i < kPlanAhead; ++i) {
      const uint32_t at = a + i * 32 + lane;
      // lanes with the same expert, a ballot for each bit of it
      unsigned same = __ballot_sync(kAll, e[i] >= 0);
      for (int b = 0; b < p.bits; ++b) {
        const bool on = e[i] >> b & 1;
        const unsigned with = __ballot_sync(kAll, on);
        same &= on ? with : ~with;
      }
      uint32_t row = 0;
      if (e[i] >= 0) row = base[e[i]] + count[e[i] * kPlanRow] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (e[i] >= 0 && lane == __ffs(same) - 1) count[e[i] * kPlanRow] += __popc(same);
      __syncwarp();
      if (at < hi) {
        const uint32_t r = at / p.per;
        p.slots[r][at - r * p.per] =
            e[i] >= 0 && row < p.capacity ? static_cast<int32_t>(static_cast<uint32_t>(e[i] / p.each) * p.capacity + row) : -1;
      }
    }
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no block ends while its counts are read
}

// ---------------------------------------------------------------------------
// moves
// ---------------------------------------------------------------------------
// A warp takes a piece of two units a lane of one row (1 KB): small enough
// that 32 tokens of 4 KB still fill 128 warps (2.2 us; pieces of 2 KB 2.6 us).
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kUnits = 2;  // 16-byte units of a thread in one piece of a row
// and of smaller ones
template <class U>
constexpr int kUnitsOf = sizeof(U) == 16 ? kUnits : sizeof(U) == 1 ? 16 : 8;

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
  int64_t n;  // units of a row (bulk copies: bytes)
  uint32_t pieces, piece_bytes;
  int64_t tiles;  // tokens * pieces
  int has_scale;
};

// One warp moves one piece of one token's row to all its places.  U: 16-byte
// vectors, or an element where rows are not made of aligned ones (elements of
// 2 bytes: 62 us for 4096 tokens, 8 choices, 4099 elements; cutting each
// place's vectors out of the row, as combine does, took 76).
template <class U>
__global__ void __launch_bounds__(kMoveThreads) dispatch_kernel(const __grid_constant__ DispatchParams p) {
  constexpr int kU = kUnitsOf<U>;
  stream_order();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMoveWarps;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5); tile < p.tiles; tile += step) {
    const uint32_t token = static_cast<uint32_t>(tile / p.pieces);
    const uint32_t piece = static_cast<uint32_t>(tile - static_cast<int64_t>(token) * p.pieces);
    const uint32_t r = token / p.s.rows, t = token - r * p.s.rows;
    const int64_t at = static_cast<int64_t>(piece) * 32 * kU + lane;
    const U* from = static_cast<const U*>(p.send[r]) + t * p.n;
    U v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (at + u * 32 < p.n) {
        if constexpr (sizeof(U) == 16) v[u] = dev::ld16(from + at + u * 32);
        else v[u] = from[at + u * 32];
      }
    U* to = nullptr;  // lane j: where choice j goes
    if (lane < p.s.topk) {
      uint32_t rank, row;
      if (locate(p.s, p.s.slots[r][static_cast<int64_t>(t) * p.s.topk + lane], &rank, &row)) {
        to = static_cast<U*>(p.recv[rank]) + row * p.n;
        if (p.has_scale && piece == 0) p.recv_scale[rank][row] = p.scale[r][t];
      }
    }
    for (int j = 0; j < p.s.topk; ++j) {
      U* d = reinterpret_cast<U*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(to), j));
      if (!d) continue;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (at + u * 32 < p.n) {
          if constexpr (sizeof(U) == 16) dev::st16(d + at + u * 32, v[u]);
          else d[at + u * 32] = v[u];
        }
    }
  }
}

// Rows of whole 16-byte vectors by bulk copies: each warp keeps kBulkStages
// pieces of rows in flight, global to shared memory (lane 0), and lane j writes
// each landed piece to choice j's place (cp.async.bulk both ways, so no data
// passes through registers).  A stage is refilled once the stores of the piece
// it held have read it.  Waits are bounded as in tma_copy_kernel.
constexpr int kBulkWarps = 4;
constexpr int kBulkStages = 3;
constexpr int kBulkBytes = 8 << 10;  // largest piece
// Taken where it measured faster: long rows to several places, together more
// than L2 holds (4096 tokens, 8 choices: rows of 8 KB 48.6 us against 53.9
// through registers, 4 KB 25.0 against 28.9, 2 KB 12.9 against 7.8 at 4
// choices; 512 tokens of 8 KB 7.8 against 6.8).
constexpr int64_t kBulkMinRow = 4 << 10, kBulkMinBytes = int64_t(128) << 20;
constexpr int kBulkMinChoices = 4;
constexpr size_t kBulkSmem = static_cast<size_t>(kBulkWarps) * kBulkStages * kBulkBytes;

__global__ void __launch_bounds__(kBulkWarps * 32) dispatch_bulk_kernel(const __grid_constant__ DispatchParams p) {
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ uint64_t bars[kBulkWarps][kBulkStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned char* stage = stages + warp * kBulkStages * kBulkBytes;
  uint64_t* bar = bars[warp];
  if (lane == 0) {
    for (int k = 0; k < kBulkStages; ++k)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(dev::smem_addr(bar + k)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  stream_order();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kBulkWarps + warp;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kBulkWarps;
  const int64_t n = first < p.tiles ? (p.tiles - first + step - 1) / step : 0;
  const int64_t width = p.n, piece_bytes = p.piece_bytes;
  struct Piece {
    uint32_t r, t, piece, bytes;
  };
  const auto piece_of = [&](int64_t i) {
    const int64_t tile = first + i * step;
    const uint32_t token = static_cast<uint32_t>(tile / p.pieces);
    Piece x;
    x.piece = static_cast<uint32_t>(tile - static_cast<int64_t>(token) * p.pieces);
    x.r = token / p.s.rows;
    x.t = token - x.r * p.s.rows;
    x.bytes = static_cast<uint32_t>(min(piece_bytes, width - x.piece * piece_bytes));
    return x;
  };
  const auto load = [&](int64_t i) {  // lane 0
    const int k = static_cast<int>(i % kBulkStages);
    const Piece x = piece_of(i);
    const char* from = static_cast<const char*>(p.send[x.r]) + static_cast<int64_t>(x.t) * width + x.piece * piece_bytes;
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(dev::smem_addr(bar + k)), "r"(x.bytes) : "memory");
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                     dev::smem_addr(stage + k * kBulkBytes)),
                 "l"(from), "r"(x.bytes), "r"(dev::smem_addr(bar + k)), "l"(dev::l2_evict_first())
                 : "memory");
  };
  int64_t issued = min(n, static_cast<int64_t>(kBulkStages));
  if (lane == 0)
    for (int64_t i = 0; i < issued; ++i) load(i);
  bool ok = true;
  int64_t i = 0;
  for (; i < n; ++i) {
    const int k = static_cast<int>(i % kBulkStages);
    const Piece x = piece_of(i);
    char* to = nullptr;  // lane j: where choice j goes
    if (lane < p.s.topk) {
      uint32_t rank, row;
      if (locate(p.s, p.s.slots[x.r][static_cast<int64_t>(x.t) * p.s.topk + lane], &rank, &row)) {
        to = static_cast<char*>(p.recv[rank]) + static_cast<int64_t>(row) * width + x.piece * piece_bytes;
        if (p.has_scale && x.piece == 0) p.recv_scale[rank][row] = p.scale[x.r][x.t];
      }
    }
    ok = dev::mbar_wait(dev::smem_addr(bar + k), static_cast<uint32_t>(i / kBulkStages & 1));
    if (!__all_sync(kAll, ok)) {
      ok = false;
      break;
    }
    if (to)
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to),
                   "r"(dev::smem_addr(stage + k * kBulkBytes)), "r"(x.bytes)
                   : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    if (i >= 1 && issued < n) {  // the stage of piece i - 1, once its stores have read it
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
      if (lane == 0) load(issued);
      ++issued;
    }
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  if (!ok && lane == 0) {
    atomicOr(&dev::g_device_error, 2u);
    // loads under way land before the block's shared memory is released
    for (int64_t j = i; j < issued; ++j)
      dev::mbar_wait(dev::smem_addr(bar + j % kBulkStages), static_cast<uint32_t>(j / kBulkStages & 1));
  }
}

struct CombineParams {
  const void* recv[VC_MAX_RANKS];
  const float* weights[VC_MAX_RANKS];
  void* out[VC_MAX_RANKS];
  Slots s;
  int64_t n;  // elements of a row
  uint32_t pieces;
  int64_t tiles;
  int has_weights;
};

constexpr int kCombineBatch = 4;  // choices whose loads are in flight together

// One warp sums one piece of one token's row over its choices, in order, four
// choices' loads in flight (4096 x 8 x 8 KB: 48 us; one at a time 129 us; 8
// choices at once 95 us, for want of registers).
template <int DT, bool VEC>
__global__ void __launch_bounds__(kMoveThreads, VEC ? 4 : 2) combine_kernel(const __grid_constant__ CombineParams p) {
  using E = El<DT>;
  using R = Row<E::kSize, VEC>;
  using Out = Span<E::kSize, 16, VEC>;
  constexpr int kN = E::kVec, kU = kUnits;
  __shared__ __align__(16) unsigned char room[kMoveWarps][Out::kRoom];
  stream_order();
  const int lane = threadIdx.x & 31;
  const int count = static_cast<int>((p.n + kN - 1) / kN);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMoveWarps, width = p.n * E::kSize;
  for (int64_t tile = static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5); tile < p.tiles; tile += step) {
    const uint32_t token = static_cast<uint32_t>(tile / p.pieces);
    const uint32_t piece = static_cast<uint32_t>(tile - static_cast<int64_t>(token) * p.pieces);
    const uint32_t r = token / p.s.rows, t = token - r * p.s.rows;
    char* to = static_cast<char*>(p.out[r]) + t * width;
    const int at = static_cast<int>(piece) * 32 * kU + lane;
    int rank = -1;  // lane j: choice j's row and weight
    uint32_t row = 0;
    float weight = 0.f;
    if (lane < p.s.topk) {
      uint32_t d;
      const int64_t j = static_cast<int64_t>(t) * p.s.topk + lane;
      if (locate(p.s, p.s.slots[r][j], &d, &row)) {
        rank = static_cast<int>(d);
        weight = p.has_weights ? p.weights[r][j] : 1.f;
      }
    }
    float sum[kU][kN];
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) sum[u][i] = 0.f;
    for (int j0 = 0; j0 < p.s.topk; j0 += kCombineBatch) {
      typename R::Raw v[kCombineBatch][kU];
      float w[kCombineBatch];
      const char *recv[kCombineBatch], *s[kCombineBatch];
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b) {
        const int j = min(j0 + b, 31);  // lanes past topk hold no row
        const int d = j0 + b < 32 ? __shfl_sync(kAll, rank, j) : -1;
        recv[b] = d >= 0 ? static_cast<const char*>(p.recv[d]) : nullptr;
        s[b] = recv[b] + __shfl_sync(kAll, row, j) * width;
        w[b] = __shfl_sync(kAll, weight, j);
        const R from(s[b], count, Bytes{recv[b], recv[b] + p.s.capacity * width});
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          v[b][u] = R::zero();
          if (recv[b] && at + u * 32 < count) v[b][u] = from.load(at + u * 32);
        }
      }
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b) {
        if (!recv[b]) continue;
        const R from(s[b], count, Bytes{recv[b], recv[b] + p.s.capacity * width});
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (at + u * 32 >= count) continue;
          float f[kN];
          E::widen(from.finish(v[b][u], at + u * 32, p.n), f);
#pragma unroll
          for (int i = 0; i < kN; ++i) sum[u][i] += w[b] * f[i];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) Out(room[threadIdx.x >> 5], E::narrow(sum[u])).write(to, at - lane + u * 32, p.n);
  }
}

struct CombineGradParams {
  const void* dout[VC_MAX_RANKS];
  const void* recv[VC_MAX_RANKS];
  const float* weights[VC_MAX_RANKS];
  void* drecv[VC_MAX_RANKS];
  float* dweights[VC_MAX_RANKS];
  Slots s;
  int64_t n;
  int has_weights, has_drecv, has_dweights;
};
constexpr int kGradBatch = 4;  // choices whose loads are in flight together

// One block takes one token, so that its dot products meet in one place
// (2048 tokens of 2048 bf16, 4 choices: 75 MB, 16.0 us; a row is read only
// after its slot, and 2.25 rounds of blocks wait for both).
template <int DT, bool VEC>
__global__ void __launch_bounds__(kMoveThreads, VEC ? 6 : 4) combine_grad_kernel(const __grid_constant__ CombineGradParams p) {
  using E = El<DT>;
  using R = Row<E::kSize, VEC>;
  using Out = Span<E::kSize, 16, VEC>;
  constexpr int kN = E::kVec;
  __shared__ const char* from[VC_ROUTE_MAX_TOPK];
  __shared__ const char* base[VC_ROUTE_MAX_TOPK];
  __shared__ char* to[VC_ROUTE_MAX_TOPK];
  __shared__ float weight[VC_ROUTE_MAX_TOPK];
  __shared__ float dots[kMoveWarps][VC_ROUTE_MAX_TOPK];
  __shared__ __align__(16) unsigned char room[kMoveWarps][Out::kRoom];
  stream_order();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const uint32_t r = blockIdx.y, t = blockIdx.x;
  const int k = p.s.topk, count = static_cast<int>((p.n + kN - 1) / kN);
  const int64_t width = p.n * E::kSize;
  if (warp == 0 && lane < k) {
    uint32_t rank, row;
    const int64_t j = static_cast<int64_t>(t) * k + lane;
    from[lane] = nullptr;
    to[lane] = nullptr;
    if (locate(p.s, p.s.slots[r][j], &rank, &row)) {
      if (p.has_dweights) {
        base[lane] = static_cast<const char*>(p.recv[rank]);
        from[lane] = base[lane] + row * width;
      }
      if (p.has_drecv) to[lane] = static_cast<char*>(p.drecv[rank]) + row * width;
      weight[lane] = p.has_weights ? p.weights[r][j] : 1.f;
    }
  }
  __syncthreads();
  const char* gradient = static_cast<const char*>(p.dout[r]);
  const R dout(gradient + t * width, count, Bytes{gradient, gradient + p.s.rows * width});
  const auto answer = [&](int j) { return R(from[j], count, Bytes{base[j], base[j] + p.s.capacity * width}); };
  for (int j0 = 0; j0 < k; j0 += kGradBatch) {
    float dot[kGradBatch];
#pragma unroll
    for (int b = 0; b < kGradBatch; ++b) dot[b] = 0.f;
    for (int c0 = warp * 32; c0 < count; c0 += blockDim.x) {  // the warp's 32 units
      const int c = c0 + lane;
      typename R::Raw graw = R::zero(), y[kGradBatch];
      if (c < count) graw = dout.load(c);
#pragma unroll
      for (int b = 0; b < kGradBatch; ++b) {
        y[b] = R::zero();
        if (j0 + b < k && from[j0 + b] && c < count) y[b] = answer(j0 + b).load(c);
      }
      float g[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) g[i] = 0.f;
      if (c < count) E::widen(dout.finish(graw, c, p.n), g);
      mask_unit<E::kSize, VEC>(c, p.n, g);
#pragma unroll
      for (int b = 0; b < kGradBatch; ++b) {
        if (j0 + b >= k) break;
        if (from[j0 + b] && c < count) {
          float f[kN];
          E::widen(answer(j0 + b).finish(y[b], c, p.n), f);
          mask_unit<E::kSize, VEC>(c, p.n, f);
#pragma unroll
          for (int i = 0; i < kN; ++i) dot[b] += g[i] * f[i];
        }
        if (to[j0 + b]) {
          float d[kN];
#pragma unroll
          for (int i = 0; i < kN; ++i) d[i] = weight[j0 + b] * g[i];
          Out(room[warp], E::narrow(d)).write(to[j0 + b], c0, p.n);
        }
      }
    }
    if (p.has_dweights) {
#pragma unroll
      for (int b = 0; b < kGradBatch; ++b) {
        const float s = warp_sum(dot[b]);
        if (lane == 0 && j0 + b < k) dots[warp][j0 + b] = s;
      }
    }
  }
  if (p.has_dweights) {
    __syncthreads();
    if (warp == 0 && lane < k) {
      float s = 0.f;
      for (int w = 0; w < warps; ++w) s += dots[w][lane];
      p.dweights[r][static_cast<int64_t>(t) * k + lane] = from[lane] ? s : 0.f;  // a skipped choice's row was not read
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

// Most blocks of a cluster of the plan: 16, above the portable size, where the
// device can place such a one with the shared memory of the most experts, else
// 8.  Asked once per device.
unsigned plan_cluster(int dev) {
  static std::atomic<unsigned> most[64];
  unsigned n = most[dev].load(std::memory_order_relaxed);
  if (n) return n;
  n = 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = plan_smem(VC_ROUTE_MAX_EXPERTS);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {16, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (allow<plan_kernel>(dev, cfg.dynamicSmemBytes, true) == VC_SUCCESS &&
      cudaOccupancyMaxActiveClusters(&clusters, plan_kernel, &cfg) == cudaSuccess && clusters >= 1)
    n = 16;
  cudaGetLastError();
  clear_error();
  most[dev].store(n, std::memory_order_relaxed);
  return n;
}
// Blocks of the cluster that sorts `total` choices: a choice per thread up to
// 16 (32768 choices: 1 block 66 us, 8 blocks 8.8 us, 16 blocks 7.1 us; 128
// choices: 1 block 3.8 us, 16 blocks 4.4 us).  The plan is the same for any.
unsigned plan_blocks(int dev, int64_t total) {
  unsigned b = 1;
  while (b < 8 && total > static_cast<int64_t>(b) * kPlanThreads) b *= 2;
  return total > 8 * kPlanThreads ? plan_cluster(dev) : b;
}

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
  const unsigned blocks = plan_blocks(dev, total);
  const int64_t warps = static_cast<int64_t>(blocks) * kPlanWarps;
  p.per = static_cast<uint32_t>(per);
  p.total = static_cast<uint32_t>(total);
  p.piece = static_cast<uint32_t>(((total + warps - 1) / warps + 31) / 32 * 32);
  p.experts = nexperts;
  p.each = static_cast<int>(each);
  while (nexperts - 1 >> p.bits) ++p.bits;
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
  if (rc == VC_SUCCESS && hidden > static_cast<size_t>(kMaxInt)) return fail(VC_ERR_INVALID_ARG, "hidden above 2^31 - 1");
  return rc;
}
// Blocks for `tiles` tiles of one warp: all of them, or as many as are resident.
template <auto K>
unsigned move_blocks(DeviceState* st, int dev, int64_t tiles) {
  const int64_t want = (tiles + kMoveWarps - 1) / kMoveWarps;
  return static_cast<unsigned>(std::min<int64_t>(want, int64_t(st->nsm) * resident_blocks<K>(dev, kMoveThreads, 0)));
}

template <class U>
vc_status_t launch_dispatch(DeviceState* st, int dev, DispatchParams& p, int64_t row, int64_t bytes, cudaStream_t s) {
  constexpr int64_t kPiece = 32 * kUnitsOf<U>;
  p.n = row / static_cast<int64_t>(sizeof(U));
  p.pieces = static_cast<uint32_t>(std::max<int64_t>(1, (p.n + kPiece - 1) / kPiece));  // one of no units moves its token's scale
  p.tiles *= p.pieces;
  return launch<dispatch_kernel<U>>(dev, Shape{move_blocks<dispatch_kernel<U>>(st, dev, p.tiles), kMoveThreads}, s, p, kDispatch, 0,
                                    bytes);
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
  if (rc != VC_SUCCESS || rows == 0 || (hidden == 0 && !scale)) return rc;
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
  if (whole && row >= kBulkMinRow && topk >= kBulkMinChoices && n * nranks * topk * row >= kBulkMinBytes) {
    p.n = row;
    p.pieces = static_cast<uint32_t>((row + kBulkBytes - 1) / kBulkBytes);
    p.piece_bytes = static_cast<uint32_t>((row / 16 + p.pieces - 1) / p.pieces) * 16;
    p.tiles *= p.pieces;
    const int64_t fit = int64_t(st->nsm) * resident_blocks<dispatch_bulk_kernel>(dev, kBulkWarps * 32, kBulkSmem);
    const Shape shape{static_cast<unsigned>(std::min<int64_t>((p.tiles + kBulkWarps - 1) / kBulkWarps, fit)), kBulkWarps * 32, kBulkSmem};
    return launch<dispatch_bulk_kernel>(dev, shape, stream, p, kDispatch, 0, bytes);
  }
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
      constexpr int64_t kPiece = 32 * kUnits;
      p.n = static_cast<int64_t>(hidden);
      p.pieces = static_cast<uint32_t>((units_of(p.n, es) + kPiece - 1) / kPiece);
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
      p.n = static_cast<int64_t>(hidden);
      const int64_t units = units_of(p.n, es);
      const unsigned threads = static_cast<unsigned>(std::max<int64_t>(32, std::min<int64_t>(kMoveThreads, (units + 31) / 32 * 32)));
      return launch<combine_grad_kernel<DT, VEC>>(dev, Shape{p.s.rows, threads, 0, 1, static_cast<unsigned>(nranks)}, stream, p,
                                                  kCombineBackward, 0, bytes);
    };
    return whole ? go(std::true_type{}) : go(std::false_type{});
  });
}

}  // namespace

cudaError_t take_exchange_errors(cudaStream_t stream, uint32_t* flags) {
  static const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(flags, dev::g_device_error, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(dev::g_device_error, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  return e;
}

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
