// The products of an expert-parallel layer: the rows that each rank's experts
// have received with the experts' weights, and their gradients (see vc.h).
//
// How many rows an expert has is known on the device alone, so every kernel
// here makes its list of tiles from the offsets and walks it with as many
// blocks as the GPU holds.  On a GB300 (copy rate 6.78 TB/s, library products of
// 8192 x 8192 x 8192 bf16 at 1.90 PFLOP/s in bursts, 1.70 under the power limit):
//   64 experts of 4096 by 2048, bf16, 128 rows in all     136 us, 6.9 TB/s
//   the same, 32768 rows                                  356 us, 1.54 PFLOP/s
//                                    (400 us under the power limit, 1.37)
//   8-bit, 128 rows                                        73 us, 6.4 TB/s
//   8-bit, 32768 rows                                     291 us, 1.89 PFLOP/s
//   32 experts of 2048 by 4096, 16384 rows, both gradients 406 us, 1.35 PFLOP/s
//                          (the weights' part 228 us; to fp32 277)
//   one expert, 8192 x 8192 x 8192: 615 us bf16 (1.79), 470 us 8-bit (2.34)
#include "tc.cuh"

namespace vc {
namespace layer {
namespace {

using tc::Rows;

constexpr int kMaxExperts = VC_ROUTE_MAX_EXPERTS;
constexpr size_t kMaxCapacity = 0x7fff0000;  // a tile past the last row still has int32 rows

// ---------------------------------------------------------------------------
// products in fp32
// ---------------------------------------------------------------------------
// out(n, m) = sum over k of b(n, k) * a(m, k) in tiles of 64 n by 128 m, 16 of
// k at a time; 256 threads with 4 n by 8 m each: 32 products for 48 bytes from
// shared memory (16 experts of 4096 by 2048: 16384 rows in all 9.1 ms, 30
// TFLOP/s; 8192 rows 4.8 ms, 29).  (The tensor cores have no fp32 products;
// splitting each factor in three bf16 parts would take six of theirs and three
// times the bytes.)
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

// One operand's 16 by W tile of k by m (or n) to shared memory.
// Neighbouring threads take neighbouring elements in memory.
template <int W>
struct SimpleTile {
  static constexpr int kEach = kSimpleK * W / kSimpleThreads;
  float v[kEach];
  static __device__ __forceinline__ void place(int i, bool k_runs, int* k, int* w) {
    const int at = i * kSimpleThreads + threadIdx.x;
    *k = k_runs ? at % kSimpleK : at / W;
    *w = k_runs ? at / kSimpleK : at % W;
  }
  __device__ __forceinline__ void load(const float* p, int64_t sw, int64_t sk, int ws, int ks) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      int k, w;
      place(i, sk == 1, &k, &w);
      v[i] = w < ws && k < ks ? __ldg(p + w * sw + k * sk) : 0.f;
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

template <bool WEIGHT>
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
    const float* a = static_cast<const float*>(p.a[d]) + (WEIGHT ? r.first * p.ak : i * p.ae) + m0 * p.am;
    const float* b = static_cast<const float*>(p.b[d]) + r.first * (WEIGHT ? p.bk : p.bn) + n0 * p.bn;
    const bool ka = p.ak == 1, kb = p.bk == 1;
    float acc[4][8] = {};
    SimpleTile<kSimpleM> ta;
    SimpleTile<kSimpleN> tb;
    const int steps = (K + kSimpleK - 1) / kSimpleK;
    __syncthreads();  // the last tile's products have read shared memory
    for (int s = 0; s <= steps; ++s) {
      if (s < steps) {
        const int k0 = s * kSimpleK;
        ta.load(a + static_cast<int64_t>(k0) * p.ak, p.am, p.ak, ms, K - k0);
        tb.load(b + static_cast<int64_t>(k0) * p.bk, p.bn, p.bk, ns, K - k0);
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
    float* out = static_cast<float*>(p.out[d]);
    const int64_t row = WEIGHT ? static_cast<int64_t>(i) * p.N + n0 : static_cast<int64_t>(r.first) + n0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = ty * 4 + j;
      if (n >= ns) continue;
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        const int m = (l / 4) * 64 + tx * 4 + l % 4;
        if (m < ms) out[(row + n) * p.M + m0 + m] = acc[j][l];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// products on the tensor cores
// ---------------------------------------------------------------------------
// A pair of blocks works a tile of 256 of m (the weights' side, or the
// contiguous side of a weights' gradient) by up to 256 of n (rows of one expert,
// or the other side), each block with 128 of m and the fp32 sums of those in its
// tensor memory.  The rows stand on the n side because n may be any multiple of
// 16: an expert's last rows cost what they are, where the m side would fill up.
// Each block loads its half of m and half of n, 64 of k a step; a pair's
// products read both halves of n, so that each block's shared memory takes two
// thirds of what a block by itself would load and read (prefill of 32768 rows,
// 4096 by 2048: 587 us with single blocks of 128 by 256).
//   warp 0: one thread loads each step's tiles by tensor maps
//   warp 1: one thread of the pair's first block issues the products
//   warp 2: rows behind an expert's last, in the last step of a weights' gradient
//   warps 4 to 7: tensor memory to global memory, while the next tile's
//     products go to the other half of tensor memory
constexpr int kTileM = 128, kTileN = 256, kTileK = 64;
constexpr int kTcThreads = 256, kMaxStages = 12;
constexpr int kTileBytesA = kTileM * kTileK * 2;
constexpr int kRoomBytes = 2 * 32 * kTileM * 2;
constexpr uint32_t kColumns = 512;  // two accumulators
constexpr size_t kTcSmem = 220 << 10;

constexpr int kRowBox = 32;  // rows of one load
template <int R>
struct ProductParams {
  CUtensorMap a[R], b[R];
  void* out[R];
  const int32_t* offsets[R];
  int32_t capacity;
  int M, N, K;  // as SimpleParams
  int experts, each;
  bool whole;     // out's rows are whole 16 bytes on 16-byte boundaries, of 16-bit elements
};

struct Tile {
  int d, i;        // rank, its expert
  int32_t first;   // its first row (of weights' gradients: of k)
  int64_t row;     // of out
  int n0, n, m0;   // m0: of this block's half
  int half;        // of n, padded: what each block loads
  int k;           // elements
};
template <bool WEIGHT, class P>
__device__ __forceinline__ Tile tile_at(const P& p, const uint32_t* ends, uint32_t t, int rank, int& e) {
  Tile x;
  const uint32_t across = (p.M + 2 * kTileM - 1) / (2 * kTileM);
  uint32_t at = t;
  if constexpr (WEIGHT) {
    const uint32_t every = across * tc::pieces(p.N, kTileN);
    e = t / every;
    at -= e * every;
  } else {
    while (ends[e] <= t) ++e;
    if (e) at -= ends[e - 1];
  }
  x.d = e / p.each;
  x.i = e % p.each;
  const Rows r = tc::rows_of(p.offsets[x.d], x.i, p.capacity);
  const int count = WEIGHT ? p.N : r.count, piece = tc::piece_of(count, kTileN, 16);
  x.n0 = static_cast<int>(at / across) * piece;
  x.n = min(piece, count - x.n0);
  x.m0 = static_cast<int>(at % across) * (2 * kTileM) + rank * kTileM;
  x.half = (x.n + 15) / 16 * 8;
  x.first = WEIGHT ? r.first : r.first + x.n0;
  x.row = WEIGHT ? static_cast<int64_t>(x.i) * p.N + x.n0 : x.first;
  x.k = WEIGHT ? r.count : p.K;
  return x;
}

// 32 accumulated columns of a warp (lane: m) to `columns` rows of out, lane 0's
// first element at `at`.
template <int OUT>
__device__ __forceinline__ void store_columns(const uint32_t (&v)[32], char* at, int64_t pitch, int columns, bool there) {
  char* to = at + (threadIdx.x & 31) * El<OUT>::kSize;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (j >= columns) break;
    if (there) El<OUT>::store(to, 0, __uint_as_float(v[j]));
    to += pitch;
  }
}
// The same of four warps' 128 m in 16-byte stores of out's rows, through
// `room` (16 pairs of rows by 128 m; callers alternate two).  A warp by itself
// would write 64 bytes of a row at a time, two bytes a lane: the weights'
// gradients of 32 experts with 512 rows each, 2048 by 4096, 8 steps a tile, took
// 352 us that way.
template <bool F16>
__device__ __forceinline__ void store_rows(const uint32_t (&v)[32], uint32_t room, char* at, int64_t pitch, int columns, int ms) {
  const int thread = threadIdx.x & 127;
#pragma unroll
  for (int j = 0; j < 32; j += 2)
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(room + j * 256 + thread * 4), "r"(dev::pack2<F16>(__uint_as_float(v[j]), __uint_as_float(v[j + 1])))
                 : "memory");
  asm volatile("bar.sync 1, 128;" ::: "memory");
  const int m = thread % 16 * 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = (thread / 16 + i * 8) * 2;
    uint32_t x[8];
#pragma unroll
    for (int h = 0; h < 8; h += 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x[h]), "=r"(x[h + 1]), "=r"(x[h + 2]), "=r"(x[h + 3])
                   : "r"(room + j * 256 + (m + h) * 4)
                   : "memory");
    if (m < ms) {
      char* to = at + j * pitch + m * 2;
      if (j < columns)
        *reinterpret_cast<uint4*>(to) = make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                                                   __byte_perm(x[4], x[5], 0x5410), __byte_perm(x[6], x[7], 0x5410));
      if (j + 1 < columns)
        *reinterpret_cast<uint4*>(to + pitch) = make_uint4(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632),
                                                           __byte_perm(x[4], x[5], 0x7632), __byte_perm(x[6], x[7], 0x7632));
    }
  }
}

// AMN: M runs along the rows of a's tiles (weights in by out; weights'
// gradients).  OUT: out's type, of the operands or fp32.
template <int DT, int OUT, bool AMN, bool WEIGHT, int R>
__global__ void __launch_bounds__(kTcThreads, 1) product_kernel(const __grid_constant__ ProductParams<R> p) {
  extern __shared__ unsigned char dynamic[];
  __shared__ uint32_t ends[WEIGHT ? 1 : kMaxExperts];
  __shared__ __align__(8) uint64_t bars[3 * kMaxStages + 5];
  __shared__ uint32_t columns, gone;
  __shared__ int longest;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = static_cast<int>(tc::rank_in_cluster());
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kMaxStages, tail = empty + 8 * kMaxStages,
                 sums_full = tail + 8 * kMaxStages, sums_empty = sums_full + 16, done = sums_empty + 16;
  const uint32_t full0 = tc::bar_of(full, 0), sums_empty0 = tc::bar_of(sums_empty, 0);  // the first block's
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) tc::bar_init(full + 8 * s, 2), tc::bar_init(empty + 8 * s, 1), tc::bar_init(tail + 8 * s, 1);
    for (int s = 0; s < 2; ++s) tc::bar_init(sums_full + 8 * s, 1), tc::bar_init(sums_empty + 8 * s, 8);
    tc::bar_init(done, 1);
    gone = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  tc::cluster_sync();  // both blocks and their barriers are there
  if (warp == 1) tc::take_columns<true>(tc::smem_addr(&columns), kColumns);
  stream_order();
  const uint32_t across = (p.M + 2 * kTileM - 1) / (2 * kTileM);
  if constexpr (!WEIGHT) {
    if (warp == 0) tc::list_tiles(p.offsets, p.experts, p.each, p.capacity, kTileN, across, ends, &longest);
  }
  // This block's list and columns; the products wait for the other block's loads,
  // which come after its own barrier here.
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  const uint32_t total = WEIGHT ? p.experts * across * tc::pieces(p.N, kTileN) : ends[p.experts - 1];
  // Stages as small as the longest piece of n allows: few rows, many stages.
  // Above kTileN rows an expert with fewer may have the longer pieces.
  const int widest = WEIGHT ? tc::piece_of(p.N, kTileN, 16) : min(kTileN, (longest + 15) / 16 * 16);
  const uint32_t stage_bytes = kTileBytesA + (WEIGHT ? (widest / 2 + 63) / 64 * 8192 : (widest / 2 + kRowBox - 1) / kRowBox * 128 * kRowBox);
  const uint32_t room = (tc::smem_addr(dynamic) + 1023) & ~1023u, tiles = room + kRoomBytes;  // of the stores; stages
  const int stages = min(kMaxStages, static_cast<int>((kTcSmem - 1024 - kRoomBytes) / stage_bytes));
  const uint32_t sums = columns, pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (warp == 0) {
    if (tc::elect()) {
      int e = 0, s = 0;
      uint32_t phase = 0, issued = 0, tails = 0, tail_phases = 0;
      bool ok = true;
      for (uint32_t t = pair; ok && t < total; t += pairs) {
        const Tile x = tile_at<WEIGHT>(p, ends, t, rank, e);
        const int boxes = WEIGHT ? (x.half + 63) / 64 : (x.half + kRowBox - 1) / kRowBox;
        const uint32_t bytes = kTileBytesA + boxes * (WEIGHT ? 8192 : 128 * kRowBox);
        const CUtensorMap *a = p.a + x.d, *b = p.b + x.d;
        for (int k = 0; k < x.k; k += kTileK) {
          if (!tc::bar_wait(empty + 8 * s, phase ^ 1, &gone)) {
            ok = false;
            break;
          }
          const uint32_t to = tiles + s * stage_bytes, bar = full0 + 8 * s;
          if constexpr (WEIGHT) {
            const int n0 = x.n0 + rank * x.half;
            if (x.k - k < kTileK && (x.k - k) % 16 != 0) {  // warp 2 has a word to say first
              const uint32_t here = tail + 8 * s;
              tails |= 1u << s;
              tail_phases ^= 1u << s;
              tc::bar_expect(here, bytes);
              tc::load2d(to, a, here, x.m0, x.first + k);
              tc::load2d(to + 8192, a, here, x.m0 + 64, x.first + k);
              for (int j = 0; j < boxes; ++j) tc::load2d(to + kTileBytesA + j * 8192, b, here, n0 + j * 64, x.first + k);
            } else {
              tails &= ~(1u << s);
              tc::bar_expect_there(bar, bytes);
              tc::load2d_pair(to, a, bar, x.m0, x.first + k);
              tc::load2d_pair(to + 8192, a, bar, x.m0 + 64, x.first + k);
              for (int j = 0; j < boxes; ++j) tc::load2d_pair(to + kTileBytesA + j * 8192, b, bar, n0 + j * 64, x.first + k);
            }
          } else {
            tc::bar_expect_there(bar, bytes);
            if constexpr (AMN) {
              tc::load3d_pair(to, a, bar, x.m0, k, x.i);
              tc::load3d_pair(to + 8192, a, bar, x.m0 + 64, k, x.i);
            } else {
              tc::load3d_pair(to, a, bar, k, x.m0, x.i);
            }
            for (int j = 0; j < boxes; ++j) tc::load2d_pair(to + kTileBytesA + j * (128 * kRowBox), b, bar, k, x.first + rank * x.half + j * kRowBox);
          }
          ++issued;
          if (++s == stages) s = 0, phase ^= 1;
        }
      }
      // The pair ends after its last loads and products, on whatever path: the
      // first block's barriers know of both blocks' loads.
      for (int j = 0; j < stages && issued > static_cast<uint32_t>(j); ++j) {
        if (s-- == 0) s = stages - 1, phase ^= 1;
        const bool alone = tails >> s & 1;
        if (ok) ok = tc::bar_wait(empty + 8 * s, phase, &gone);
        if (!ok && (rank == 0 || alone)) {
          const uint32_t bar = alone ? tail + 8 * s : full + 8 * s, parity = alone ? ~tail_phases >> s & 1 : phase;
          for (uint32_t it = 0; it < tc::kSoon && !tc::bar_test(bar, parity); ++it) __nanosleep(64);
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    if (tc::elect()) {
      int e = 0, s = 0, half = 0;
      uint32_t phase = 0, half_phase = 0;
      bool ok = true;
      const uint64_t a0 = AMN ? tc::desc_mn(tiles, 8192) : tc::desc_k(tiles);
      const uint64_t b0 = WEIGHT ? tc::desc_mn(tiles + kTileBytesA, 8192) : tc::desc_k(tiles + kTileBytesA);
      constexpr uint32_t kNextA = (AMN ? 2048 : 32) / 16, kNextB = (WEIGHT ? 2048 : 32) / 16;  // 16 of k on
      for (uint32_t t = pair; ok && t < total; t += pairs) {
        const Tile x = tile_at<WEIGHT>(p, ends, t, rank, e);
        if (!tc::bar_wait(sums_empty + 8 * half, half_phase ^ 1, &gone)) break;
        tc::after_sync();
        const uint32_t to = sums + half * kTileN;
        const uint32_t how = tc::instruction(DT == VC_BFLOAT16, AMN, WEIGHT, 2 * x.half, 2 * kTileM);
        for (int k = 0; k < x.k; k += kTileK) {
          const int left = x.k - k;
          // Rows that a warp of each block has set to 0: the other block's write
          // is this block's to read at the cluster's scope only.  (Both gradients of
          // 32 experts of 2048 by 4096, 16384 rows, take 406 us so and took 392
          // with the default scope; with this one in every step the forward
          // product took three times as long.)
          const bool zeroed = WEIGHT && left < kTileK && left % 16 != 0;
          if (!(zeroed ? tc::bar_wait<true>(full + 8 * s, phase, &gone) : tc::bar_wait(full + 8 * s, phase, &gone))) {
            ok = false;
            break;
          }
          tc::after_sync();
          const uint64_t a = a0 + (s * stage_bytes >> 4), b = b0 + (s * stage_bytes >> 4);
#pragma unroll
          for (int j = 0; j < kTileK / 16; ++j)
            if (j * 16 < left) tc::mma16_pair(to, a + j * kNextA, b + j * kNextB, how, k + j > 0);
          tc::commit_pair(empty + 8 * s);
          if (++s == stages) s = 0, phase ^= 1;
        }
        if (ok) tc::commit_pair(sums_full + 8 * half);
        if (half ^= 1; half == 0) half_phase ^= 1;
      }
      if (gone) {  // products in flight end before tensor memory is freed
        tc::commit_pair(done);
        for (uint32_t it = 0; it < tc::kSoon && !tc::bar_test(done, 0); ++it) __nanosleep(64);
      }
    }
  } else if (WEIGHT && warp == 2) {
    // The last step's rows behind the expert's last, up to 16, are not its own:
    // 0 instead, on both sides (either may be NaN).
    int e = 0;
    uint32_t step = 0, phases = 0;  // of the stages; of each stage's barrier
    for (uint32_t t = pair; t < total; t += pairs) {
      const Tile x = tile_at<WEIGHT>(p, ends, t, rank, e);
      const uint32_t steps = (static_cast<uint32_t>(x.k) + kTileK - 1) / kTileK;
      const int left = x.k % kTileK;
      step = (step + steps % stages) % stages;
      if (left % 16 == 0) continue;
      const int s = static_cast<int>(step == 0 ? stages - 1 : step - 1);
      if (!tc::warp_wait(tail + 8 * s, phases >> s & 1, &gone, tc::kLate)) break;
      phases ^= 1u << s;
      const int n = (16 - left % 16) * 8, boxes = 2 + (x.half + 63) / 64;
      for (int j = lane; j < n * boxes; j += 32)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tiles + s * stage_bytes + j / n * 8192 + left * 128 + j % n * 16),
                     "r"(0)
                     : "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tc::bar_release_there(full0 + 8 * s);
    }
  } else if (warp >= 4) {
    int e = 0, half = 0, turn = 0;
    uint32_t half_phase = 0;
    const int part = warp & 3;  // the lanes of tensor memory that this warp reaches
    constexpr int es = El<OUT>::kSize;
    const int64_t pitch = static_cast<int64_t>(p.M) * es;
    for (uint32_t t = pair; t < total; t += pairs) {
      const Tile x = tile_at<WEIGHT>(p, ends, t, rank, e);
      const bool ok = tc::warp_wait(sums_full + 8 * half, half_phase, &gone, tc::kLate);
      // the four warps meet below, and give up together
      int all;
      asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 2, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                   : "=r"(all)
                   : "r"(static_cast<int>(ok))
                   : "memory");
      if (!all) break;
      tc::after_sync();
      char* out = static_cast<char*>(p.out[x.d]) + x.row * pitch + static_cast<int64_t>(x.m0) * es;
      const uint32_t from = sums + (part << 21) + half * kTileN;
      const int ms = p.M - x.m0;
      // Columns 32 at a time, the next ones on their way from tensor memory.
      const auto take = [&](uint32_t(&now)[32], uint32_t(&next)[32], int c) {
        const int columns = x.n - c;
        if (x.k > 0) {
          tc::loaded(now);
          if (columns > 32) tc::load_columns(from + c + 32, next);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) now[j] = 0;
        }
        if (columns <= 32) {
          tc::before_sync();
          __syncwarp();
          if (lane == 0) tc::bar_arrive_there(sums_empty0 + 8 * half);
        }
        if (OUT != VC_FLOAT32 && p.whole)
          store_rows<OUT == VC_FLOAT16>(now, room + (turn ^= 1) * (32 * kTileM * 2), out + c * pitch, pitch, columns, ms);
        else
          store_columns<OUT>(now, out + c * pitch + static_cast<int64_t>(part * 32) * es, pitch, columns, part * 32 + lane < ms);
      };
      uint32_t v[32], w[32];
      if (x.k > 0) tc::load_columns(from, v);
      for (int c = 0; c < x.n; c += 64) {
        take(v, w, c);
        if (c + 32 < x.n) take(w, v, c + 32);
      }
      if (half ^= 1; half == 0) half_phase ^= 1;
    }
  }
  tc::before_sync();
  __syncwarp();
  tc::cluster_sync();  // neither block ends while the other may reach it
  tc::after_sync();
  if (warp == 1) {
    tc::take_no_more<true>();
    tc::free_columns<true>(sums, kColumns);
  }
  __syncwarp();
  tc::cluster_sync();
  if (gone && threadIdx.x == 0) atomicOr(&dev::g_device_error, 4u);
}

// ---------------------------------------------------------------------------
// products of 8-bit operands
// ---------------------------------------------------------------------------
// out(row, o) = sum over blocks b of 128 k of s(row, b) * w(o / 128, b) * (the
// block's products, summed in tensor memory).  Each block's sums go to one of
// two accumulators in turn; eight warps take them from there, scaled, into
// registers, while the products of the next block go to the other one.  The
// rows stand on the m side here, so that a thread has one row's scale, in a
// register.  (With rows on the n side it would take its columns' scales from
// shared memory, four to a read; that was not measured.)
//   warp 0 loads, warp 1 issues the products, warps 4 to 11 scale and store;
// these hold 128 sums a thread and take the registers that the first four warps
// give up (launched with 168 each: 4 x 40 + 8 x 232 = 12 x 168).
constexpr int kTile8N = 256, kTile8K = 128;
constexpr int kTc8Threads = 384, kTc8Warps = 8;
constexpr int kRoom8Bytes = kTc8Warps * 32 * 64;

template <int R>
struct Product8Params {
  CUtensorMap rows[R], weight[R];
  const float* row_scale[R];
  const float* weight_scale[R];
  void* out[R];
  const int32_t* offsets[R];
  int32_t capacity;
  int M, K;       // outputs, inputs
  int experts, each;
  bool whole;     // out's rows are whole 16 bytes on 16-byte boundaries
};

struct Tile8 {
  int d, i;
  int32_t first;  // row
  int n, m0;      // rows, first output
};
template <class P>
__device__ __forceinline__ Tile8 tile8_at(const P& p, const uint32_t* ends, uint32_t t, int& e) {
  Tile8 x;
  while (ends[e] <= t) ++e;
  const uint32_t at = e ? t - ends[e - 1] : t, across = (p.M + kTile8N - 1) / kTile8N;
  x.d = e / p.each;
  x.i = e % p.each;
  const Rows r = tc::rows_of(p.offsets[x.d], x.i, p.capacity);
  const int n0 = static_cast<int>(at / across) * kTileM;
  x.n = min(kTileM, r.count - n0);
  x.first = r.first + n0;
  x.m0 = static_cast<int>(at % across) * kTile8N;
  return x;
}

// A thread's 128 sums of one row to out in whole 16 bytes, 64 bytes of a row at a
// time through the warp's `room`, so that a store is eight rows' 64 bytes (16
// bytes a lane and row took 12% of a product of 8192 by 8192 by 8192; a room of
// 128 bytes a row would take the fourth stage's place).
template <int OUT>
__device__ __forceinline__ void store_sums(const float (&acc)[128], uint32_t room, char* out, int64_t pitch, int rows, int left) {
  using E = El<OUT>;
  constexpr int kEach = 64 / E::kSize;  // elements of 64 bytes
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 128; c += kEach) {
    if (c >= left) break;
    __syncwarp();  // the last ones have been read
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 x = E::narrow(acc + c + j * E::kVec);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(room + lane * 64 + ((j ^ lane >> 1) & 3) * 16), "r"(x.x), "r"(x.y),
                   "r"(x.z), "r"(x.w)
                   : "memory");
    }
    __syncwarp();
    const int j = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + lane / 4;
      uint4 x;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                   : "r"(room + r * 64 + ((j ^ r >> 1) & 3) * 16)
                   : "memory");
      if (r < rows && c + j * E::kVec < left) *reinterpret_cast<uint4*>(out + r * pitch + c * E::kSize + j * 16) = x;
    }
  }
}

// A tile is 128 rows by 256 outputs.  (Pairs of blocks with 256 rows, each
// loading half of the weights, measured 321 us against 310 at the prefill of
// 32768 rows, 4096 by 2048, and 103 against 74 with a few rows an expert: a
// pair's products take as long for 32 rows as for 256.  That was before the sums
// were taken 16 at a time, which brought the 310 to 291.)
template <int OUT, int R>
__global__ void __launch_bounds__(kTc8Threads, 1) product8_kernel(const __grid_constant__ Product8Params<R> p) {
  extern __shared__ unsigned char dynamic[];
  __shared__ uint32_t ends[kMaxExperts];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
  __shared__ uint32_t columns, gone;
  __shared__ int longest;
  constexpr uint32_t kWeightBytes = kTile8N * kTile8K;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kMaxStages, sums_full = empty + 8 * kMaxStages,
                 sums_empty = sums_full + 16, done = sums_empty + 16;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) tc::bar_init(full + 8 * s, 1), tc::bar_init(empty + 8 * s, 1);
    for (int s = 0; s < 2; ++s) tc::bar_init(sums_full + 8 * s, 1), tc::bar_init(sums_empty + 8 * s, kTc8Warps);
    tc::bar_init(done, 1);
    gone = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tc::take_columns<false>(tc::smem_addr(&columns), kColumns);
  stream_order();
  if (warp == 0)
    tc::list_tiles(p.offsets, p.experts, p.each, p.capacity, kTileM, (p.M + kTile8N - 1) / kTile8N, ends, &longest);
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  const uint32_t total = ends[p.experts - 1];
  const uint32_t row_bytes = (min(kTileM, longest) + 31) / 32 * 4096, stage_bytes = kWeightBytes + row_bytes;
  const uint32_t room = (tc::smem_addr(dynamic) + 1023) & ~1023u, tiles = room + kRoom8Bytes;
  // The products read 128 rows whatever was loaded: past the last stage's there
  // is room for them.  What they make of the others is not looked at.
  const int stages = min(kMaxStages, static_cast<int>((kTcSmem - 1024 - kRoom8Bytes - (kTileM * kTile8K - row_bytes)) / stage_bytes));
  const uint32_t sums = columns;
  const int blocks = (p.K + kTile8K - 1) / kTile8K;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      if (tc::elect()) {
        int e = 0, s = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true;
        for (uint32_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
          const Tile8 x = tile8_at(p, ends, t, e);
          const int boxes = (x.n + 31) / 32;
          const CUtensorMap *rows = p.rows + x.d, *weight = p.weight + x.d;
          for (int k = 0; k < blocks; ++k) {
            if (!tc::bar_wait(empty + 8 * s, phase ^ 1, &gone)) {
              ok = false;
              break;
            }
            const uint32_t to = tiles + s * stage_bytes;
            const uint32_t bar = full + 8 * s;
            tc::bar_expect(bar, kWeightBytes + boxes * 4096);
            tc::load3d(to, weight, bar, k * kTile8K, x.m0, x.i);
            for (int j = 0; j < boxes; ++j) tc::load2d(to + kWeightBytes + j * 4096, rows, bar, k * kTile8K, x.first + j * 32);
            ++issued;
            if (++s == stages) s = 0, phase ^= 1;
          }
        }
        for (int j = 0; j < stages && issued > static_cast<uint32_t>(j); ++j) {  // as in product_kernel
          if (s-- == 0) s = stages - 1, phase ^= 1;
          if (ok) ok = tc::bar_wait(empty + 8 * s, phase, &gone);
          if (!ok)
            for (uint32_t it = 0; it < tc::kSoon && !tc::bar_test(full + 8 * s, phase); ++it) __nanosleep(64);
        }
      }
    } else if (warp == 1) {
      if (tc::elect()) {
        int e = 0, s = 0, half = 0;
        uint32_t phase = 0, half_phase = 0;
        bool ok = true;
        const uint64_t b0 = tc::desc_k(tiles), a0 = tc::desc_k(tiles + kWeightBytes);
        for (uint32_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
          const Tile8 x = tile8_at(p, ends, t, e);
          const uint32_t how = tc::instruction(0, false, false, (min(kTile8N, p.M - x.m0) + 15) / 16 * 16, kTileM);
          for (int k = 0; k < blocks; ++k) {
            ok = tc::bar_wait(sums_empty + 8 * half, half_phase ^ 1, &gone) && tc::bar_wait(full + 8 * s, phase, &gone);
            if (!ok) break;
            tc::after_sync();
            const uint64_t a = a0 + (s * stage_bytes >> 4), b = b0 + (s * stage_bytes >> 4);
            const int left = p.K - k * kTile8K;
#pragma unroll
            for (int j = 0; j < kTile8K / 32; ++j)
              if (j * 32 < left) tc::mma8(sums + half * kTile8N, a + j * 2, b + j * 2, how, j > 0);
            tc::commit(empty + 8 * s);
            tc::commit(sums_full + 8 * half);
            if (++s == stages) s = 0, phase ^= 1;
            if (half ^= 1; half == 0) half_phase ^= 1;
          }
        }
        if (gone) {
          tc::commit(done);
          for (uint32_t it = 0; it < tc::kSoon && !tc::bar_test(done, 0); ++it) __nanosleep(64);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    int e = 0, half = 0;
    uint32_t half_phase = 0;
    bool ok = true;
    const int part = warp & 3, side = (warp - 4) / 4;  // lanes of tensor memory; which 128 of the 256 outputs
    const int64_t down = (p.M + VC_FP8_BLOCK - 1) / VC_FP8_BLOCK, pitch = static_cast<int64_t>(p.M) * El<OUT>::kSize;
    for (uint32_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile8 x = tile8_at(p, ends, t, e);
      const int m = x.m0 + side * 128, row = part * 32 + lane;
      const bool busy = m < p.M && part * 32 < x.n, there = row < x.n;
      const float* rs = p.row_scale[x.d] + (there ? (static_cast<int64_t>(x.first) + row) * blocks : 0);
      const float* ws = p.weight_scale[x.d] + (x.i * down + (m < p.M ? m / VC_FP8_BLOCK : 0)) * blocks;
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.f;
      float sr = blocks > 0 && there ? __ldg(rs) : 0.f, sw = blocks > 0 ? __ldg(ws) : 0.f;
      for (int k = 0; k < blocks; ++k) {
        const float by = sr * sw;
        if (k + 1 < blocks) {
          sr = there ? __ldg(rs + k + 1) : 0.f;
          sw = __ldg(ws + k + 1);
        }
        ok = tc::warp_wait(sums_full + 8 * half, half_phase, &gone, tc::kLate);
        if (!ok) break;
        if (busy) {
          tc::after_sync();
          const uint32_t from = sums + (part << 21) + half * kTile8N + side * 128;
          uint32_t v[2][16];  // 16 sums at a time, the next ones on their way: 32 do not fit with the 128
          tc::load_columns(from, v[0]);
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            tc::loaded(v[c / 16 & 1]);
            if (c < 112) tc::load_columns(from + c + 16, v[~(c / 16) & 1]);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(__uint_as_float(v[c / 16 & 1][j]), by, acc[c + j]);
          }
          tc::before_sync();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(sums_empty + 8 * half);
        } else if (lane == 0) {
          tc::bar_arrive(sums_empty + 8 * half);
        }
        if (half ^= 1; half == 0) half_phase ^= 1;
      }
      if (!ok || !busy) continue;
      char* out = static_cast<char*>(p.out[x.d]) + (static_cast<int64_t>(x.first) + part * 32) * pitch + static_cast<int64_t>(m) * El<OUT>::kSize;
      const int left = min(128, p.M - m);
      if (p.whole) {
        store_sums<OUT>(acc, room + (warp - 4) * (32 * 64), out, pitch, x.n - part * 32, left);
      } else if (there) {
#pragma unroll
        for (int j = 0; j < 128; ++j)
          if (j < left) El<OUT>::store(out + lane * pitch, j, acc[j]);
      }
    }
  }
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  if (warp == 1) {
    tc::take_no_more<false>();
    tc::free_columns<false>(sums, kColumns);
  }
  if (gone && threadIdx.x == 0) atomicOr(&dev::g_device_error, 4u);
}

// -- a drill of the products' waits ------------------------------------------------
// As in the products, with nothing in flight: one thread waits for what never
// comes and gives up, which ends the wait of a whole warp; a wait for what has
// come goes on.  kDrill polls are less than a millisecond.
constexpr uint32_t kDrill = 1u << 12;
__global__ void __launch_bounds__(96) wait_drill_kernel() {
  __shared__ __align__(8) uint64_t bars[3];
  __shared__ uint32_t gone;
  const uint32_t never = tc::smem_addr(bars), late = never + 8, there = late + 8;
  const int warp = threadIdx.x / 32;
  stream_order();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) tc::bar_init(never + 8 * i, 1);
    gone = 0;
    tc::bar_arrive(there);
  }
  __syncthreads();
  bool as_it_should = true;
  if (warp == 0) {
    if (tc::elect()) as_it_should = !tc::bar_wait(never, 0, &gone, kDrill) && gone;
  } else if (warp == 1) {
    as_it_should = !tc::warp_wait(late, 0, &gone);
  } else {
    as_it_should = tc::warp_wait(there, 0, &gone) && tc::bar_wait<true>(there, 0, &gone);
  }
  if (__syncthreads_and(as_it_should) && gone && threadIdx.x == 0) atomicOr(&dev::g_device_error, 4u);
}

// -- operands off 16-byte boundaries --------------------------------------------
// Tensor maps want them, so such rows are copied to scratch first, a row each
// 16 bytes' multiple apart: the rows that the experts have, the weights of
// experts that have rows.
struct PadRows {
  const void* from[VC_MAX_RANKS];
  char* to;
  int64_t rows;   // of each rank
  int64_t group;  // rows of each expert's weights; 0: the experts' rows
  int width;      // elements
  int units;      // of 16 bytes that a row takes
};
struct PadParams {
  PadRows op[3];
  const int32_t* offsets[VC_MAX_RANKS];
  int32_t capacity;
  int ranks, each;
};
constexpr int kPadThreads = 256, kPadAhead = 4;

// Blocks' second dimension: operands by ranks.
template <int ES>
__global__ void __launch_bounds__(kPadThreads) pad_kernel(const __grid_constant__ PadParams p) {
  stream_order();
  const int lane = threadIdx.x & 31;
  const int d = blockIdx.y % p.ranks;
  const PadRows& op = p.op[blockIdx.y / p.ranks];
  const int64_t warps = gridDim.x * (kPadThreads / 32), pitch = static_cast<int64_t>(op.width) * ES;
  int64_t last = op.rows;
  if (op.group == 0) {
    int32_t most = 0;
    for (int i = lane; i < p.each; i += 32) {
      const Rows r = tc::rows_of(p.offsets[d], i, p.capacity);
      most = max(most, r.first + r.count);
    }
    last = __reduce_max_sync(0xffffffffu, most);
  }
  const char* from = static_cast<const char*>(op.from[d]);
  const Bytes ends{from, from + op.rows * pitch};
  for (int64_t r = blockIdx.x * (kPadThreads / 32) + threadIdx.x / 32; r < last; r += warps) {
    if (op.group != 0 && tc::rows_of(p.offsets[d], static_cast<int>(r / op.group), p.capacity).count == 0) continue;
    const Row<ES, false> row(from + r * pitch, op.units, ends);
    uint4* to = reinterpret_cast<uint4*>(op.to) + (d * op.rows + r) * op.units;
    for (int c0 = lane; c0 < op.units; c0 += 32 * kPadAhead) {
      typename Row<ES, false>::Raw raw[kPadAhead];
#pragma unroll
      for (int i = 0; i < kPadAhead; ++i) raw[i] = c0 + i * 32 < op.units ? row.load(c0 + i * 32) : row.zero();
#pragma unroll
      for (int i = 0; i < kPadAhead; ++i)
        if (c0 + i * 32 < op.units) to[c0 + i * 32] = row.finish(raw[i], c0 + i * 32, op.width);
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
  if (capacity > kMaxCapacity) return fail(VC_ERR_INVALID_ARG, "too many rows");
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

// Groups of `blocks` blocks, one on each multiprocessor, for `tiles` of them at most.
unsigned grid_of(DeviceState* st, int64_t tiles, int blocks) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(tiles, st->nsm / blocks)));
}

// Scratch of one call, from the library's pool.
class Scratch {
 public:
  Scratch(DeviceState* st, int dev, cudaStream_t stream) : st_(st), dev_(dev), stream_(stream) {}
  ~Scratch() {
    if (mem_) cudaFreeAsync(mem_, stream_);
  }
  vc_status_t take(int64_t bytes) {
    cudaMemPool_t pool;
    vc_status_t rc = scratch_pool(st_, dev_, &pool);
    if (rc != VC_SUCCESS) return rc;
    cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void**>(&mem_), static_cast<size_t>(bytes), pool, stream_);
    if (e == cudaErrorMemoryAllocation) {
      cudaGetLastError();
      mem_ = nullptr;
      return fail(VC_ERR_NOMEM, "scratch allocation of " + std::to_string(bytes) + " bytes failed");
    }
    return e == cudaSuccess ? VC_SUCCESS : cuda_fail(e, "cudaMallocFromPoolAsync");
  }
  char* mem() const { return mem_; }

 private:
  DeviceState* st_;
  int dev_;
  cudaStream_t stream_;
  char* mem_ = nullptr;
};

// What a tensor map reads: rows of `width` elements, `pitch` bytes apart.
struct Operand {
  const void* p[VC_MAX_RANKS];
  int64_t rows, width, pitch, group;  // group: as PadParams
  int es;
  int64_t padded = -1;  // where its copy is in scratch

  Operand(const void* const* a, const Sizes& z, int64_t rows, int64_t width, int64_t group, int es)
      : rows(rows), width(width), pitch(width * es), group(group), es(es) {
    uintptr_t all = static_cast<uintptr_t>(pitch);
    for (int r = 0; r < z.nranks; ++r) {
      p[r] = a[r];
      all |= reinterpret_cast<uintptr_t>(a[r]);
    }
    if (rows != 0 && width != 0 && all % 16 != 0) padded = 0;
  }
};

// Copies the operands that want it to scratch, in one launch.
vc_status_t pad(DeviceState* st, int dev, const Sizes& z, const int32_t* const* offsets, Operand* const* ops, int n, Scratch* scratch,
                int* step, cudaStream_t stream) {
  int64_t need = 0;
  for (int i = 0; i < n; ++i)
    if (ops[i]->padded >= 0) {
      Operand& o = *ops[i];
      o.pitch = (o.width * o.es + 15) / 16 * 16;
      o.padded = need;
      need += (z.nranks * o.rows * o.pitch + 255) / 256 * 256;
    }
  if (need == 0) return VC_SUCCESS;
  vc_status_t rc = scratch->take(need);
  if (rc != VC_SUCCESS) return rc;
  PadParams p = {};
  int used = 0, es = 1;
  int64_t most = 0, bytes = 0;
  for (int i = 0; i < n; ++i)
    if (ops[i]->padded >= 0) {
      Operand& o = *ops[i];
      PadRows& to = p.op[used++];
      std::copy(o.p, o.p + z.nranks, to.from);
      to.to = scratch->mem() + o.padded;
      to.rows = o.rows;
      to.group = o.group;
      to.width = static_cast<int>(o.width);
      to.units = static_cast<int>(o.pitch / 16);
      es = o.es;
      most = std::max(most, o.rows);
      bytes += z.nranks * o.rows * (o.width * o.es + o.pitch);
      for (int r = 0; r < z.nranks; ++r) o.p[r] = to.to + r * o.rows * o.pitch;
    }
  std::copy(offsets, offsets + z.nranks, p.offsets);
  p.capacity = static_cast<int32_t>(z.capacity);
  p.ranks = z.nranks;
  p.each = z.each;
  const auto go = [&](auto size) {
    constexpr auto K = pad_kernel<size()>;
    const unsigned parts = static_cast<unsigned>(used * z.nranks);
    const int64_t fit = (int64_t(st->nsm) * resident_blocks<K>(dev, kPadThreads, 0) + parts - 1) / parts;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((most + 7) / 8, fit));
    return launch<K>(dev, Shape{blocks, kPadThreads, 0, 1, parts}, stream, p, kPad, (*step)++, bytes);
  };
  return es == 2 ? go(std::integral_constant<int, 2>{}) : go(std::integral_constant<int, 1>{});
}

CUtensorMapDataType map_type(vc_dtype_t d) {
  return d == VC_BFLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : d == VC_FLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}

vc_status_t map_rows(CUtensorMap* map, vc_dtype_t dtype, const Operand& o, int r, uint32_t box) {
  const uint64_t dims[2] = {static_cast<uint64_t>(o.width), static_cast<uint64_t>(o.rows)}, strides[1] = {static_cast<uint64_t>(o.pitch)};
  return tc::tensor_map(map, map_type(dtype), 2, o.p[r], dims, strides, 128 / o.es, box);
}
vc_status_t map_weights(CUtensorMap* map, vc_dtype_t dtype, const Operand& o, int r, uint32_t box) {
  const uint64_t dims[3] = {static_cast<uint64_t>(o.width), static_cast<uint64_t>(o.group), static_cast<uint64_t>(o.rows / o.group)};
  const uint64_t strides[2] = {static_cast<uint64_t>(o.pitch), static_cast<uint64_t>(o.pitch * o.group)};
  return tc::tensor_map(map, map_type(dtype), 3, o.p[r], dims, strides, 128 / o.es, box);
}

// Runs f with the 16-bit type, and how many ranks there is room for, as constants.
template <class F>
vc_status_t for_sizes(vc_dtype_t dtype, int nranks, F&& f) {
  using Few = std::integral_constant<int, 8>;
  using Many = std::integral_constant<int, VC_MAX_RANKS>;
  if (dtype == VC_BFLOAT16) {
    using T = std::integral_constant<int, VC_BFLOAT16>;
    return nranks <= 8 ? f(T{}, Few{}) : f(T{}, Many{});
  }
  using T = std::integral_constant<int, VC_FLOAT16>;
  return nranks <= 8 ? f(T{}, Few{}) : f(T{}, Many{});
}

// One launch of the tensor-core kernel.  a: weights or the right side of their
// gradient; b: rows or the left side.
template <int DT, int OUT, bool AMN, bool WEIGHT, int R>
vc_status_t launch_product(DeviceState* st, int dev, const Sizes& z, const Operand& a, const Operand& b, const int32_t* const* offsets,
                           void* const* out, int64_t M, int64_t N, int64_t K, int64_t tiles,
                           int64_t bytes, int step, cudaStream_t stream) {
  constexpr vc_dtype_t dtype = static_cast<vc_dtype_t>(DT);
  ProductParams<R> p;
  p.whole = M % 8 == 0;
  for (int r = 0; r < z.nranks; ++r) {
    vc_status_t rc = VC_SUCCESS;
    if (a.rows != 0 && a.width != 0 && b.rows != 0 && b.width != 0) {  // else no step loads anything
      rc = WEIGHT ? map_rows(&p.a[r], dtype, a, r, 64) : map_weights(&p.a[r], dtype, a, r, AMN ? 64 : 128);
      if (rc == VC_SUCCESS) rc = map_rows(&p.b[r], dtype, b, r, WEIGHT ? 64 : kRowBox);
    }
    if (rc != VC_SUCCESS) return rc;
    p.out[r] = out[r];
    p.offsets[r] = offsets[r];
    p.whole = p.whole && reinterpret_cast<uintptr_t>(out[r]) % 16 == 0;
  }
  p.capacity = static_cast<int32_t>(z.capacity);
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.experts = z.nexperts;
  p.each = z.each;
  return launch<product_kernel<DT, OUT, AMN, WEIGHT, R>>(dev, Shape{2 * grid_of(st, tiles, 2), kTcThreads, kTcSmem, 2}, stream, p,
                                                WEIGHT ? kExpertWeight : kExpertProduct, step, bytes);
}

// rows (capacity, in) times weights, in by width or width by in, to out (capacity, width).
vc_status_t rows_product(DeviceState* st, int dev, const Sizes& z, const Operand& rows, const Operand& weight,
                         const int32_t* const* offsets, void* const* out, int64_t in, int64_t width, bool transposed,
                         vc_dtype_t dtype, int step, cudaStream_t stream) {
  const int64_t bytes = (z.nranks * z.capacity * (in + width) + z.nexperts * in * width) * dtype_size(dtype);
  if (dtype != VC_FLOAT32) {
    const int64_t tiles = row_tiles(z, kTileN) * ((width + 2 * kTileM - 1) / (2 * kTileM));
    return for_sizes(dtype, z.nranks, [&](auto type, auto ranks) {
      const auto go = [&](auto mn) {
        return launch_product<type(), type(), mn(), false, ranks()>(st, dev, z, weight, rows, offsets, out, width, 0, in, tiles, bytes, step, stream);
      };
      return transposed ? go(std::false_type{}) : go(std::true_type{});
    });
  }
  SimpleParams p = {};
  for (int r = 0; r < z.nranks; ++r) {
    p.a[r] = weight.p[r];
    p.b[r] = rows.p[r];
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
  const int64_t tiles = row_tiles(z, kSimpleN) * ((width + kSimpleM - 1) / kSimpleM);
  constexpr auto K = product_simple_kernel<false>;
  return launch<K>(dev, Shape{simple_blocks<K>(st, dev, tiles), kSimpleThreads}, stream, p, kExpertProduct, step, bytes);
}

// dweight(n, m) = sum over the expert's rows of left(row, n) * right(row, m).
vc_status_t weights_gradient(DeviceState* st, int dev, const Sizes& z, const Operand& left, const Operand& right,
                             const int32_t* const* offsets, void* const* dweight, int64_t N, int64_t M, vc_dtype_t dtype,
                             vc_dtype_t out_dtype, int step, cudaStream_t stream) {
  const int64_t bytes = z.nranks * z.capacity * (N + M) * dtype_size(dtype) + z.nexperts * N * M * dtype_size(out_dtype);
  if (dtype != VC_FLOAT32) {
    const int64_t tiles = z.nexperts * ((N + kTileN - 1) / kTileN) * ((M + 2 * kTileM - 1) / (2 * kTileM));
    return for_sizes(dtype, z.nranks, [&](auto type, auto ranks) {
      const auto go = [&](auto to) {
        return launch_product<type(), to(), true, true, ranks()>(st, dev, z, right, left, offsets, dweight, M, N, 0, tiles, bytes, step, stream);
      };
      return out_dtype == VC_FLOAT32 ? go(std::integral_constant<int, VC_FLOAT32>{}) : go(type);
    });
  }
  SimpleParams p = {};
  for (int r = 0; r < z.nranks; ++r) {
    p.a[r] = right.p[r];
    p.b[r] = left.p[r];
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
  const int64_t tiles = z.nexperts * ((N + kSimpleN - 1) / kSimpleN) * ((M + kSimpleM - 1) / kSimpleM);
  constexpr auto K = product_simple_kernel<true>;
  return launch<K>(dev, Shape{simple_blocks<K>(st, dev, tiles), kSimpleThreads}, stream, p, kExpertWeight, step, bytes);
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
  Operand x(rows, z, z.capacity, z.in, 0, es);
  Operand w(weight, z, z.each * (transposed ? z.out : z.in), transposed ? z.in : z.out, transposed ? z.out : z.in, es);
  Scratch scratch(st, dev, stream);
  int step = 0;
  if (dtype != VC_FLOAT32) {
    Operand* const ops[] = {&x, &w};
    rc = pad(st, dev, z, offsets, ops, 2, &scratch, &step, stream);
  }
  if (rc != VC_SUCCESS) return rc;
  return rows_product(st, dev, z, x, w, offsets, out, z.in, z.out, transposed != 0, dtype, step, stream);
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
  const bool to_rows = drows && z.capacity != 0 && z.in != 0, to_weight = dweight && z.in != 0 && z.out != 0;
  if (!to_rows && !to_weight) return VC_SUCCESS;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  const int64_t outer = transposed ? z.out : z.in, inner = transposed ? z.in : z.out;
  Operand dy(dout, z, z.capacity, z.out, 0, es);
  Operand x(to_weight ? rows : dout, z, to_weight ? z.capacity : 0, z.in, 0, es);
  Operand w(to_rows ? weight : dout, z, to_rows ? z.each * outer : 0, inner, outer, es);
  Scratch scratch(st, dev, stream);
  int step = 0;
  if (dtype != VC_FLOAT32) {
    Operand* const ops[] = {&dy, &x, &w};
    rc = pad(st, dev, z, offsets, ops, 3, &scratch, &step, stream);
  }
  if (rc == VC_SUCCESS && to_rows)
    rc = rows_product(st, dev, z, dy, w, offsets, drows, z.out, z.in, !transposed, dtype, step++, stream);
  if (rc == VC_SUCCESS && to_weight)
    rc = transposed ? weights_gradient(st, dev, z, dy, x, offsets, dweight, z.out, z.in, dtype, dweight_dtype, step, stream)
                    : weights_gradient(st, dev, z, x, dy, offsets, dweight, z.in, z.out, dtype, dweight_dtype, step, stream);
  return rc;
}

vc_status_t product8(const void* const* rows, const float* const* row_scale, const void* const* weight, const float* const* weight_scale,
                     const int32_t* const* offsets, void* const* out, int nranks, int nexperts, size_t capacity, size_t in,
                     size_t width, vc_dtype_t out_dtype, cudaStream_t stream) {
  Sizes z;
  vc_status_t rc = check_sizes(&z, nranks, nexperts, capacity, in, width);
  if (rc == VC_SUCCESS) rc = check_float(out_dtype);
  if (rc != VC_SUCCESS) return rc;
  const int es = dtype_size(out_dtype);
  const int64_t blocks = (z.in + VC_FP8_BLOCK - 1) / VC_FP8_BLOCK, down = (z.out + VC_FP8_BLOCK - 1) / VC_FP8_BLOCK;
  const auto floats = [](const float* const* a) { return reinterpret_cast<const void* const*>(a); };
  Buffers b;
  rc = b.add(rows, nranks, z.capacity * z.in, 1, false, "rows");
  if (rc == VC_SUCCESS) rc = b.add(floats(row_scale), nranks, z.capacity * blocks * 4, 4, false, "row_scale");
  if (rc == VC_SUCCESS) rc = b.add(weight, nranks, z.each * z.in * z.out, 1, false, "weight");
  if (rc == VC_SUCCESS) rc = b.add(floats(weight_scale), nranks, z.each * down * blocks * 4, 4, false, "weight_scale");
  if (rc == VC_SUCCESS) rc = b.add(untyped(offsets), nranks, (z.each + 1) * 4, 4, false, "offsets");
  if (rc == VC_SUCCESS) rc = b.add(out, nranks, z.capacity * z.out * es, es, true, "out");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || z.capacity == 0 || z.out == 0) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  Operand x(rows, z, z.capacity, z.in, 0, 1), w(weight, z, z.each * z.out, z.in, z.out, 1);
  Scratch scratch(st, dev, stream);
  Operand* const ops[] = {&x, &w};
  int step = 0;
  rc = pad(st, dev, z, offsets, ops, 2, &scratch, &step, stream);
  if (rc != VC_SUCCESS) return rc;
  const int64_t bytes = z.nranks * z.capacity * (z.in + 4 * blocks + z.out * es) + z.nexperts * (z.in * z.out + 4 * down * blocks);
  const auto go = [&](auto code, auto ranks) {
    constexpr int R = ranks();
    Product8Params<R> p;
    p.whole = z.out * es % 16 == 0;
    for (int r = 0; r < nranks; ++r) {
      if (z.in != 0) {
        vc_status_t rc = map_rows(&p.rows[r], VC_INT8, x, r, 32);
        if (rc == VC_SUCCESS) rc = map_weights(&p.weight[r], VC_INT8, w, r, kTile8N);
        if (rc != VC_SUCCESS) return rc;
      }
      p.row_scale[r] = row_scale[r];
      p.weight_scale[r] = weight_scale[r];
      p.out[r] = out[r];
      p.offsets[r] = offsets[r];
      p.whole = p.whole && reinterpret_cast<uintptr_t>(out[r]) % 16 == 0;
    }
    p.capacity = static_cast<int32_t>(z.capacity);
    p.M = static_cast<int>(z.out);
    p.K = static_cast<int>(z.in);
    p.experts = z.nexperts;
    p.each = z.each;
    const int64_t tiles = row_tiles(z, kTileM) * ((z.out + kTile8N - 1) / kTile8N);
    return launch<product8_kernel<code(), R>>(dev, Shape{grid_of(st, tiles, 1), kTc8Threads, kTcSmem}, stream, p, kExpertProduct8, step, bytes);
  };
  return for_dtype(out_dtype, [&](auto code) {
    return nranks <= 8 ? go(code, std::integral_constant<int, 8>{}) : go(code, std::integral_constant<int, VC_MAX_RANKS>{});
  });
}

}  // namespace

cudaError_t take_product_errors(cudaStream_t stream, uint32_t* flags) {
  static const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(flags, dev::g_device_error, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(dev::g_device_error, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  return e;
}

namespace {
vc_status_t wait_drill(cudaStream_t stream, uint32_t* flags) {
  if (!flags) return fail(VC_ERR_INVALID_ARG, "null output pointer");
  *flags = 0;
  DeviceState* st = nullptr;
  int dev = 0;
  vc_status_t rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  uint32_t before = 0;
  cudaError_t e = take_product_errors(stream, &before);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(96);
    cfg.stream = stream;
    e = cudaLaunchKernelEx(&cfg, wait_drill_kernel);
  }
  if (e == cudaSuccess) e = take_product_errors(stream, flags);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e == cudaSuccess ? VC_SUCCESS : cuda_fail(e, "the waits' drill");
}
}  // namespace

namespace tc {
vc_status_t tensor_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* data, const uint64_t* dims,
                       const uint64_t* strides, uint32_t box0, uint32_t box1) {
  // the driver's call, found once through the runtime: nothing links with the driver
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<Encode> found{nullptr};
  Encode encode = found.load(std::memory_order_acquire);
  if (!encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult seen;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &seen);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDriverEntryPointByVersion");
    if (seen != cudaDriverEntryPointSuccess || !f) return fail(VC_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    encode = reinterpret_cast<Encode>(f);
    found.store(encode, std::memory_order_release);
  }
  cuuint64_t d[3], s[2];
  cuuint32_t box[3] = {box0, box1, 1}, one[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = dims[i];
  for (int i = 0; i + 1 < rank; ++i) s[i] = strides[i];
  const auto go = [&] {
    return encode(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(data), d, s, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = go();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // A thread's first call: unlike the runtime's calls the driver's does not
    // make the device's context current.
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
    r = go();
  }
  if (r != CUDA_SUCCESS) return fail(VC_ERR_CUDA, "cuTensorMapEncodeTiled: error " + std::to_string(static_cast<int>(r)));
  return VC_SUCCESS;
}
}  // namespace tc
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

VC_EXPORT vc_status_t vc_product_selftest(vc_stream_t stream, uint32_t* flags) {
  return entry([&] { return layer::wait_drill(reinterpret_cast<cudaStream_t>(stream), flags); });
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

VC_EXPORT vc_status_t vc_expert_product_fp8(const void* const* rows, const float* const* row_scale,
                                            const void* const* weight, const float* const* weight_scale,
                                            const int32_t* const* offsets, void* const* out, int nranks, int nexperts,
                                            size_t capacity, size_t in_width, size_t out_width, vc_dtype_t out_dtype,
                                            vc_stream_t stream) {
  return entry([&] {
    return layer::product8(rows, row_scale, weight, weight_scale, offsets, out, nranks, nexperts, capacity, in_width,
                           out_width, out_dtype, reinterpret_cast<cudaStream_t>(stream));
  });
}
