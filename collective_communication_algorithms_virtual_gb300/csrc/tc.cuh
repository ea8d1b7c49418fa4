// What the tensor-core kernels of expert.cu share: bounded waits, tensor-map
// loads, tcgen05 instructions and their descriptors, and the list of tiles that
// ragged experts make.
#pragma once

#include <cuda.h>

#include "layer.cuh"

namespace vc {
namespace layer {
namespace tc {

// ---------------------------------------------------------------------------
// device: barriers
// ---------------------------------------------------------------------------
using dev::smem_addr;

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A barrier of another block of the cluster (at the same place there): `rank`
// is the block's.
__device__ __forceinline__ uint32_t bar_of(uint32_t bar, uint32_t rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(bar), "r"(rank));
  return at;
}
__device__ __forceinline__ void bar_expect_there(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive_there(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same for what this block has written itself and the other one will read,
// which the default scope (this block) does not cover; with a wait of CLUSTER at
// the other end.
__device__ __forceinline__ void bar_release_there(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t rank_in_cluster() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// CLUSTER: what other blocks of the cluster have written before their arrival is
// there too.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
  return ok != 0;
}
// Polls with test_wait, which never blocks.  `gone` (shared memory) is set by
// whichever role gives up first and ends every other role's waits, so that the
// block returns.  Loads, single steps of a product and the reading of an
// accumulator end within microseconds: kSoon is some 0.3 s.  A whole product
// may have 2^25 steps: kLate is some 20 s.
constexpr uint32_t kSoon = 1u << 22, kLate = 1u << 28;
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gone, uint32_t limit = kSoon) {
  for (uint32_t it = 0; it < limit; ++it) {
    if (bar_test<CLUSTER>(bar, parity)) return true;
    if (it >= 256) {
      if (*gone) return false;
      __nanosleep(64);
    }
  }
  *gone = 1;
  return false;
}

// The same of a whole warp, whose lanes go on or give up together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gone, uint32_t limit = kSoon) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, gone, limit));
}

// ---------------------------------------------------------------------------
// device: loads by tensor maps
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load2d(uint32_t to, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(to),
               "l"(map), "r"(bar), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void load3d(uint32_t to, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(to),
               "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// The same into this block of a pair, whose first block's barrier (`bar`, from
// bar_of) is told.
__device__ __forceinline__ void load2d_pair(uint32_t to, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(to),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void load3d_pair(uint32_t to, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(to),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// ---------------------------------------------------------------------------
// device: tcgen05
// ---------------------------------------------------------------------------
// Tiles lie in shared memory in rows of 128 bytes, 128-byte swizzled in groups
// of eight rows (1024 bytes), as the tensor maps write them.  Operands whose
// rows run along K ("K-major"): a row is an element of M or N, 64 elements of K
// (128 of an 8-bit type); one step of the product (32 bytes of K) starts 32
// bytes on.  Operands whose rows run along M or N: a row is an element of K,
// blocks of 64 elements of M or N lie `block` bytes apart, and one step (16
// elements of K) starts 2048 bytes on.
constexpr uint64_t kDescriptor = (uint64_t(1) << 46) | (uint64_t(2) << 61);  // version 1, 128-byte swizzle
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return kDescriptor | ((addr >> 4) & 0x3fff) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t block) {
  return kDescriptor | ((addr >> 4) & 0x3fff) | (static_cast<uint64_t>(block >> 4) << 16) | (uint64_t(1024 >> 4) << 32);
}
// The instruction descriptor: fp32 sums, operand type (kind::f16: 0 fp16, 1
// bf16; kind::f8f6f4: 0 e4m3), which operands run along M or N, and N and M.
__device__ __forceinline__ uint32_t instruction(uint32_t type, bool a_mn, bool b_mn, uint32_t n, uint32_t m) {
  return (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         ((n >> 3) << 17) | ((m >> 4) << 24);
}
// Pairs of blocks: 256 of M, 128 in each block's tensor memory; each block's
// shared memory holds its half of A and half of B's N, at the same place.
__device__ __forceinline__ void mma16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t how, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
               "l"(a), "l"(b), "r"(how), "r"(static_cast<uint32_t>(add))
               : "memory");
}
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t how, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
               "l"(a), "l"(b), "r"(how), "r"(static_cast<uint32_t>(add))
               : "memory");
}
// One thread of a warp, which the compiler knows to be one.
__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
// The barrier is arrived at once every product issued so far has been done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The same at this place in both blocks of the pair.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"(static_cast<uint16_t>(3))
               : "memory");
}
__device__ __forceinline__ void before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One warp (of each block of a pair) takes the accumulators' columns, and gives up
// the right to take more and frees them.  A pair's blocks take theirs together:
// the one that starts first must not ask before the other one is there (behind
// a kernel that leaves its multiprocessors one by one they start far enough
// apart that once in some ten thousand launches its request was never answered),
// nor may either end or give up while the other one takes or frees.  So a pair
// meets (cluster_sync) before it takes, before it gives up and frees, and after.
template <bool PAIR>
__device__ __forceinline__ void take_columns(uint32_t to, uint32_t n) {
  if constexpr (PAIR) asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(n) : "memory");
  else asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(n) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void take_no_more() {
  if constexpr (PAIR) asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  else asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <bool PAIR>
__device__ __forceinline__ void free_columns(uint32_t at, uint32_t n) {
  if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(n) : "memory");
  else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(n) : "memory");
}
// 32 columns of the warp's 32 lanes; complete after loaded().
__device__ __forceinline__ void load_columns(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// The values pass through, so that no use of them comes before the wait.
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// The same of 16 columns.
__device__ __forceinline__ void load_columns(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void loaded(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// ---------------------------------------------------------------------------
// device: the tiles of ragged experts
// ---------------------------------------------------------------------------
// The rows of a rank's expert i, whatever the offsets hold: within the buffer.
struct Rows {
  int32_t first, count;
};
__device__ __forceinline__ Rows rows_of(const int32_t* offsets, int i, int32_t capacity) {
  const int32_t lo = min(max(__ldg(offsets + i), 0), capacity), hi = min(max(__ldg(offsets + i + 1), lo), capacity);
  return Rows{lo, hi - lo};
}
// `count` in as few pieces of at most `most` as it takes, all but the last as
// long as each other and a multiple of `unit`.
__device__ __forceinline__ int pieces(int count, int most) { return (count + most - 1) / most; }
__device__ __forceinline__ int piece_of(int count, int most, int unit) {
  const int n = max(pieces(count, most), 1);
  return ((count + n - 1) / n + unit - 1) / unit * unit;
}

// Each expert's tiles counted up: ends[e] is where expert e's end in the list
// of all.  By the first warp; `longest` gets the largest count of rows.
__device__ __forceinline__ void list_tiles(const int32_t* const* offsets, int experts, int each, int32_t capacity, int most,
                                           uint32_t across, uint32_t* ends, int* longest) {
  const int lane = threadIdx.x & 31;
  uint32_t before = 0;
  int top = 0;
  for (int base = 0; base < experts; base += 32) {
    const int e = base + lane;
    uint32_t n = 0;
    if (e < experts) {
      const int count = rows_of(offsets[e / each], e % each, capacity).count;
      top = max(top, count);
      n = static_cast<uint32_t>(pieces(count, most)) * across;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += x;
    }
    n += before;
    if (e < experts) ends[e] = n;
    before = __shfl_sync(0xffffffffu, n, 31);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) *longest = top;
}

// ---------------------------------------------------------------------------
// host: tensor maps
// ---------------------------------------------------------------------------
// A map of `data`, dims[0] contiguous and strides[i] (bytes) between elements
// of dims[i + 1]; boxes of 128 bytes by `box` rows, 128-byte swizzled.
vc_status_t tensor_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* data, const uint64_t* dims,
                       const uint64_t* strides, uint32_t box0, uint32_t box1);

}  // namespace tc
}  // namespace layer
}  // namespace vc
