// A stand-in for the CUDA runtime calls by which the library's host code sets
// up and makes a launch, so that this code runs without a GPU and its calls
// can be made to fail, wait or interleave.  No kernel runs; a launch is checked
// against what its kernel was allowed, and recorded.  Linked with the
// library's objects in place of those calls; every other symbol is the real
// runtime's.
#include <cuda_runtime_api.h>

#include <chrono>
#include <condition_variable>
#include <map>
#include <mutex>
#include <vector>

#define HOOK extern "C" __attribute__((visibility("default")))
#define FAKE extern "C" __attribute__((visibility("hidden")))

namespace {
constexpr int kOptIn = 232448, kStatic = 1024, kFree = 48 << 10;  // shared memory: of a block, of every kernel, without leave

struct Kernel {
  int most = kFree - kStatic;  // dynamic shared memory
  bool wide = false;           // clusters above 8 blocks
};
struct Launch {
  int grid, block, smem, cluster, status;
};
std::mutex mu;
std::condition_variable changed;
std::map<const void*, Kernel> kernels;
std::vector<Launch> launches;
int largest_cluster = 16, occupancy_queries = 0;
int held = 0;             // launches that a held thread waits for; 0: none is held
bool holding = false;     // a thread is held
cudaError_t last = cudaSuccess;

cudaError_t set_last(cudaError_t e) {
  if (e != cudaSuccess) last = e;
  return e;
}
int cluster_of(const cudaLaunchConfig_t* c) {
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return static_cast<int>(c->attrs[i].val.clusterDim.x);
  return 1;
}
}  // namespace

// -- what a test sets and reads -------------------------------------------------
HOOK void fake_reset() {
  std::lock_guard<std::mutex> lk(mu);
  kernels.clear();
  launches.clear();
  largest_cluster = 16;
  occupancy_queries = 0;
  held = 0;
  last = cudaSuccess;
}
HOOK void fake_largest_cluster(int n) {
  std::lock_guard<std::mutex> lk(mu);
  largest_cluster = n;
}
// The next thread that sets a kernel's shared memory is held, once that is
// set, until another thread has launched (10 s at most).
HOOK void fake_hold_next_setter() {
  std::lock_guard<std::mutex> lk(mu);
  held = 1;
}
// Waits until a thread is held (10 s at most); whether one is.
HOOK int fake_wait_held() {
  std::unique_lock<std::mutex> lk(mu);
  return changed.wait_for(lk, std::chrono::seconds(10), [] { return holding; });
}
HOOK int fake_launches() {
  std::lock_guard<std::mutex> lk(mu);
  return static_cast<int>(launches.size());
}
HOOK void fake_launch(int i, int* five) {
  std::lock_guard<std::mutex> lk(mu);
  const Launch& l = launches[i];
  const int v[5] = {l.grid, l.block, l.smem, l.cluster, l.status};
  for (int k = 0; k < 5; ++k) five[k] = v[k];
}

// -- the runtime's calls --------------------------------------------------------
FAKE cudaError_t cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
FAKE cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr attr, int) {
  *value = attr == cudaDevAttrMultiProcessorCount            ? 152
           : attr == cudaDevAttrMaxSharedMemoryPerBlockOptin ? kOptIn
                                                             : 0;
  return cudaSuccess;
}
FAKE cudaError_t cudaGetLastError() {
  std::lock_guard<std::mutex> lk(mu);
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
FAKE cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void* f) {
  std::lock_guard<std::mutex> lk(mu);
  *a = cudaFuncAttributes{};
  a->sharedSizeBytes = kStatic;
  a->maxDynamicSharedSizeBytes = kernels[f].most;
  return cudaSuccess;
}
FAKE cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute attr, int value) {
  std::unique_lock<std::mutex> lk(mu);
  if (attr == cudaFuncAttributeNonPortableClusterSizeAllowed) {
    kernels[f].wide = value != 0;
  } else if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) {
    if (value < 0 || value + kStatic > kOptIn) return set_last(cudaErrorInvalidValue);
    kernels[f].most = value;
    if (held) {
      held = 0;
      holding = true;
      changed.notify_all();
      const size_t before = launches.size();
      changed.wait_for(lk, std::chrono::seconds(10), [&] { return launches.size() > before; });
      holding = false;
    }
  }
  return cudaSuccess;
}
FAKE cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  std::lock_guard<std::mutex> lk(mu);
  ++occupancy_queries;
  *n = 1;
  return cudaSuccess;
}
FAKE cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int block, size_t smem) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(n, f, block, smem, 0);
}
FAKE cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  std::lock_guard<std::mutex> lk(mu);
  const Kernel& k = kernels[f];
  const int cluster = cluster_of(c);
  *n = 0;
  if ((cluster > 8 && !k.wide) || static_cast<int>(c->dynamicSmemBytes) > k.most) return set_last(cudaErrorInvalidValue);
  if (cluster > largest_cluster) return set_last(cudaErrorInvalidClusterSize);
  *n = 1;
  return cudaSuccess;
}
FAKE cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  std::lock_guard<std::mutex> lk(mu);
  const Kernel& k = kernels[f];
  const int cluster = cluster_of(c), smem = static_cast<int>(c->dynamicSmemBytes);
  cudaError_t e = cudaSuccess;
  if (smem > k.most) e = cudaErrorInvalidValue;
  else if (cluster > largest_cluster || (cluster > 8 && !k.wide)) e = cudaErrorInvalidClusterSize;
  launches.push_back(Launch{static_cast<int>(c->gridDim.x), static_cast<int>(c->blockDim.x), smem, cluster, static_cast<int>(e)});
  changed.notify_all();
  return set_last(e);
}
// scratch: addresses that nothing reads
FAKE cudaError_t cudaMemPoolCreate(cudaMemPool_t* pool, const cudaMemPoolProps*) {
  *pool = reinterpret_cast<cudaMemPool_t>(0x10);
  return cudaSuccess;
}
FAKE cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void*) { return cudaSuccess; }
FAKE cudaError_t cudaMallocFromPoolAsync(void** p, size_t, cudaMemPool_t, cudaStream_t) {
  *p = reinterpret_cast<void*>(uintptr_t(1) << 44);
  return cudaSuccess;
}
FAKE cudaError_t cudaFreeAsync(void*, cudaStream_t) { return cudaSuccess; }
