// Host services the library's translation units share: error reporting, the
// C entry guard, per-device state with the scratch pool, and the launch trace.
// Defined in vc.cu but for what says otherwise.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <new>
#include <string>
#include <vector>

#include "vc.h"

#define VC_EXPORT extern "C" __attribute__((visibility("default")))

namespace vc {

// Record the calling thread's last error and return its status.
vc_status_t fail(vc_status_t s, const std::string& msg);
vc_status_t cuda_fail(cudaError_t e, const char* what);
void clear_error();
// VC_PDL=0 launches every kernel in plain stream order (for comparison).
bool pdl_enabled();
bool log_enabled();

// Blocks of one kernel resident per SM.
struct Residency {
  int blocks = 1;
};
struct DeviceState {
  bool init = false;
  int nsm = 0;
  cudaMemPool_t pool = nullptr;
  std::map<const void*, Residency> occupancy;
};
vc_status_t device_state(DeviceState** out, int* dev_out);
vc_status_t scratch_pool(DeviceState* st, int dev, cudaMemPool_t* pool);

// One launch on `stream`, bracketed by events and recorded while the trace
// is on (`rec` without its time).
vc_status_t launch_traced(cudaStream_t stream, const vc_trace_record_t& rec, cudaError_t (*launch)(void*), void* arg);

namespace layer {
// Copies the exchange kernels' own device error word to *flags and clears it,
// in stream order (exchange.cu).
cudaError_t take_exchange_errors(cudaStream_t stream, uint32_t* flags);
// The same of the experts' products (expert.cu).
cudaError_t take_product_errors(cudaStream_t stream, uint32_t* flags);
}  // namespace layer

// No exception leaves a C entry point.
template <class F>
vc_status_t entry(F&& f) {
  clear_error();
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(VC_ERR_NOMEM, "host allocation failed");
  } catch (...) {
    return fail(VC_ERR_INVALID_ARG, "internal error");
  }
}

}  // namespace vc
