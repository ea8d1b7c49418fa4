/* The layer operators from plain C99: declarations, the routing description,
 * and the argument checks, which come before any CUDA call. */
#include <stdio.h>

#include "vc.h"

int main(void) {
  /* addresses that nothing reads: every call below is refused or empty */
  const void* in[2] = {(void*)0x10000000, (void*)0x20000000};
  void* out[2] = {(void*)0x30000000, (void*)0x40000000};
  int32_t* ids[2] = {(int32_t*)0x50000000, (int32_t*)0x60000000};
  float* weights[2] = {(float*)0x70000000, (float*)0x78000000};
  vc_route_t how = {VC_SCORE_SIGMOID, 2, 4, 2, 2, 1, 2.5f};
  if (sizeof(vc_route_t) != 28) return 1;
  if (vc_route(in, NULL, ids, weights, 2, 0, 16, &how, VC_BFLOAT16, NULL) != VC_SUCCESS) return 2;
  how.topk_groups = 5;
  if (vc_route(in, NULL, ids, weights, 2, 4, 16, &how, VC_BFLOAT16, NULL) != VC_ERR_INVALID_ARG) return 3;
  how.topk_groups = 2;
  if (vc_route(in, NULL, ids, weights, 2, 4, VC_ROUTE_MAX_EXPERTS + 1, &how, VC_BFLOAT16, NULL) != VC_ERR_INVALID_ARG)
    return 4;
  if (vc_reduce_scatter_norm(in, NULL, in, NULL, out, NULL, NULL, 2, 4, VC_NORM_MAX_HIDDEN + 1, 1e-6, VC_FLOAT32,
                             VC_FLOAT32, NULL) != VC_ERR_UNSUPPORTED)
    return 5;
  if (vc_reduce_scatter_norm(in, NULL, in, NULL, out, NULL, NULL, 2, 4, 64, 1e-6, VC_FLOAT32, VC_INT8, NULL) !=
      VC_ERR_INVALID_ARG)
    return 6; /* 8 bits want scales */
  if (vc_dispatch_plan((const int32_t* const*)ids, ids, ids, 2, 4, 2, 16, 8, NULL) != VC_ERR_INVALID_ARG) return 7;
  if (vc_combine(in, (const int32_t* const*)ids, NULL, out, 2, 0, 64, 2, 8, VC_FLOAT16, NULL) != VC_SUCCESS) return 8;
  printf("ok\n");
  return 0;
}
