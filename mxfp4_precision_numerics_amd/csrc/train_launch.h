// train_launch.h - internal launchers behind include/mxq_train.h (arguments
// already validated on the host by train_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxq_train.h"

namespace mxq {

// The runtime refuses a launch of 2^32 threads; calls that need as many go out
// in launches of up to this many.
constexpr int64_t LAUNCH_THREADS = (int64_t)1 << 31;

hipError_t launch_moe_topk(const void* z, int src, int64_t T, int64_t E, int64_t ld, int k, int renorm, int32_t* ids,
                           float* w, hipStream_t st);
hipError_t launch_moe_topk_backward(const void* z, int src, int64_t T, int64_t E, int64_t ld, const int32_t* ids,
                                    int k, int renorm, const float* dw, void* dz, int64_t ld_d, hipStream_t st);

int64_t moe_sort_bytes(int64_t n, int64_t G);
hipError_t launch_moe_sort(const int32_t* ids, int64_t n, int k, int G, int64_t* off, int32_t* src, int32_t* pos,
                           void* ws, hipStream_t st);

hipError_t launch_moe_dispatch_mx(const void* x, int src, int64_t T, int64_t C, int64_t ld, const int32_t* pos, int k,
                                  int fmt, int64_t R, uint8_t* q, uint8_t* s, hipStream_t st);
hipError_t launch_moe_combine(const void* x, int src, int64_t R, int64_t C, int64_t ld_x, const int32_t* pos,
                              int64_t T, int k, const float* w, void* y, int64_t ld_y, hipStream_t st);
hipError_t launch_moe_combine_backward(const void* dy, int src, int64_t T, int64_t C, int64_t ld_dy,
                                       const int32_t* pos, int k, const float* w, const void* x, int64_t ld_x,
                                       int64_t R, void* dx, int64_t ld_dx, float* dw, hipStream_t st);

// Cross entropy against a vocabulary projection (loss.hip).
struct LceArgs {
    const uint8_t *x, *w;      // bf16 [T, H], [V, H]
    int64_t ld_x, ld_w;        // bytes
    const int64_t* targets;
    int64_t T, H, V;
    float *loss, *lse;
    const float *lse_in, *dloss;
    uint8_t *dx, *dw;          // bf16, or nullptr
    int64_t ld_dx, ld_dw;      // bytes
    uint8_t* ws;
};
int64_t lce_bytes(int64_t T, int64_t H, int64_t V, bool backward);
hipError_t launch_lce(const LceArgs& a, hipStream_t st);
hipError_t launch_lce_backward(const LceArgs& a, hipStream_t st);

hipError_t launch_clip(const mxq_clip_tensor* t, const int32_t* chunk_of, int64_t chunks, float max_norm, float* norm,
                       double* parts, hipStream_t st);

}  // namespace mxq
