// dense_launch.h - internal launchers behind include/mxq_dense.h (arguments
// already validated on the host by dense_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxq_dense.h"
#include "train_launch.h"

namespace mxq {

// Linear and gated layers (linear.hip).  inter > 0: gated, N = 2 inter.  Pitches in bytes.
struct LinearArgs {
    const uint8_t *x, *w;        // bf16 [T, H], [N, H]
    int64_t ld_x, ld_w;
    int64_t T, H, N, inter;
    int act;
    const float* bias;
    const uint8_t* residual;     // forward: of y's type; backward: bf16, joins dx
    int64_t ld_r;
    uint8_t* out;                // y or h
    int64_t ld_out;
    int f32;                     // y (forward), dw (backward)
    uint8_t* z_out;
    const uint8_t *z, *dy;       // backward
    int64_t ld_z, ld_dy;
    uint8_t *dx, *dw;
    int64_t ld_dx, ld_dw;
    float* dbias;
    int accumulate;
    uint8_t* ws;
    int64_t ws_part;             // where in the workspace the forward product's partial sums go
};
int64_t linear_bytes(int64_t T, int64_t H, int64_t N, int64_t inter, bool backward);
hipError_t launch_linear(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_backward(const LinearArgs& a, hipStream_t st);

// AdamW (adamw.hip) and the norm alone (clip.hip).
struct AdamwArgs {
    const mxq_adamw_tensor* tensors;
    const int32_t* chunk_of;
    int64_t chunks;
    int states;
    double rate, beta1, beta2, eps, weight_decay, max_norm;
    int64_t step;
    const float *rate_at, *norm;
    const int64_t* step_at;
    uint64_t seed;
};
hipError_t launch_adamw(const AdamwArgs& a, hipStream_t st);
hipError_t launch_grad_norm(const mxq_clip_tensor* t, const int32_t* chunk_of, int64_t chunks, float* norm,
                            double* parts, hipStream_t st);

}  // namespace mxq
