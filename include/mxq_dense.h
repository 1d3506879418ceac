/*
 * mxq_dense.h - C ABI of the layers and the update that a low-precision
 * recipe keeps out of FP8 (same library, libmxq.so): linear layers with bias,
 * activation and residual, gated layers, the gradients of both, and AdamW.
 *
 * Conventions are those of mxq.h and mxq_train.h: device pointers owned by
 * the caller, asynchronous calls on `stream`, statuses, workspaces whose size a
 * *_workspace function gives (16-byte aligned, free for other use after the call
 * in stream order), results that are the same from run to run.
 *
 * Matrices are row-major with a row pitch in elements: rows start on 16-byte
 * boundaries and a pitch is at most 4 MiB.  Outputs overlap no input, except
 * where a call says so.
 */
#ifndef MXQ_DENSE_H
#define MXQ_DENSE_H

#include "mxq_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Activations: z; max(z, 0); z / (1 + e^-z); z Phi(z), Phi the normal
 * distribution's; z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2.  In binary32.
 * The gradient of max(z, 0) is 0 at 0.
 */
enum { MXQ_ACT_NONE = 0, MXQ_ACT_RELU = 1, MXQ_ACT_SILU = 2, MXQ_ACT_GELU = 3, MXQ_ACT_GELU_TANH = 4 };

/* Workspace bytes of mxq_linear (backward == 0) or of mxq_linear_backward (!= 0); negative: a status. */
int64_t mxq_linear_workspace(int64_t tokens, int64_t hidden, int64_t features, int backward);

/*
 * mxq_linear - z[t, n] = sum_h x[t, h] w[n, h] + bias[n],  y = act(z) + residual:
 * binary32 sums of exact products, one rounding to y's type.
 *  x         BF16 [tokens, hidden], pitch ld_x;  w  BF16 [features, hidden], pitch ld_w
 *  bias      float [features], or NULL
 *  residual  [tokens, features] of y's type, pitch ld_r, or NULL; may be y itself (the same pitch)
 *  y         [tokens, features], MXQ_OUT_F32 or MXQ_OUT_BF16 (out), pitch ld_y
 *  z         BF16 [tokens, features], pitch ld_z, or NULL: receives z for the backward pass
 * Rules: hidden and features multiples of 8, from 8 to 2^20; tokens < 2^31 - 256.
 */
int mxq_linear(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const float* bias, int act,
               const void* residual, int64_t ld_r, int64_t tokens, int64_t hidden, int64_t features, void* y, int out,
               int64_t ld_y, void* z, int64_t ld_z, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * mxq_linear_backward - its gradients:  dz = dy act'(z),  dx = dz w + add,
 * dw = dz^T x,  dbias[n] = sum_t dz[t, n].
 *  dy     BF16 [tokens, features], pitch ld_dy
 *  z      BF16 as the forward call left it; NULL with MXQ_ACT_NONE
 *  add    BF16 [tokens, hidden], pitch ld_add, or NULL: joins dx (a skip connection's gradient); may be dx itself
 *  dx     BF16 [tokens, hidden], pitch ld_dx, or NULL (then add is NULL)
 *  dw     [features, hidden], MXQ_OUT_F32 or MXQ_OUT_BF16 (out), pitch ld_dw, or NULL
 *  dbias  float [features], or NULL
 *  accumulate  != 0: dw and dbias are added to what is there, in binary32, one rounding
 * With an activation dz is held in bf16 for the products (half a step, 2^-9, of each
 * entry at most); dbias adds it up before that rounding.
 * Rules: as mxq_linear; one of dx, dw, dbias non-NULL.
 */
int mxq_linear_backward(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const void* dy, int64_t ld_dy,
                        int act, const void* z, int64_t ld_z, const void* add, int64_t ld_add, int64_t tokens,
                        int64_t hidden, int64_t features, void* dx, int64_t ld_dx, void* dw, int out, int64_t ld_dw,
                        float* dbias, int accumulate, void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of mxq_gated_linear (backward == 0) or of mxq_gated_linear_backward (!= 0); negative: a status. */
int64_t mxq_gated_linear_workspace(int64_t tokens, int64_t hidden, int64_t inter, int backward);

/*
 * mxq_gated_linear - both projections of a gated layer, its activation and product
 * in one kernel:  gate = x w[0 .. inter)^T,  up = x w[inter .. 2 inter)^T,
 * h = act(gate) up, rounded once.
 *  x  BF16 [tokens, hidden], pitch ld_x;  w  BF16 [2 inter, hidden], pitch ld_w, the gate's rows first
 *  h  BF16 [tokens, inter], pitch ld_h
 *  z  BF16 [tokens, 2 inter], pitch ld_z, or NULL: receives gate and up for the backward pass
 * Rules: hidden and inter multiples of 8, hidden from 8 to 2^20, inter from 8 to 2^19; tokens < 2^31 - 256.
 */
int mxq_gated_linear(const void* x, int64_t ld_x, const void* w, int64_t ld_w, int act, int64_t tokens,
                     int64_t hidden, int64_t inter, void* h, int64_t ld_h, void* z, int64_t ld_z, void* workspace,
                     int64_t workspace_bytes, void* stream);

/*
 * mxq_gated_linear_backward - its gradients:  dgate = dh up act'(gate),
 * dup = dh act(gate),  dx = dgate w[0 .. inter) + dup w[inter ..) + add,
 * dw = [dgate, dup]^T x.
 *  dh   BF16 [tokens, inter], pitch ld_dh
 *  z    BF16 as the forward call left it, or NULL: gate and up are computed again, and stay in binary32
 *  add, dx, dw, out, accumulate  as mxq_linear_backward, dw of [2 inter, hidden]
 * dgate and dup are held in bf16 for the products.
 * Rules: as mxq_gated_linear; dx or dw non-NULL.
 */
int mxq_gated_linear_backward(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const void* dh, int64_t ld_dh,
                              int act, const void* z, int64_t ld_z, const void* add, int64_t ld_add, int64_t tokens,
                              int64_t hidden, int64_t inter, void* dx, int64_t ld_dx, void* dw, int out,
                              int64_t ld_dw, int accumulate, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_DENSE_H */
