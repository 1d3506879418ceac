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

/* Workspace bytes of mxq_linear (backward == 0) or of mxq_linear_backward (!= 0), with any activation and outputs (the gradients
 * of a layer without one leave 2 tokens features bytes of it alone, where the others hold dz); 0 without tokens; negative: a
 * status. */
int64_t mxq_linear_workspace(int64_t tokens, int64_t hidden, int64_t features, int backward);

/*
 * mxq_linear - z[t, n] = sum_h x[t, h] w[n, h] + bias[n],  y = act(z) + residual:
 * binary32 sums of exact products, one rounding to y's type.
 *  x         BF16 [tokens, hidden], pitch ld_x;  w  BF16 [features, hidden], pitch ld_w
 *  bias      float [features], 16-byte aligned, or NULL
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
 *  dbias  float [features], 16-byte aligned, or NULL
 *  accumulate  != 0: dw and dbias are added to what is there, in binary32, one rounding
 * With an activation dz is held in bf16 for the products (half a step, 2^-8, of each
 * entry at most); dbias adds it up before that rounding.
 * Rules: as mxq_linear; one of dx, dw, dbias non-NULL.
 */
int mxq_linear_backward(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const void* dy, int64_t ld_dy,
                        int act, const void* z, int64_t ld_z, const void* add, int64_t ld_add, int64_t tokens,
                        int64_t hidden, int64_t features, void* dx, int64_t ld_dx, void* dw, int out, int64_t ld_dw,
                        float* dbias, int accumulate, void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of mxq_gated_linear (backward == 0) or of mxq_gated_linear_backward (!= 0), as above. */
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

/* One tensor of an update (an array of these is in device memory). */
typedef struct {
    void* param;        /* dense elements, aligned to their type, as all that follow */
    const void* grad;
    void* m;            /* the moments: float, or bytes (8-bit states) */
    void* v;
    float* m_scale;     /* 8-bit states: one for each MXQ_STATE_BLOCK elements, the last one for what is left */
    float* v_scale;
    void* copy;         /* BF16, receives the rounded parameters; may be NULL */
    int64_t numel;
    int64_t first;      /* the tensor's first chunk; its chunks are ceil(numel / MXQ_CLIP_CHUNK) */
    int32_t param_src;  /* MXQ_SRC_F32 or MXQ_SRC_BF16, as grad_src */
    int32_t grad_src;
    int32_t decay;      /* 0: no weight decay */
    int32_t pad;        /* 0 */
} mxq_adamw_tensor;
enum { MXQ_STATE_F32 = 0, MXQ_STATE_8BIT = 1, MXQ_STATE_BLOCK = 128 };

/*
 * mxq_adamw - one AdamW step over all tensors, in binary32:
 *   g = grad * min(1, max_norm / (norm + 1e-6))   (norm NULL: grad; in binary64 where binary32 would leave its normal numbers)
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - rate weight_decay) - rate / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 * parameters and copies rounded once (to nearest even) to their types.
 *  tensors   DEVICE mxq_adamw_tensor[count]
 *  chunk_of  DEVICE int32[chunks]: the tensor of each chunk
 *  rate_at, step_at  DEVICE float[1], int64_t[1], or NULL: read by the kernel in place of `rate` and
 *            `step`, so that a captured call follows them from replay to replay
 *  norm      DEVICE float[1] or NULL, as mxq_grad_norm leaves it
 * 8-bit states: a block of MXQ_STATE_BLOCK elements holds scale = max(A * (1 / F), 2^-120), A its largest finite
 * magnitude, F the format's largest value, 1 / F rounded to binary32, and codes of x / scale, saturating, a NaN staying one:
 *  m  E4M3, F = 448, rounded to nearest even
 *  v  E5M2, F = 57344, rounded up with the probability of what is cut off, and never to 0 if
 *     it was above.  (A rounding to nearest would lose changes of less than half a step: beta2
 *     near 1 makes no others.)
 * Scales and codes are those that the operations give one by one, each rounded to binary32: beta m + (1 - beta) g as two
 * products and a sum, ((1 - beta2) g) g, the coefficient as (1 / (norm + 1e-6)) max_norm, the constants rounded from binary64.
 * The chance: element e of a tensor lies at P = first * MXQ_CLIP_CHUNK + e of the list.  With R the low
 * word of the mixed 64-bit seed + step * 0x9E3779B97F4A7C15 (x ^= x >> 30, x *= 0xBF58476D1CE4E5B9, x ^= x >> 27,
 * x *= 0x94D049BB133111EB, x ^= x >> 31: SplitMix64, Steele, Lea and Flood 2014), the 32-bit r = lo(P/2) ^ R ^
 * hi(P/2) * 0x9E3779B1 is mixed (r ^= r >> 16, r *= 0x85EBCA6B, r ^= r >> 13, r *= 0xC2B2AE35, r ^= r >> 16: the finalizer of
 * Appleby's MurmurHash3); an even P takes its low half, an odd one its high half u, and the code is
 * floor(y / unit + u / 2^16) unit, y = v / scale, unit E5M2's step at y (below 2^-14 the sum is rounded to binary32).
 * Rules: fewer than 2^31 chunks; 0 <= beta < 1; 2^-126 <= eps <= 1e30; rate and weight_decay finite and not negative; step >= 1;
 * max_norm finite and not negative.  No tensor that is written overlaps another one.  (With eps below 2^-34, or
 * below 2^-39 / sqrt(1 - beta2), a v above 2^96 counts as infinite.)
 */
int mxq_adamw(const mxq_adamw_tensor* tensors, int64_t count, const int32_t* chunk_of, int64_t chunks, int states,
              double rate, const float* rate_at, double beta1, double beta2, double eps, double weight_decay,
              int64_t step, const int64_t* step_at, const float* norm, double max_norm, uint64_t seed, void* stream);

/*
 * mxq_grad_norm - the norm of mxq_clip_grad_norm alone, in binary64 and rounded to binary32; no tensor is written
 * (`out` is not looked at).  Arguments as there.
 */
int mxq_grad_norm(const mxq_clip_tensor* tensors, int64_t count, const int32_t* chunk_of, int64_t chunks, float* norm,
                  double* parts, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_DENSE_H */
