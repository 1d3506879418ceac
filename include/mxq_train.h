/*
 * mxq_train.h - C ABI of the training-step operators around the scaled GEMMs
 * (same library, libmxq.so): the mixture-of-experts router and the movement of
 * token rows to and from their experts, softmax cross entropy against a
 * vocabulary projection, and clipping by the global gradient norm.
 *
 * Conventions (streams, ownership, statuses, alignment, zero sizes) are those
 * of mxq.h, with one addition: calls that need scratch memory take a
 * `workspace` of the bytes that the matching *_workspace function gives,
 * 16-byte aligned, owned by the caller and free for other use after the call
 * in stream order.  No call relies on what an earlier one left there.
 *
 * Every result is the same from run to run: no sum depends on the order in
 * which blocks finish.
 */
#ifndef MXQ_TRAIN_H
#define MXQ_TRAIN_H

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mxq_moe_topk - the router's choice: per token the topk largest logits, in
 * descending order, equal ones by the lower expert first, and their softmax
 * weights.
 *  logits  [tokens, experts] F32 or BF16 (src), row pitch ld elements
 *  ids     int32 [tokens, topk] the chosen experts
 *  weights float [tokens, topk]: renormalize == 0: exp(z_e - m) / sum over all
 *          experts; != 0: over the chosen ones only (m: the largest logit)
 * A NaN logit ranks above every number and makes its row's weights NaN; a row
 * whose largest logit is infinite has NaN weights, as the formula gives.
 * Rules: 1 <= topk <= min(experts, 64), experts <= 1024, ld >= experts,
 * tokens <= 2^33 - 4; logits aligned to its element.
 */
int mxq_moe_topk(const void* logits, int src, int64_t tokens, int64_t experts, int64_t ld, int64_t topk,
                 int renormalize, int32_t* ids, float* weights, void* stream);

/*
 * mxq_moe_topk_backward - the gradient of mxq_moe_topk's weights.  With p the
 * softmax (over all experts, or over the chosen ones) and g the weights'
 * gradients placed at their experts:  dlogits_e = p_e (g_e - sum_c p_c g_c);
 * renormalized, experts that were not chosen get zero.
 *  ids      int32 [tokens, topk], distinct per token; an id outside
 *           [0, experts) is left out
 *  dweights float [tokens, topk]
 *  dlogits  [tokens, experts], the logits' type, row pitch ld_d elements
 * Rules: as mxq_moe_topk.
 */
int mxq_moe_topk_backward(const void* logits, int src, int64_t tokens, int64_t experts, int64_t ld,
                          const int32_t* ids, int64_t topk, int renormalize, const float* dweights, void* dlogits,
                          int64_t ld_d, void* stream);

/* Workspace bytes of mxq_moe_sort for n = tokens * topk assignments; negative: a status. */
int64_t mxq_moe_sort_workspace(int64_t tokens, int64_t topk, int64_t groups);

/*
 * mxq_moe_sort - the assignments in expert order (a stable counting sort).
 *  ids   int32 [tokens, topk]; assignments to an expert outside [0, groups)
 *        (another rank's) are left out
 *  off   int64 [groups + 1]: group g holds rows off[g] .. off[g+1]-1, the
 *        layout that the grouped GEMMs take
 *  src   int32 [tokens * topk]: the token of each row, in expert order and
 *        within an expert in the order of ids; -1 at and past off[groups].
 *        May be NULL.
 *  pos   int32 [tokens, topk]: each assignment's row, or -1
 * Rules: topk >= 1, 1 <= groups <= 4096, tokens * topk < 2^31.
 */
int mxq_moe_sort(const int32_t* ids, int64_t tokens, int64_t topk, int64_t groups, int64_t* off, int32_t* src,
                 int32_t* pos, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * mxq_moe_dispatch_mx - token rows to their experts' rows, MX block-32
 * quantized on the way: the codes and scales that mxq_quantize_mx gives for
 * x, written to row pos[t, j] for every j.
 *  x    [tokens, cols], src F32 or BF16, row pitch ld_x elements
 *  pos  int32 [tokens, topk]; an entry outside [0, rows) is left out (rows is
 *       the buffers' capacity)
 *  q    [rows, cols] codes (E2M1: [rows, cols/2]), s [rows, cols/32] scales;
 *       rows that no entry names are not written
 * Rules: cols % 32 == 0, topk >= 1, tokens * cols / 16 < 2^31; x and its row
 * pitch and q 16-byte aligned.  Entries must name distinct rows.
 */
int mxq_moe_dispatch_mx(const void* x, int src, int64_t tokens, int64_t cols, int64_t ld_x, const int32_t* pos,
                        int64_t topk, int fmt, int64_t rows, uint8_t* q, uint8_t* s, void* stream);

/*
 * mxq_moe_combine - expert rows back to their tokens:
 * y[t] = sum_j weights[t, j] * x[pos[t, j]] in binary32, in the order of j,
 * rounded once; weights NULL: the plain sum (the gradient of a dispatch).
 *  x    [rows, cols], F32 or BF16 (src), row pitch ld_x elements
 *  y    [tokens, cols], the same type, row pitch ld_y elements
 *  pos  int32 [tokens, topk]; an entry outside [0, rows) adds nothing
 * Rules: cols and both pitches a multiple of 16 bytes; topk >= 1;
 * tokens * (16-byte units of a row) < 2^31.
 */
int mxq_moe_combine(const void* x, int src, int64_t rows, int64_t cols, int64_t ld_x, const int32_t* pos,
                    int64_t tokens, int64_t topk, const float* weights, void* y, int64_t ld_y, void* stream);

/*
 * mxq_moe_combine_backward - the gradients of mxq_moe_combine:
 * dx[pos[t, j]] = weights[t, j] * dy[t], dweights[t, j] = <x[pos[t, j]], dy[t]>
 * (binary32 sums; 0 where pos names no row).
 *  dy       [tokens, cols], dx [rows, cols] and x alike: one type (src)
 *  weights  float [tokens, topk], or NULL for ones
 *  dx       may be NULL; rows that no entry names are not written
 *  dweights float [tokens, topk], may be NULL; takes x (else x may be NULL)
 * Rules: cols and pitches as mxq_moe_combine; tokens < 2^31; 1 <= topk <= 64;
 * dx or dweights non-NULL.  Entries must name distinct rows.
 */
int mxq_moe_combine_backward(const void* dy, int src, int64_t tokens, int64_t cols, int64_t ld_dy,
                             const int32_t* pos, int64_t topk, const float* weights, const void* x, int64_t ld_x,
                             int64_t rows, void* dx, int64_t ld_dx, float* dweights, void* stream);

/* Workspace bytes of mxq_linear_cross_entropy (backward == 0) or of both it
 * and its gradient (!= 0); negative: a status. */
int64_t mxq_linear_cross_entropy_workspace(int64_t tokens, int64_t hidden, int64_t vocab, int backward);

/*
 * mxq_linear_cross_entropy - softmax cross entropy of hidden states against a
 * vocabulary projection, without the logits in memory:
 * z[t, v] = sum_h x[t, h] w[v, h] (binary32 sums of exact products),
 * lse[t] = log sum_v exp(z[t, v]),  loss[t] = lse[t] - z[t, targets[t]].
 *  x        BF16 [tokens, hidden], pitch ld_x;  w  BF16 [vocab, hidden], pitch ld_w
 *  targets  int64 [tokens]; outside [0, vocab): the token is ignored, loss 0
 *           (its lse is written all the same)
 *  loss, lse  float [tokens]; lse >= the largest logit, loss >= 0; NaN where a
 *           logit is NaN or +infinity
 * Rules: hidden % 8 == 0, hidden >= 8, vocab >= 1, tokens and vocab < 2^31 - 256;
 * pitches a multiple of 16 bytes and at most 4 MiB; x, w, workspace aligned.
 */
int mxq_linear_cross_entropy(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const int64_t* targets,
                             int64_t tokens, int64_t hidden, int64_t vocab, float* loss, float* lse,
                             void* workspace, int64_t workspace_bytes, void* stream);

/*
 * mxq_linear_cross_entropy_backward - its gradients, the logits computed again
 * in pieces of the vocabulary:  g[t, v] = (exp(z[t, v] - lse[t]) -
 * [v == targets[t]]) * dloss[t] (0 for ignored tokens),
 * dx = g w,  dw = g^T x.
 *  lse    float [tokens] as the forward call wrote it
 *  dloss  float [tokens]
 *  dx     BF16 [tokens, hidden], pitch ld_dx, or NULL
 *  dw     BF16 [vocab, hidden], pitch ld_dw, or NULL
 * g is held in bf16 (2^-8 of each entry at most), relative to the largest
 * |dloss| (the usual mean gives every token the same dloss, whose own rounding
 * then drops out); the sums are binary32 and rounded once.  An ignored token's
 * g is 0 and enters dw as 0 x: a NaN or an infinity in its x reaches dw, as the
 * formula gives.
 * Rules: as the forward call's; dx or dw non-NULL.
 */
int mxq_linear_cross_entropy_backward(const void* x, int64_t ld_x, const void* w, int64_t ld_w,
                                      const int64_t* targets, int64_t tokens, int64_t hidden, int64_t vocab,
                                      const float* lse, const float* dloss, void* dx, int64_t ld_dx, void* dw,
                                      int64_t ld_dw, void* workspace, int64_t workspace_bytes, void* stream);

/* One tensor of a clipping call (an array of these is in device memory). */
typedef struct {
    const void* in;     /* dense elements, aligned to their type */
    void* out;          /* as many; may be `in` itself */
    int64_t numel;
    int32_t src;        /* MXQ_SRC_F32 or MXQ_SRC_BF16 */
    int32_t pad;        /* 0 */
    int64_t first;      /* the tensor's first chunk; its chunks are ceil(numel / MXQ_CLIP_CHUNK) */
} mxq_clip_tensor;
enum { MXQ_CLIP_CHUNK = 8192, MXQ_CLIP_PARTS = 2048 };

/*
 * mxq_clip_grad_norm - the norm over all tensors and the clipped tensors:
 * norm = sqrt(sum of squares), out = in * min(1, max_norm / (norm + 1e-6)),
 * in binary64 and rounded to binary32 (BF16: from there to bf16).  A norm that is NaN (or infinite) reaches every output as
 * the formula gives.
 *  tensors   DEVICE mxq_clip_tensor[count]
 *  chunk_of  DEVICE int32[chunks]: the tensor of each chunk
 *  norm      float[1], the norm before clipping
 *  parts     DEVICE double[MXQ_CLIP_PARTS] scratch
 * Rules: fewer than 2^31 chunks; max_norm finite and not negative.
 * Outputs may be their inputs; otherwise they overlap no input.
 */
int mxq_clip_grad_norm(const mxq_clip_tensor* tensors, int64_t count, const int32_t* chunk_of, int64_t chunks,
                       float max_norm, float* norm, double* parts, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_TRAIN_H */
