// train_api.hip - the extern "C" entry points declared in include/mxq_train.h.
// Every argument is validated on the host before any HIP call.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "train_launch.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
int hip_status(hipError_t e) { return e == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }
bool valid_src(int s) { return s == MXQ_SRC_F32 || s == MXQ_SRC_BF16; }
int64_t size_of(int src) { return src == MXQ_SRC_BF16 ? 2 : 4; }
constexpr int64_t LIM31 = (int64_t)1 << 31;
// a * b < lim for non-negative a, b, without overflow
bool product_below(int64_t a, int64_t b, int64_t lim) { return a == 0 || b <= (lim - 1) / a; }

int check_topk(int src, int64_t tokens, int64_t experts, int64_t ld, int64_t topk) {
    if (!valid_src(src)) return MXQ_ERR_FORMAT;
    if (tokens < 0 || experts < 1 || experts > 1024 || topk < 1 || topk > 64 || topk > experts || ld < experts)
        return MXQ_ERR_SHAPE;
    if ((tokens + 3) / 4 >= LIM31) return MXQ_ERR_SHAPE;
    return MXQ_OK;
}

// Rows of cols elements in 16-byte units.
int check_rows(int src, int64_t tokens, int64_t cols, int64_t topk, int64_t rows) {
    if (!valid_src(src)) return MXQ_ERR_FORMAT;
    if (tokens < 0 || cols < 0 || rows < 0 || topk < 1 || topk > LIM31 - 1) return MXQ_ERR_SHAPE;
    if (cols % (16 / size_of(src)) != 0) return MXQ_ERR_SHAPE;
    if (cols / (16 / size_of(src)) >= LIM31 || tokens >= LIM31) return MXQ_ERR_SHAPE;
    return MXQ_OK;
}

int check_lce(int64_t ld_x, int64_t ld_w, int64_t tokens, int64_t hidden, int64_t vocab) {
    if (tokens < 0 || hidden < 8 || hidden % 8 != 0 || vocab < 1) return MXQ_ERR_SHAPE;
    if (tokens >= LIM31 - 256 || vocab >= LIM31 - 256) return MXQ_ERR_SHAPE;
    if (ld_x < hidden || ld_w < hidden || ld_x > (1 << 21) || ld_w > (1 << 21)) return MXQ_ERR_SHAPE;
    if (ld_x % 8 != 0 || ld_w % 8 != 0) return MXQ_ERR_ALIGN;
    // blocks of any product: tiles of 64 x 64 at the least, 64 splits at the most
    if (!product_below((vocab + 63) / 64, (tokens + 63) / 64, LIM31) ||
        !product_below((vocab + 63) / 64, (hidden + 63) / 64, LIM31) ||
        !product_below((tokens + 63) / 64, ((hidden + 63) / 64) * 64, LIM31))
        return MXQ_ERR_SHAPE;
    return MXQ_OK;
}

}  // namespace

extern "C" {

int mxq_moe_topk(const void* logits, int src, int64_t tokens, int64_t experts, int64_t ld, int64_t topk,
                 int renormalize, int32_t* ids, float* weights, void* stream) {
    const int st = check_topk(src, tokens, experts, ld, topk);
    if (st != MXQ_OK || tokens == 0) return st;
    if (!logits || !ids || !weights) return MXQ_ERR_NULL;
    if (!aligned(logits, size_of(src)) || !aligned(ids, 4) || !aligned(weights, 4)) return MXQ_ERR_ALIGN;
    return hip_status(mxq::launch_moe_topk(logits, src, tokens, experts, ld, (int)topk, renormalize != 0, ids, weights,
                                           as_stream(stream)));
}

int mxq_moe_topk_backward(const void* logits, int src, int64_t tokens, int64_t experts, int64_t ld,
                          const int32_t* ids, int64_t topk, int renormalize, const float* dweights, void* dlogits,
                          int64_t ld_d, void* stream) {
    const int st = check_topk(src, tokens, experts, ld, topk);
    if (st != MXQ_OK) return st;
    if (ld_d < experts) return MXQ_ERR_SHAPE;
    if (tokens == 0) return MXQ_OK;
    if (!logits || !ids || !dweights || !dlogits) return MXQ_ERR_NULL;
    if (!aligned(logits, size_of(src)) || !aligned(dlogits, size_of(src)) || !aligned(ids, 4) ||
        !aligned(dweights, 4))
        return MXQ_ERR_ALIGN;
    return hip_status(mxq::launch_moe_topk_backward(logits, src, tokens, experts, ld, ids, (int)topk,
                                                    renormalize != 0, dweights, dlogits, ld_d, as_stream(stream)));
}

int64_t mxq_moe_sort_workspace(int64_t tokens, int64_t topk, int64_t groups) {
    if (tokens < 0 || topk < 1 || groups < 1 || groups > 4096 || !product_below(tokens, topk, LIM31))
        return MXQ_ERR_SHAPE;
    return mxq::moe_sort_bytes(tokens * topk, groups);
}

int mxq_moe_sort(const int32_t* ids, int64_t tokens, int64_t topk, int64_t groups, int64_t* off, int32_t* src,
                 int32_t* pos, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = mxq_moe_sort_workspace(tokens, topk, groups);
    if (need < 0) return (int)need;
    if (!off || (tokens > 0 && (!ids || !pos))) return MXQ_ERR_NULL;
    if (need > 0 && !workspace) return MXQ_ERR_NULL;
    if (need > workspace_bytes) return MXQ_ERR_SHAPE;
    if (!aligned(off, 8) || !aligned(ids, 4) || !aligned(src, 4) || !aligned(pos, 4) ||
        (need > 0 && !aligned(workspace, 16)))
        return MXQ_ERR_ALIGN;
    return hip_status(mxq::launch_moe_sort(ids, tokens * topk, (int)topk, (int)groups, off, src, pos, workspace,
                                           as_stream(stream)));
}

int mxq_moe_dispatch_mx(const void* x, int src, int64_t tokens, int64_t cols, int64_t ld_x, const int32_t* pos,
                        int64_t topk, int fmt, int64_t rows, uint8_t* q, uint8_t* s, void* stream) {
    if (fmt != MXQ_E4M3 && fmt != MXQ_E5M2 && fmt != MXQ_E2M1) return MXQ_ERR_FORMAT;
    const int st = check_rows(src, tokens, cols, topk, rows);
    if (st != MXQ_OK) return st;
    if (cols % 32 != 0 || ld_x < cols || !product_below(tokens, cols / 16, LIM31)) return MXQ_ERR_SHAPE;
    if (tokens == 0 || cols == 0 || rows == 0) return MXQ_OK;
    if (!x || !pos || !q || !s) return MXQ_ERR_NULL;
    if (!aligned(x, 16) || (ld_x * size_of(src)) % 16 != 0 || !aligned(q, 16) || !aligned(pos, 4))
        return MXQ_ERR_ALIGN;
    return hip_status(mxq::launch_moe_dispatch_mx(x, src, tokens, cols, ld_x, pos, (int)topk, fmt, rows, q, s,
                                                  as_stream(stream)));
}

int mxq_moe_combine(const void* x, int src, int64_t rows, int64_t cols, int64_t ld_x, const int32_t* pos,
                    int64_t tokens, int64_t topk, const float* weights, void* y, int64_t ld_y, void* stream) {
    const int st = check_rows(src, tokens, cols, topk, rows);
    if (st != MXQ_OK) return st;
    if (ld_x < cols || ld_y < cols || !product_below(tokens, cols * size_of(src) / 16, LIM31)) return MXQ_ERR_SHAPE;
    if (tokens == 0 || cols == 0) return MXQ_OK;
    if ((rows > 0 && !x) || !pos || !y) return MXQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(y, 16) || (ld_x * size_of(src)) % 16 != 0 || (ld_y * size_of(src)) % 16 != 0 ||
        !aligned(pos, 4) || !aligned(weights, 4))
        return MXQ_ERR_ALIGN;
    return hip_status(mxq::launch_moe_combine(x, src, rows, cols, ld_x, pos, tokens, (int)topk, weights, y, ld_y,
                                              as_stream(stream)));
}

int mxq_moe_combine_backward(const void* dy, int src, int64_t tokens, int64_t cols, int64_t ld_dy,
                             const int32_t* pos, int64_t topk, const float* weights, const void* x, int64_t ld_x,
                             int64_t rows, void* dx, int64_t ld_dx, float* dweights, void* stream) {
    const int st = check_rows(src, tokens, cols, topk, rows);
    if (st != MXQ_OK) return st;
    if (topk > 64 || ld_dy < cols || (dx && ld_dx < cols) || (x && ld_x < cols)) return MXQ_ERR_SHAPE;
    if (!dx && !dweights) return MXQ_ERR_NULL;
    // with no columns (or no rows) the weights' gradient is still written: zeros
    if (tokens == 0) return MXQ_OK;
    if (!pos || (cols > 0 && !dy) || (dweights && rows > 0 && cols > 0 && !x)) return MXQ_ERR_NULL;
    const int64_t e = size_of(src);
    if (!aligned(dy, 16) || (ld_dy * e) % 16 != 0 || !aligned(pos, 4) || !aligned(weights, 4) ||
        !aligned(dweights, 4) || (x && (!aligned(x, 16) || (ld_x * e) % 16 != 0)) ||
        (dx && (!aligned(dx, 16) || (ld_dx * e) % 16 != 0)))
        return MXQ_ERR_ALIGN;
    return hip_status(mxq::launch_moe_combine_backward(dy, src, tokens, cols, ld_dy, pos, (int)topk, weights, x, ld_x,
                                                       rows, dx, ld_dx, dweights, as_stream(stream)));
}

int64_t mxq_linear_cross_entropy_workspace(int64_t tokens, int64_t hidden, int64_t vocab, int backward) {
    const int st = check_lce(hidden, hidden, tokens, hidden, vocab);
    if (st != MXQ_OK) return st;
    return mxq::lce_bytes(tokens, hidden, vocab, backward != 0);
}

int mxq_linear_cross_entropy(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const int64_t* targets,
                             int64_t tokens, int64_t hidden, int64_t vocab, float* loss, float* lse,
                             void* workspace, int64_t workspace_bytes, void* stream) {
    const int st = check_lce(ld_x, ld_w, tokens, hidden, vocab);
    if (st != MXQ_OK || tokens == 0) return st;
    if (!x || !w || !targets || !loss || !lse || !workspace) return MXQ_ERR_NULL;
    if (workspace_bytes < mxq::lce_bytes(tokens, hidden, vocab, false)) return MXQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(workspace, 16) || !aligned(targets, 8) || !aligned(loss, 4) ||
        !aligned(lse, 4))
        return MXQ_ERR_ALIGN;
    mxq::LceArgs a{};
    a.x = (const uint8_t*)x; a.w = (const uint8_t*)w; a.ld_x = ld_x * 2; a.ld_w = ld_w * 2;
    a.targets = targets; a.T = tokens; a.H = hidden; a.V = vocab;
    a.loss = loss; a.lse = lse; a.ws = (uint8_t*)workspace;
    return hip_status(mxq::launch_lce(a, as_stream(stream)));
}

int mxq_linear_cross_entropy_backward(const void* x, int64_t ld_x, const void* w, int64_t ld_w,
                                      const int64_t* targets, int64_t tokens, int64_t hidden, int64_t vocab,
                                      const float* lse, const float* dloss, void* dx, int64_t ld_dx, void* dw,
                                      int64_t ld_dw, void* workspace, int64_t workspace_bytes, void* stream) {
    const int st = check_lce(ld_x, ld_w, tokens, hidden, vocab);
    if (st != MXQ_OK) return st;
    if ((dx && ld_dx < hidden) || (dw && ld_dw < hidden)) return MXQ_ERR_SHAPE;
    if (!dx && !dw) return tokens == 0 ? MXQ_OK : MXQ_ERR_NULL;  // an empty dx is NULL
    if ((dx && (!aligned(dx, 16) || ld_dx % 8 != 0)) || (dw && (!aligned(dw, 16) || ld_dw % 8 != 0)))
        return MXQ_ERR_ALIGN;
    mxq::LceArgs a{};
    a.x = (const uint8_t*)x; a.w = (const uint8_t*)w; a.ld_x = ld_x * 2; a.ld_w = ld_w * 2;
    a.targets = targets; a.T = tokens; a.H = hidden; a.V = vocab;
    a.lse_in = lse; a.dloss = dloss; a.ws = (uint8_t*)workspace;
    a.dx = (uint8_t*)dx; a.dw = (uint8_t*)dw; a.ld_dx = ld_dx * 2; a.ld_dw = ld_dw * 2;
    if (tokens > 0) {
        if (!x || !w || !targets || !lse || !dloss || !workspace) return MXQ_ERR_NULL;
        if (workspace_bytes < mxq::lce_bytes(tokens, hidden, vocab, true)) return MXQ_ERR_SHAPE;
        if (!aligned(x, 16) || !aligned(w, 16) || !aligned(workspace, 16) || !aligned(targets, 8) ||
            !aligned(lse, 4) || !aligned(dloss, 4))
            return MXQ_ERR_ALIGN;
    }
    return hip_status(mxq::launch_lce_backward(a, as_stream(stream)));
}

int mxq_clip_grad_norm(const mxq_clip_tensor* tensors, int64_t count, const int32_t* chunk_of, int64_t chunks,
                       float max_norm, float* norm, double* parts, void* stream) {
    if (count < 0 || count >= LIM31 || chunks < 0 || chunks >= LIM31 || !(max_norm >= 0.0f) || isinf(max_norm)) return MXQ_ERR_SHAPE;
    if (!norm || !parts || (chunks > 0 && (!tensors || !chunk_of))) return MXQ_ERR_NULL;
    if (!aligned(tensors, 8) || !aligned(chunk_of, 4) || !aligned(norm, 4) || !aligned(parts, 8)) return MXQ_ERR_ALIGN;
    return hip_status(mxq::launch_clip(tensors, chunk_of, chunks, max_norm, norm, parts, as_stream(stream)));
}

}  // extern "C"
