// dense_api.hip - the extern "C" entry points declared in include/mxq_dense.h.
// Every argument is validated on the host before any HIP call.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dense_launch.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
int hip_status(hipError_t e) { return e == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }
constexpr int64_t LIM31 = (int64_t)1 << 31, PITCH = (int64_t)4 << 20;

// A row pitch in bytes; nobody looks at that of a matrix that is not there.
int64_t in_bytes(const void* p, int64_t ld, int64_t size) { return p ? ld * size : 0; }

bool valid_out(int out) { return out == MXQ_OUT_F32 || out == MXQ_OUT_BF16; }
bool valid_act(int act) { return act >= MXQ_ACT_NONE && act <= MXQ_ACT_GELU_TANH; }

// width: features, or a gated layer's inter (most: 2^20, 2^19).
int check_sizes(int64_t tokens, int64_t hidden, int64_t width, int64_t most) {
    if (tokens < 0 || tokens >= LIM31 - 256) return MXQ_ERR_SHAPE;
    if (hidden < 8 || hidden % 8 != 0 || hidden > (1 << 20)) return MXQ_ERR_SHAPE;
    if (width < 8 || width % 8 != 0 || width > most) return MXQ_ERR_SHAPE;
    return MXQ_OK;
}

// A matrix of `cols` elements of `size` bytes a row, or none: statuses join in `st`, the first one stays.
struct Checks {
    int st = MXQ_OK;
    void fail(int s) { if (st == MXQ_OK) st = s; }
    void pitch(const void* p, int64_t ld, int64_t cols, int64_t size) {
        if (p && (ld < cols || ld > PITCH / size)) fail(MXQ_ERR_SHAPE);
    }
    void rows(const void* p, int64_t ld, int64_t size) {
        if (p && (!aligned(p, 16) || ld * size % 16 != 0)) fail(MXQ_ERR_ALIGN);
    }
};

int64_t workspace(int64_t tokens, int64_t hidden, int64_t width, bool gated, int backward) {
    const int st = check_sizes(tokens, hidden, width, gated ? 1 << 19 : 1 << 20);
    if (st != MXQ_OK) return st;
    return mxq::linear_bytes(tokens, hidden, gated ? 2 * width : width, gated ? width : 0, backward != 0);
}
// What is left to check once shapes hold.
int check_workspace(const void* ws, int64_t bytes, int64_t need) {
    if (need > 0 && !ws) return MXQ_ERR_NULL;
    if (bytes < need) return MXQ_ERR_SHAPE;
    return need > 0 && !aligned(ws, 16) ? MXQ_ERR_ALIGN : MXQ_OK;
}

int backward(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const void* dy, int64_t ld_dy, int act,
             const void* z, int64_t ld_z, const void* add, int64_t ld_add, int64_t tokens, int64_t hidden,
             int64_t width, bool gated, void* dx, int64_t ld_dx, void* dw, int out, int64_t ld_dw, float* dbias,
             int accumulate, void* ws, int64_t ws_bytes, void* stream) {
    if (!valid_act(act) || !valid_out(out)) return MXQ_ERR_FORMAT;
    const int64_t need = workspace(tokens, hidden, width, gated, 1);
    if (need < 0) return (int)need;
    const int64_t N = gated ? 2 * width : width, es = out == MXQ_OUT_F32 ? 4 : 2;
    Checks c;
    c.pitch(x, ld_x, hidden, 2); c.pitch(w, ld_w, hidden, 2); c.pitch(dy, ld_dy, width, 2); c.pitch(z, ld_z, N, 2);
    c.pitch(add, ld_add, hidden, 2); c.pitch(dx, ld_dx, hidden, 2); c.pitch(dw, ld_dw, hidden, es);
    if (c.st != MXQ_OK) return c.st;
    if (tokens > 0) {
        // dx takes w, dw takes x; computing a gated layer's sums again takes both
        const bool again = gated && !z;
        if (!dx && !dw && !dbias) return MXQ_ERR_NULL;
        if (!dy || (!x && (dw || again)) || (!w && (dx || again)) || (add && !dx)) return MXQ_ERR_NULL;
        if (!gated && act != MXQ_ACT_NONE && !z) return MXQ_ERR_NULL;
    }
    c.rows(x, ld_x, 2); c.rows(w, ld_w, 2); c.rows(dy, ld_dy, 2); c.rows(z, ld_z, 2); c.rows(add, ld_add, 2);
    c.rows(dx, ld_dx, 2); c.rows(dw, ld_dw, es);
    if (!aligned(dbias, 16)) c.fail(MXQ_ERR_ALIGN);
    if (c.st != MXQ_OK) return c.st;
    if (tokens > 0) {
        const int st = check_workspace(ws, ws_bytes, need);
        if (st != MXQ_OK) return st;
    }
    mxq::LinearArgs a{};
    a.x = (const uint8_t*)x; a.ld_x = in_bytes(x, ld_x, 2);
    a.w = (const uint8_t*)w; a.ld_w = in_bytes(w, ld_w, 2);
    a.T = tokens; a.H = hidden; a.N = N; a.inter = gated ? width : 0;
    a.act = act;
    a.dy = (const uint8_t*)dy; a.ld_dy = in_bytes(dy, ld_dy, 2);
    a.z = gated || act != MXQ_ACT_NONE ? (const uint8_t*)z : nullptr; a.ld_z = in_bytes(z, ld_z, 2);
    a.residual = (const uint8_t*)add; a.ld_r = in_bytes(add, ld_add, 2);
    a.dx = (uint8_t*)dx; a.ld_dx = in_bytes(dx, ld_dx, 2);
    a.dw = (uint8_t*)dw; a.ld_dw = in_bytes(dw, ld_dw, es); a.f32 = out == MXQ_OUT_F32;
    a.dbias = dbias;
    a.accumulate = accumulate != 0;
    a.ws = (uint8_t*)ws;
    return hip_status(mxq::launch_linear_backward(a, as_stream(stream)));
}

}  // namespace

extern "C" {

int64_t mxq_linear_workspace(int64_t tokens, int64_t hidden, int64_t features, int backward) {
    return workspace(tokens, hidden, features, false, backward);
}

int mxq_linear(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const float* bias, int act,
               const void* residual, int64_t ld_r, int64_t tokens, int64_t hidden, int64_t features, void* y, int out,
               int64_t ld_y, void* z, int64_t ld_z, void* ws, int64_t ws_bytes, void* stream) {
    if (!valid_act(act) || !valid_out(out)) return MXQ_ERR_FORMAT;
    const int64_t need = workspace(tokens, hidden, features, false, 0);
    if (need < 0) return (int)need;
    const int64_t es = out == MXQ_OUT_F32 ? 4 : 2;
    Checks c;
    c.pitch(x, ld_x, hidden, 2); c.pitch(w, ld_w, hidden, 2); c.pitch(residual, ld_r, features, es);
    c.pitch(y, ld_y, features, es); c.pitch(z, ld_z, features, 2);
    if (c.st != MXQ_OK || tokens == 0) return c.st;
    if (!x || !w || !y) return MXQ_ERR_NULL;
    c.rows(x, ld_x, 2); c.rows(w, ld_w, 2); c.rows(residual, ld_r, es); c.rows(y, ld_y, es); c.rows(z, ld_z, 2);
    if (!aligned(bias, 16)) c.fail(MXQ_ERR_ALIGN);
    c.fail(check_workspace(ws, ws_bytes, need));
    if (c.st != MXQ_OK) return c.st;
    mxq::LinearArgs a{};
    a.x = (const uint8_t*)x; a.ld_x = in_bytes(x, ld_x, 2);
    a.w = (const uint8_t*)w; a.ld_w = in_bytes(w, ld_w, 2);
    a.T = tokens; a.H = hidden; a.N = features;
    a.act = act; a.bias = bias;
    a.residual = (const uint8_t*)residual; a.ld_r = in_bytes(residual, ld_r, es);
    a.out = (uint8_t*)y; a.ld_out = in_bytes(y, ld_y, es); a.f32 = out == MXQ_OUT_F32;
    a.z_out = (uint8_t*)z; a.ld_z = in_bytes(z, ld_z, 2);
    a.ws = (uint8_t*)ws;
    return hip_status(mxq::launch_linear(a, as_stream(stream)));
}

int mxq_linear_backward(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const void* dy, int64_t ld_dy,
                        int act, const void* z, int64_t ld_z, const void* add, int64_t ld_add, int64_t tokens,
                        int64_t hidden, int64_t features, void* dx, int64_t ld_dx, void* dw, int out, int64_t ld_dw,
                        float* dbias, int accumulate, void* ws, int64_t ws_bytes, void* stream) {
    return backward(x, ld_x, w, ld_w, dy, ld_dy, act, z, ld_z, add, ld_add, tokens, hidden, features, false, dx,
                    ld_dx, dw, out, ld_dw, dbias, accumulate, ws, ws_bytes, stream);
}

int64_t mxq_gated_linear_workspace(int64_t tokens, int64_t hidden, int64_t inter, int backward) {
    return workspace(tokens, hidden, inter, true, backward);
}

int mxq_gated_linear(const void* x, int64_t ld_x, const void* w, int64_t ld_w, int act, int64_t tokens,
                     int64_t hidden, int64_t inter, void* h, int64_t ld_h, void* z, int64_t ld_z, void* ws,
                     int64_t ws_bytes, void* stream) {
    if (!valid_act(act)) return MXQ_ERR_FORMAT;
    const int64_t need = workspace(tokens, hidden, inter, true, 0);
    if (need < 0) return (int)need;
    Checks c;
    c.pitch(x, ld_x, hidden, 2); c.pitch(w, ld_w, hidden, 2); c.pitch(h, ld_h, inter, 2); c.pitch(z, ld_z, 2 * inter, 2);
    if (c.st != MXQ_OK || tokens == 0) return c.st;
    if (!x || !w || !h) return MXQ_ERR_NULL;
    c.rows(x, ld_x, 2); c.rows(w, ld_w, 2); c.rows(h, ld_h, 2); c.rows(z, ld_z, 2);
    c.fail(check_workspace(ws, ws_bytes, need));
    if (c.st != MXQ_OK) return c.st;
    mxq::LinearArgs a{};
    a.x = (const uint8_t*)x; a.ld_x = in_bytes(x, ld_x, 2);
    a.w = (const uint8_t*)w; a.ld_w = in_bytes(w, ld_w, 2);
    a.T = tokens; a.H = hidden; a.N = 2 * inter; a.inter = inter;
    a.act = act;
    a.out = (uint8_t*)h; a.ld_out = in_bytes(h, ld_h, 2);
    a.z_out = (uint8_t*)z; a.ld_z = in_bytes(z, ld_z, 2);
    a.ws = (uint8_t*)ws;
    return hip_status(mxq::launch_linear(a, as_stream(stream)));
}

int mxq_gated_linear_backward(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const void* dh, int64_t ld_dh,
                              int act, const void* z, int64_t ld_z, const void* add, int64_t ld_add, int64_t tokens,
                              int64_t hidden, int64_t inter, void* dx, int64_t ld_dx, void* dw, int out,
                              int64_t ld_dw, int accumulate, void* ws, int64_t ws_bytes, void* stream) {
    return backward(x, ld_x, w, ld_w, dh, ld_dh, act, z, ld_z, add, ld_add, tokens, hidden, inter, true, dx, ld_dx, dw,
                    out, ld_dw, nullptr, accumulate, ws, ws_bytes, stream);
}

int mxq_adamw(const mxq_adamw_tensor* tensors, int64_t count, const int32_t* chunk_of, int64_t chunks, int states,
              double rate, const float* rate_at, double beta1, double beta2, double eps, double weight_decay,
              int64_t step, const int64_t* step_at, const float* norm, double max_norm, uint64_t seed, void* stream) {
    if (states != MXQ_STATE_F32 && states != MXQ_STATE_8BIT) return MXQ_ERR_FORMAT;
    auto none_negative = [](double v) { return v >= 0.0 && !isinf(v); };
    if (count < 0 || count >= LIM31 || chunks < 0 || chunks >= LIM31) return MXQ_ERR_SHAPE;
    if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0x1p-126) || eps > 1e30 ||
        !none_negative(weight_decay) || !none_negative(max_norm) || (!rate_at && !none_negative(rate)) ||
        (!step_at && step < 1))
        return MXQ_ERR_SHAPE;
    if (chunks == 0) return MXQ_OK;
    if (!tensors || !chunk_of) return MXQ_ERR_NULL;
    if (!aligned(tensors, 8) || !aligned(chunk_of, 4) || !aligned(rate_at, 4) || !aligned(step_at, 8) || !aligned(norm, 4))
        return MXQ_ERR_ALIGN;
    const mxq::AdamwArgs a{tensors, chunk_of, chunks,   states, rate, beta1,   beta2, eps, weight_decay,
                           max_norm, step,    rate_at, norm,   step_at, seed};
    return hip_status(mxq::launch_adamw(a, as_stream(stream)));
}

int mxq_grad_norm(const mxq_clip_tensor* tensors, int64_t count, const int32_t* chunk_of, int64_t chunks, float* norm,
                  double* parts, void* stream) {
    if (count < 0 || count >= LIM31 || chunks < 0 || chunks >= LIM31) return MXQ_ERR_SHAPE;
    if (!norm || !parts || (chunks > 0 && (!tensors || !chunk_of))) return MXQ_ERR_NULL;
    if (!aligned(tensors, 8) || !aligned(chunk_of, 4) || !aligned(norm, 4) || !aligned(parts, 8)) return MXQ_ERR_ALIGN;
    return hip_status(mxq::launch_grad_norm(tensors, chunk_of, chunks, norm, parts, as_stream(stream)));
}

}  // extern "C"
