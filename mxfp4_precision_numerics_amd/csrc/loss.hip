// loss.hip - softmax cross entropy of hidden states against a vocabulary
// projection, and its gradients, for gfx950: no logits in memory.
//
//   forward   z = x w^T tile by tile; each tile leaves a (max, sum of exp) per
//             token, a second launch joins them:  lse, loss = lse - z[target]
//   backward  per piece of the vocabulary:  g = (exp(z - lse) - onehot) dloss,
//             z computed again, g held in bf16;  dx += g w,  dw = g^T x
//
// The products are 2 T V H operations forward and 6 T V H backward, two more
// than with the logits kept.
#include "loss_gemm.h"

namespace mxq {
namespace {

// Tiles: 256 x 256 with 8 waves, or 128 (m) x 64 (n) with 4.
struct Big { static constexpr int BM = 256, BN = 256, WGM = 2, WGN = 4, NSL = 2; };
struct Small { static constexpr int BM = 128, BN = 64, WGM = 4, WGN = 1, NSL = 3; };

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class C, bool TA, bool TB, int EPI> hipError_t gemm_cfg(LossGemm g, int splits, hipStream_t st) {
    g.ntm = ceil_div(g.M, C::BM);
    g.ntn = ceil_div(g.N, C::BN);
    const int64_t nk = ceil_div(g.K, KT);
    g.per = ceil_div(nk > 0 ? nk : 1, splits);
    g.splits = splits;
    const unsigned nb = (unsigned)(g.ntm * g.ntn * splits);
    if constexpr (C::BM == 256) k_loss_gemm_pipe<TA, TB, EPI><<<nb, 512, 0, st>>>(g);
    else k_loss_gemm<C::BM, C::BN, C::WGM, C::WGN, C::NSL, TA, TB, EPI><<<nb, 64 * C::WGM * C::WGN, 0, st>>>(g);
    return hipGetLastError();
}

// Few rows along n: small tiles.
bool small_n(int64_t n) { return n <= 128; }

template <bool TA, bool TB, int EPI> hipError_t gemm(const LossGemm& g, int splits, hipStream_t st) {
    return small_n(g.N) ? gemm_cfg<Small, TA, TB, EPI>(g, splits, st) : gemm_cfg<Big, TA, TB, EPI>(g, splits, st);
}

// Join the tiles' statistics: a block takes 8 tokens, 128 lanes for the tiles
// of each (64-byte pieces of the tiles' rows).
constexpr int JT = 8, JL = 128;
__device__ __forceinline__ float2 join(float2 a, float2 b) {  // (max, sum of exp relative to it)
    const float n = max_num(a.x, b.x), ref = n == -__builtin_inff() ? 0.0f : n;
    return make_float2(n, a.y * __expf(a.x - ref) + b.y * __expf(b.x - ref));
}
__global__ void __launch_bounds__(JT * JL) k_lse_join(const float2* __restrict__ part, int64_t ntm, int64_t T,
                                                      int64_t V, const float* __restrict__ zt,
                                                      const int64_t* __restrict__ targets, float* __restrict__ loss,
                                                      float* __restrict__ lse) {
    __shared__ float2 red[JT * JL / 64][JT];
    const int k = threadIdx.x % JT, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * JT + k;
    float2 a = make_float2(-__builtin_inff(), 0.0f);
    if (t < T)
#pragma unroll 4
        for (int64_t i = threadIdx.x / JT; i < ntm; i += JL) a = join(a, part[i * T + t]);
#pragma unroll
    for (int off = 32; off >= JT; off >>= 1)
        a = join(a, make_float2(__shfl_xor(a.x, off, 64), __shfl_xor(a.y, off, 64)));
    if ((threadIdx.x & 63) < JT) red[wave][k] = a;
    __syncthreads();
    if (threadIdx.x >= JT || t >= T) return;
    for (int w = 1; w < JT * JL / 64; ++w) a = join(a, red[w][k]);
    const float l = a.x + logf(a.y);
    const int64_t tg = targets[t];
    lse[t] = l;
    loss[t] = (uint64_t)tg < (uint64_t)V ? l - zt[t] : 0.0f;
}

// The largest |dloss| of the tokens that count; 1 where that is 0 or not finite.
__global__ void __launch_bounds__(1024) k_gscale(const float* __restrict__ dloss, const int64_t* __restrict__ targets,
                                                 int64_t T, int64_t V, float* __restrict__ out) {
    __shared__ uint32_t part[16];
    uint32_t m = 0u;
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
        const uint32_t u = as_uint(dloss[t]) & 0x7FFFFFFFu;
        if ((uint64_t)targets[t] < (uint64_t)V) m = u > m ? u : m;
    }
    m = wave_max_u32(m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i) m = part[i] > m ? part[i] : m;
        *out = m == 0u || m >= 0x7F800000u ? 1.0f : as_float(m);
    }
}

// dx = gscale * the sum of the splits, rounded once.  A thread takes 8.
__global__ void __launch_bounds__(256) k_dx_join(const float* __restrict__ part, int splits, int64_t T, int64_t H,
                                                 const float* __restrict__ gscale, uint8_t* __restrict__ dx,
                                                 int64_t ld) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, upr = H / 8;
    if (i >= T * upr) return;
    const int64_t t = i / upr, u = i - t * upr;
    float s[8] = {};
    for (int p = 0; p < splits; ++p) {
        const v4f* q = (const v4f*)(part + ((int64_t)p * T + t) * H + u * 8);
        const v4f a = q[0], b = q[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) { s[e] += a[e]; s[4 + e] += b[e]; }
    }
    const float gs = *gscale;
    *(uint4*)(dx + t * ld + u * 16) = make_uint4(pack_bf16(s[0] * gs, s[1] * gs), pack_bf16(s[2] * gs, s[3] * gs),
                                                 pack_bf16(s[4] * gs, s[5] * gs), pack_bf16(s[6] * gs, s[7] * gs));
}

// No tokens: the projection's gradient is zero.
__global__ void __launch_bounds__(256) k_zero_rows(uint8_t* __restrict__ p, int64_t rows, int64_t upr, int64_t ld) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * upr; i += (int64_t)gridDim.x * 256)
        *(uint4*)(p + i / upr * ld + i % upr * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// How the call is cut: the piece of the vocabulary whose g fits 512 MiB, and
// the splits of dx's sum over it that give every CU two tiles.
struct Plan {
    int64_t piece, pitch;   // vocabulary per piece; bytes per row of g
    int splits;
    int64_t parts, zt, gscale, g, dx, bytes;  // offsets
};
Plan plan(int64_t T, int64_t H, int64_t V, bool backward) {
    Plan p{};
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    const int64_t bm = small_n(T) ? Small::BM : Big::BM, bn = small_n(T) ? Small::BN : Big::BN;
    const int64_t fwd = up(ceil_div(V, bm) * T * 8) + up(T * 4);
    p.parts = 0;
    p.zt = up(ceil_div(V, bm) * T * 8);
    p.bytes = fwd;
    if (!backward) return p;
    const int64_t most = ((int64_t)256 << 20) / (T > 0 ? T : 1) / 256 * 256;
    p.piece = most < 2048 ? 2048 : most;
    if (p.piece > (V + 255) / 256 * 256) p.piece = (V + 255) / 256 * 256;
    p.pitch = p.piece * 2;
    const int64_t tiles = ceil_div(H, bm) * ceil_div(T > 0 ? T : 1, bn);
    int64_t s = ceil_div(512, tiles);
    const int64_t most_s = p.piece / KT / 8;  // at least eight k tiles each
    s = s > most_s ? most_s : s;
    p.splits = (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
    p.gscale = 0;
    p.g = 256;
    p.dx = p.g + up(T * p.pitch);
    const int64_t bwd = p.dx + up(p.splits * T * H * 4);
    p.bytes = bwd > fwd ? bwd : fwd;
    return p;
}

}  // namespace

int64_t lce_bytes(int64_t T, int64_t H, int64_t V, bool backward) { return plan(T, H, V, backward).bytes; }

hipError_t launch_lce(const LceArgs& a, hipStream_t st) {
    if (a.T == 0) return hipSuccess;
    const Plan p = plan(a.T, a.H, a.V, false);
    LossGemm g{};
    g.A = a.w; g.lda = a.ld_w; g.M = a.V;
    g.B = a.x; g.ldb = a.ld_x; g.N = a.T;
    g.K = a.H;
    g.m_first = 0; g.vocab = a.V;
    g.targets = a.targets;
    g.part = (float2*)(a.ws + p.parts);
    g.zt = (float*)(a.ws + p.zt);
    hipError_t e = gemm<false, false, EPI_LSE>(g, 1, st);
    if (e != hipSuccess) return e;
    const int64_t ntm = ceil_div(a.V, small_n(a.T) ? Small::BM : Big::BM);
    k_lse_join<<<(unsigned)ceil_div(a.T, JT), JT * JL, 0, st>>>(g.part, ntm, a.T, a.V, g.zt, a.targets, a.loss, a.lse);
    return hipGetLastError();
}

hipError_t launch_lce_backward(const LceArgs& a, hipStream_t st) {
    if (a.T == 0) {
        if (a.dw) k_zero_rows<<<1024, 256, 0, st>>>(a.dw, a.V, a.H / 8, a.ld_dw);
        return hipGetLastError();
    }
    const Plan p = plan(a.T, a.H, a.V, true);
    float* gscale = (float*)(a.ws + p.gscale);
    k_gscale<<<1, 1024, 0, st>>>(a.dloss, a.targets, a.T, a.V, gscale);
    for (int64_t v0 = 0; v0 < a.V; v0 += p.piece) {
        const int64_t n = a.V - v0 < p.piece ? a.V - v0 : p.piece;
        LossGemm g{};
        g.A = a.w + v0 * a.ld_w; g.lda = a.ld_w; g.M = n;
        g.B = a.x; g.ldb = a.ld_x; g.N = a.T;
        g.K = a.H;
        g.m_first = v0; g.vocab = a.V;
        g.targets = a.targets; g.lse = a.lse_in; g.dloss = a.dloss; g.gscale = gscale;
        g.out = a.ws + p.g; g.ldo = p.pitch;
        g.m_store = (n + 63) / 64 * 64;  // zeros to the end of the last k tile of dx's product
        hipError_t e = gemm<false, false, EPI_G>(g, 1, st);
        if (e != hipSuccess) return e;
        if (a.dx) {
            LossGemm d{};
            d.A = a.w + v0 * a.ld_w; d.lda = a.ld_w; d.M = a.H;
            d.B = a.ws + p.g; d.ldb = p.pitch; d.N = a.T;
            d.K = n;
            d.out = a.ws + p.dx; d.ldo = a.H * 4;
            d.add = v0 > 0;
            e = gemm<true, false, EPI_DX>(d, p.splits, st);
            if (e != hipSuccess) return e;
        }
        if (a.dw) {
            LossGemm d{};
            d.A = a.x; d.lda = a.ld_x; d.M = a.H;
            d.B = a.ws + p.g; d.ldb = p.pitch; d.N = n;
            d.K = a.T;
            d.gscale = gscale;
            d.out = a.dw + v0 * a.ld_dw; d.ldo = a.ld_dw;
            e = gemm<true, true, EPI_DW>(d, 1, st);
            if (e != hipSuccess) return e;
        }
    }
    if (a.dx)
        k_dx_join<<<(unsigned)ceil_div(a.T * (a.H / 8), 256), 256, 0, st>>>((const float*)(a.ws + p.dx), p.splits, a.T,
                                                                          a.H, gscale, a.dx, a.ld_dx);
    return hipGetLastError();
}

}  // namespace mxq
