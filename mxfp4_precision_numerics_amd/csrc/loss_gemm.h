// loss_gemm.h - the matrix products of the vocabulary cross entropy: bf16_gemm.h
// with the loss's own epilogues.  With m the vocabulary and n the tokens a softmax
// over the vocabulary is a reduction inside lanes.
#pragma once
#include "bf16_gemm.h"
#include "train_launch.h"

namespace mxq {

enum { EPI_LSE = 0, EPI_G = 1, EPI_DX = 2, EPI_DW = 3 };

struct LossGemm : GemmBf16 {
    int64_t m_first, vocab;  // vocabulary index of m = 0, and its size (EPI_LSE, EPI_G)
    const int64_t* targets;
    float2* part;          // EPI_LSE: [ntm][N] (max, sum of exp)
    float* zt;             // EPI_LSE: the targets' logits
    const float *lse, *dloss;
    float* gscale;         // EPI_G, EPI_DW: the largest |dloss|
    int own_scale;         // EPI_G: find it, and leave it there for the next launches
    uint8_t* out;          // EPI_G, EPI_DW: bf16 rows; EPI_DX: fp32 [splits][N][M]
    int64_t ldo;           // bytes
    int64_t m_store;       // EPI_G: columns written per row (zeros at and past M)
    int add;               // EPI_DX: add to what is there
};

constexpr float LOG2E = 1.44269504f;
// e^(z - ref), ref at or above z (but for rounding).  The difference is taken
// before it is scaled: a logit equal to ref gives exactly 1, the others no more,
// so that a sum is at least 1, lse no less than the largest logit and a loss not
// negative.  (exp2(fma(z, log2 e, -ref log2 e)) is an instruction less, 0.3% of
// 8192 tokens x 4096 x 131072 and 0.7% of 3155 x 264 x 85226 forward and
// gradients, but keeps the rounding of ref log2 e: lse up to 6e-5 too low at
// logits of 700, and nothing right above 1e9.)
__device__ __forceinline__ float exp_below(float z, float ref) { return __builtin_amdgcn_exp2f((z - ref) * LOG2E); }
// The larger number; a NaN is passed over.
__device__ __forceinline__ float max_num(float a, float b) {
    return __builtin_amdgcn_fmed3f(a, b, __builtin_inff());
}

// Epilogues on the accumulators of a wave (of the first group of waves; the
// others of WGK pass its barriers and help to store).
template <int BM, int BN, int WGM, int WGN, int EPI, bool HALVES = false, int WGK = 1>
__device__ __forceinline__ void loss_epilogue(const LossGemm& g, const GemmTile& t, float gscale,
                                              v4f (&acc)[BM / WGM / 16][BN / WGN / 16], uint8_t* smem, int tid) {
    constexpr int FM = BM / WGM / 16, FN = BN / WGN / 16, NT = 64 * WGM * WGN * WGK;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WGN, wn = wave % WGN;
    const bool on = WGK == 1 || wave < WGM * WGN;
    using PM = FragPlace<BM, WGM, HALVES>;
    using PN = FragPlace<BN, WGN, HALVES>;
    const int wrow = PM::base(wm) + 4 * (lane >> 4), wcol = PN::base(wn) + (lane & 15);
    const int64_t mb = t.m0 + wrow;  // + PM::at(i, wm) + r
    if constexpr (EPI == EPI_LSE) {
        float2* red = (float2*)smem;  // [WGM][BN]
        const bool whole = t.m0 + BM <= g.M;
        if (on)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int col = wcol + PN::at(j, wn);
            const int64_t n = t.n0 + col;
            const int64_t want = (n < g.N ? g.targets[n] : -1) - g.m_first - mb;  // relative to this lane's rows
            if (__any(want >= 0 && want < BM)) {  // rare in a large vocabulary
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int d = PM::at(i, wm) + r;
                        if (want == d && mb + d < g.M) g.zt[n] = acc[i][j][r];
                    }
            }
            if (!whole) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (mb + PM::at(i, wm) + r >= g.M) acc[i][j][r] = -__builtin_inff();
            }
            float mx = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = max_num(acc[i][j][r], mx);
            mx = max_num(__shfl_xor(mx, 16, 64), mx);
            mx = max_num(__shfl_xor(mx, 32, 64), mx);
            const float ref = mx == -__builtin_inff() ? 0.0f : mx;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) s += exp_below(acc[i][j][r], ref);
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            if (lane < 16) red[wm * BN + col] = make_float2(mx, s);  // (-inf, 0) if no row is inside
        }
        __syncthreads();
        for (int c = tid; c < BN; c += NT) {
            const int64_t n = t.n0 + c;
            if (n >= g.N) continue;
            float m = red[c].x, s;
#pragma unroll
            for (int w = 1; w < WGM; ++w) m = red[w * BN + c].x > m ? red[w * BN + c].x : m;
            s = 0.0f;
            const float ref = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
            for (int w = 0; w < WGM; ++w) s = fmaf(red[w * BN + c].y, __expf(red[w * BN + c].x - ref), s);
            g.part[(t.m0 / BM) * g.N + n] = make_float2(m, s);
        }
    } else if constexpr (EPI == EPI_DX) {
        // buffer accesses, whose range check takes the place of a branch for
        // rows and columns past the end (branches around each access spilled
        // the accumulators)
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
            g.out + ((int64_t)t.split * g.N + t.n0) * g.ldo + t.m0 * 4, 0, (int)EXTENT, 0x00020000);
        if (on)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int col = wcol + PN::at(j, wn);
            uint32_t off[FM];
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int m = wrow + PM::at(i, wm);  // M % 8 == 0: the four are in or out together
                off[i] = t.n0 + col < g.N && t.m0 + m < g.M ? (uint32_t)(col * g.ldo) + 4 * m : NOWHERE;
            }
            if (g.add) {  // every load of the column before its first store
                v4f old[FM];
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    old[i] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off[i], 0, 0));
#pragma unroll
                for (int i = 0; i < FM; ++i) acc[i][j] += old[i];
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, acc[i][j]), rsrc, off[i], 0, 0);
        }
    } else {
        // bf16 rows through LDS: [BN][BM], rows padded by 16 bytes
        constexpr int RB = BM * 2 + 16;
        const bool whole = t.m0 + BM <= g.M;
        if (on)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int col = wcol + PN::at(j, wn);
            const int64_t n = t.n0 + col;
            float r = gscale, ref = 0.0f;
            int64_t want = -1;
            if constexpr (EPI == EPI_G) {
                r = 0.0f;
                if (n < g.N) {
                    const int64_t tg = g.targets[n];
                    ref = g.lse[n];
                    r = (uint64_t)tg < (uint64_t)g.vocab ? g.dloss[n] / gscale : 0.0f;
                    want = tg - g.m_first - mb;
                }
                // exp(z - lse) r, where r = 0 gives 0 whatever the logits are
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = exp_below(acc[i][j][e], ref);
                if (!whole || __any(want >= 0 && want < BM)) {
#pragma unroll
                    for (int i = 0; i < FM; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int d = PM::at(i, wm) + e;
                            if (want == d) acc[i][j][e] -= 1.0f;
                            if (mb + d >= g.M) acc[i][j][e] = 0.0f;
                        }
                }
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = EPI == EPI_G && r == 0.0f ? 0.0f : acc[i][j][e] * r;
                const int m = wrow + PM::at(i, wm);
                *(uint2*)(smem + col * RB + m * 2) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            }
        }
        __syncthreads();
        const int64_t cols = EPI == EPI_G ? g.m_store : g.M;
        constexpr int CPR = BM / 8;  // 16-byte chunks per row
        for (int c = tid; c < BN * CPR; c += NT) {
            const int row = c / CPR, ch = c % CPR;
            const int64_t n = t.n0 + row, m = t.m0 + ch * 8;
            if (n >= g.N || m >= cols) continue;
            const uint4 v = *(const uint4*)(smem + row * RB + ch * 16);
            uint8_t* to = g.out + n * g.ldo + m * 2;
            if constexpr (EPI == EPI_DW) st_nt16(to, v);  // plain: 8% more at 48 tokens x 4096 x 131072
            else *(uint4*)to = v;
        }
    }
}

// The largest |dloss| of the tokens that count; 1 where that is 0 or not
// finite.  Every thread of the block returns it.
template <int NT>
__device__ __forceinline__ float largest_dloss(const float* dloss, const int64_t* targets, int64_t T, int64_t V) {
    __shared__ uint32_t part[NT / 64];
    uint32_t m = 0u;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < T; t += NT) {
        const uint32_t u = as_uint(dloss[t]) & 0x7FFFFFFFu;
        if ((uint64_t)targets[t] < (uint64_t)V) m = u > m ? u : m;
    }
    m = wave_max_u32(m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = part[0];
    for (int i = 1; i < NT / 64; ++i) m = part[i] > m ? part[i] : m;
    return m == 0u || m >= 0x7F800000u ? 1.0f : as_float(m);
}

template <int EPI> struct LossEpi {
    using Args = LossGemm;
    static constexpr bool PAIRED = false, STREAMS = false;
    template <int NT> static __device__ __forceinline__ float before(const LossGemm& g, uint32_t block, int tid) {
        float gscale = 1.0f;
        if constexpr (EPI == EPI_DW) gscale = *g.gscale;
        if constexpr (EPI == EPI_G) {
            gscale = g.own_scale ? largest_dloss<NT>(g.dloss, g.targets, g.N, g.vocab) : *g.gscale;
            if (g.own_scale && block == 0 && tid == 0) *g.gscale = gscale;
        }
        return gscale;
    }
    static __device__ __forceinline__ float after(const LossGemm& g) {
        return EPI == EPI_G || EPI == EPI_DW ? *g.gscale : 1.0f;
    }
    template <int BM, int BN, int WGM, int WGN, bool HALVES, int WGK>
    static __device__ __forceinline__ void finish(const LossGemm& g, const GemmTile& t, float gscale,
                                                  v4f (&acc)[BM / WGM / 16][BN / WGN / 16], uint8_t* smem, int tid) {
        loss_epilogue<BM, BN, WGM, WGN, EPI, HALVES, WGK>(g, t, gscale, acc, smem, tid);
    }
};

template <class C, bool TA, bool TB, int EPI>
__global__ void __launch_bounds__(threads_of<C>()) k_loss_gemm(const LossGemm g) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LdsOf<C>::BYTES];
    gemm_plain<C::BM, C::BN, C::WGM, C::WGN, C::WGK, C::NSL, TA, TB, LossEpi<EPI>>(g, g.first + blockIdx.x, smem);
}

// dx's and dw's products of a piece in one launch: both wait for g alone.
template <class X, class W>
__global__ void __launch_bounds__(threads_of<X>()) k_loss_grads(const LossGemm x, const LossGemm w, uint32_t nx) {
    static_assert(threads_of<X>() == threads_of<W>(), "one block size");
    constexpr int BYTES = LdsOf<X>::BYTES > LdsOf<W>::BYTES ? LdsOf<X>::BYTES : LdsOf<W>::BYTES;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[BYTES];
    if (blockIdx.x < nx)
        gemm_plain<X::BM, X::BN, X::WGM, X::WGN, X::WGK, X::NSL, true, false, LossEpi<EPI_DX>>(x, blockIdx.x, smem);
    else
        gemm_plain<W::BM, W::BN, W::WGM, W::WGN, W::WGK, W::NSL, true, true, LossEpi<EPI_DW>>(w, blockIdx.x - nx, smem);
}
template <int BM, bool TA, bool TB, int EPI>
__global__ void __launch_bounds__(512) k_loss_gemm_pipe(const LossGemm g) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[GemmLds<256, 256, 2>::BYTES];
    gemm_pipe<BM, TA, TB, LossEpi<EPI>>(g, g.first + blockIdx.x, smem);
}

}  // namespace mxq
