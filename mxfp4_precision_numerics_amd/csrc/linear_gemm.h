// linear_gemm.h - linear and gated layers: the products of bf16_gemm.h with bias,
// activation, product of a pair and residual in their epilogue.
#pragma once
#include "bf16_gemm.h"
#include "dense_launch.h"

namespace mxq {

struct LinearGemm : GemmBf16 {
    int act;
    const float* bias;       // [M], or nullptr
    const uint8_t* residual; // [N][M] of the output's type, or nullptr
    int64_t ldr;             // bytes, as every pitch here
    uint8_t* out;            // [N][M], paired [N][pairs] (with dh: [N][2 pairs]); fp32 or bf16
    int64_t ldo;
    int f32;                 // out (and residual) are fp32
    uint8_t* z;              // bf16 [N][M], paired [N][2 pairs]: the sums before the activation, or nullptr
    int64_t ldz;
    const uint8_t* dh;       // paired: bf16 [N][pairs], and out takes the gradients of the pair's sums
    int64_t ldh;
    float* part;             // splits > 1: fp32 [splits][N][M], joined by k_linear_join
};

__device__ __forceinline__ uint32_t pack2(float a, float b) { return pack_bf16(a, b); }
__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = as_float(u[k] << 16);
        f[2 * k + 1] = as_float(u[k] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// 1 / (1 + e^-z) from e^-|z|, which cannot overflow.
__device__ __forceinline__ float sigmoid(float z) {
    const float e = expf(-__builtin_fabsf(z));
    return (z < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
}
constexpr float TANH_A = 1.59576912f, TANH_B = 0.044715f;  // 2 sqrt(2 / pi)
// act(z) and, D, act'(z).  The tanh form of the GELU is z sigmoid(2 u), u the
// tanh's argument: its lower tail keeps its precision, as erfc keeps the other's.
template <int ACT, bool D> __device__ __forceinline__ float2 activation(float z) {
    if constexpr (ACT == MXQ_ACT_RELU) {
        return make_float2(z <= 0.0f ? 0.0f : z, z <= 0.0f ? 0.0f : 1.0f);  // a NaN stays one
    } else if constexpr (ACT == MXQ_ACT_SILU) {
        const float p = sigmoid(z);
        return make_float2(z * p, D ? p * fmaf(z, sigmoid(-z), 1.0f) : 0.0f);
    } else if constexpr (ACT == MXQ_ACT_GELU) {
        const float q = 0.5f * erfcf(__builtin_fabsf(z) * 0.70710678f), p = z < 0.0f ? q : 1.0f - q;
        return make_float2(z * p, D ? fmaf(z, 0.39894228f * expf(-0.5f * z * z), p) : 0.0f);
    } else if constexpr (ACT == MXQ_ACT_GELU_TANH) {
        const float u = TANH_A * fmaf(TANH_B * z * z, z, z), p = sigmoid(u);
        return make_float2(z * p,
                           D ? fmaf(z * p * sigmoid(-u), TANH_A * fmaf(3.0f * TANH_B * z, z, 1.0f), p) : 0.0f);
    } else {
        return make_float2(z, 1.0f);
    }
}
// f(integral_constant<int, act>), act being the same for every thread
template <class F> __device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case MXQ_ACT_RELU: f(std::integral_constant<int, MXQ_ACT_RELU>()); break;
        case MXQ_ACT_SILU: f(std::integral_constant<int, MXQ_ACT_SILU>()); break;
        case MXQ_ACT_GELU: f(std::integral_constant<int, MXQ_ACT_GELU>()); break;
        case MXQ_ACT_GELU_TANH: f(std::integral_constant<int, MXQ_ACT_GELU_TANH>()); break;
        default: f(std::integral_constant<int, MXQ_ACT_NONE>());
    }
}

// What an output chunk (8 of a row) reads besides its sums; loaded for several
// chunks before the first of them is stored.
struct Beside { uint4 lo, hi; };
template <bool PAIRED> __device__ __forceinline__ Beside load_beside(const LinearGemm& g, int64_t n, int64_t m) {
    Beside b{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if constexpr (PAIRED) {
        if (g.dh) b.lo = *(const uint4*)(g.dh + n * g.ldh + m * 2);
    } else if (g.residual) {
        const uint8_t* r = g.residual + n * g.ldr + m * (g.f32 ? 4 : 2);
        b.lo = *(const uint4*)r;
        if (g.f32) b.hi = *(const uint4*)(r + 16);
    }
    return b;
}
__device__ __forceinline__ void store8(const LinearGemm& g, int64_t n, int64_t m, const float (&v)[8]) {
    if (g.f32) {
        uint4* o = (uint4*)(g.out + n * g.ldo + m * 4);
        o[0] = make_uint4(as_uint(v[0]), as_uint(v[1]), as_uint(v[2]), as_uint(v[3]));
        o[1] = make_uint4(as_uint(v[4]), as_uint(v[5]), as_uint(v[6]), as_uint(v[7]));
    } else {
        *(uint4*)(g.out + n * g.ldo + m * 2) = pack8(v);
    }
}
// Chunk (n, m .. m + 7) of a linear layer from its sums.  PLAIN: neither bias nor activation.
template <bool PLAIN>
__device__ __forceinline__ void finish_linear(const LinearGemm& g, int64_t n, int64_t m, float (&v)[8], const Beside& b) {
    if constexpr (!PLAIN) {
        if (g.bias) {
            const float4 lo = *(const float4*)(g.bias + m), hi = *(const float4*)(g.bias + m + 4);
            const float c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += c[k];
        }
        if (g.z) st_nt16(g.z + n * g.ldz + m * 2, pack8(v));
        with_act(g.act, [&](auto a) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = activation<decltype(a)::value, false>(v[k]).x;
        });
    }
    if (g.residual) {
        float r[8];
        if (g.f32) {
            const uint32_t u[8] = {b.lo.x, b.lo.y, b.lo.z, b.lo.w, b.hi.x, b.hi.y, b.hi.z, b.hi.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = as_float(u[k]);
        } else {
            unpack8(b.lo, r);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += r[k];
    }
    store8(g, n, m, v);
}
// dgate = dh up act'(gate), dup = dh act(gate)
template <int ACT>
__device__ __forceinline__ void gated_gradient(float (&gate)[8], float (&up)[8], const float (&dh)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 a = activation<ACT, true>(gate[k]);
        gate[k] = dh[k] * up[k] * a.y;
        up[k] = dh[k] * a.x;
    }
}
// Chunk (n, features m .. m + 7) of a gated layer.
__device__ __forceinline__ void finish_gated(const LinearGemm& g, int64_t n, int64_t m, float (&gate)[8], float (&up)[8],
                                             const Beside& b) {
    if (g.dh) {
        float dh[8];
        unpack8(b.lo, dh);
        with_act(g.act, [&](auto a) { gated_gradient<decltype(a)::value>(gate, up, dh); });
        *(uint4*)(g.out + n * g.ldo + m * 2) = pack8(gate);
        *(uint4*)(g.out + n * g.ldo + (m + g.pairs) * 2) = pack8(up);
        return;
    }
    if (g.z) {
        st_nt16(g.z + n * g.ldz + m * 2, pack8(gate));
        st_nt16(g.z + n * g.ldz + (m + g.pairs) * 2, pack8(up));
    }
    with_act(g.act, [&](auto a) {
#pragma unroll
        for (int k = 0; k < 8; ++k) gate[k] = activation<decltype(a)::value, false>(gate[k]).x * up[k];
    });
    *(uint4*)(g.out + n * g.ldo + m * 2) = pack8(gate);
}

// The epilogue.  The sums go through LDS in bands, one fragment column of every
// wave at a time, in two buffers, so that a thread has 8 consecutive m of a row:
// residuals, sums before the activation and outputs move 16 or 32 bytes at a
// time, and a chunk's work is the same here, in the join and for few rows.
template <bool PAIR, bool PLAIN, bool STREAM = false> struct LinearEpi {
    using Args = LinearGemm;
    static constexpr bool PAIRED = PAIR, STREAMS = STREAM;
    template <int NT> static __device__ __forceinline__ float before(const LinearGemm&, uint32_t, int) { return 0.0f; }
    static __device__ __forceinline__ float after(const LinearGemm&) { return 0.0f; }
    template <int BM, int BN, int WGM, int WGN, bool HALVES, int WGK>
    static __device__ __forceinline__ void finish(const LinearGemm& g, const GemmTile& t, float,
                                                  v4f (&acc)[BM / WGM / 16][BN / WGN / 16], uint8_t* smem, int tid) {
        constexpr int FM = BM / WGM / 16, FN = BN / WGN / 16, NT = 64 * WGM * WGN * WGK;
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WGN, wn = wave % WGN;
        const bool on = WGK == 1 || wave < WGM * WGN;
        using PM = FragPlace<BM, WGM, HALVES>;
        using PN = FragPlace<BN, WGN, HALVES>;
        const int wrow = PM::base(wm) + 4 * (lane >> 4), wcol = PN::base(wn) + (lane & 15);
        int64_t m_end = g.M;
        if constexpr (STREAM) m_end = t.m0 + g.stride < g.M ? t.m0 + g.stride : g.M;
        if (g.part) {  // buffer stores, whose range check takes the place of a branch for rows and columns past the end
            const int64_t ld = g.M * 4;
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
                (uint8_t*)g.part + ((int64_t)t.split * g.N + t.n0) * ld + t.m0 * 4, 0, (int)EXTENT, 0x00020000);
            if (on)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int col = wcol + PN::at(j, wn);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const int m = wrow + PM::at(i, wm);  // M % 8 == 0: the four are in or out together
                    const uint32_t off = t.n0 + col < g.N && t.m0 + m < m_end ? (uint32_t)(col * ld) + 4 * m : NOWHERE;
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, acc[i][j]), rsrc, off, 0, 0);
                }
            }
            return;
        }
        constexpr int ROWS = 16 * WGN, RB = BM * 4 + 16, BAND = ROWS * RB;  // of a band; bytes of a row, of a band
        constexpr int CPR = PAIR ? BM / 16 : BM / 8;                        // chunks of a row
        constexpr int EACH = (ROWS * CPR + NT - 1) / NT;
        const int64_t width = PAIR ? m_end / 2 : m_end, m0 = PAIR ? t.m0 / 2 : t.m0;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            uint8_t* buf = smem + (j & 1) * BAND;
            if (on)
#pragma unroll
            for (int i = 0; i < FM; ++i)
                *(v4f*)(buf + (wn * 16 + (lane & 15)) * RB + (wrow + PM::at(i, wm)) * 4) = acc[i][j];
            Beside beside[EACH];
            int64_t ns[EACH], ms[EACH];
#pragma unroll
            for (int e = 0; e < EACH; ++e) {
                const int c = tid + e * NT, row = c / CPR, w = row >> 4;
                ns[e] = t.n0 + PN::base(w) + PN::at(j, w) + (row & 15);
                ms[e] = m0 + c % CPR * 8;
                if ((ROWS * CPR % NT != 0 && c >= ROWS * CPR) || ns[e] >= g.N || ms[e] >= width) ns[e] = -1;
                if (ns[e] >= 0) beside[e] = load_beside<PAIR>(g, ns[e], ms[e]);
            }
            __syncthreads();  // the band is written; the one before the last has been read
#pragma unroll
            for (int e = 0; e < EACH; ++e) {
                if (ns[e] < 0) continue;
                const int c = tid + e * NT, row = c / CPR, ch = c % CPR;
                const uint8_t* p = buf + row * RB + ch * (PAIR ? 64 : 32);
                float v[8];
                *(v4f*)v = *(const v4f*)p;
                *(v4f*)(v + 4) = *(const v4f*)(p + 16);
                if constexpr (PAIR) {
                    float u[8];
                    *(v4f*)u = *(const v4f*)(p + 32);
                    *(v4f*)(u + 4) = *(const v4f*)(p + 48);
                    finish_gated(g, ns[e], ms[e], v, u, beside[e]);
                } else {
                    finish_linear<PLAIN>(g, ns[e], ms[e], v, beside[e]);
                }
            }
        }
    }
};

template <int BM, int WGN> constexpr int band_bytes() { return 2 * 16 * WGN * (BM * 4 + 16); }
template <class C, bool TA, bool TB, bool PAIR>
__global__ void __launch_bounds__(threads_of<C>()) k_linear_gemm(const LinearGemm g) {
    static_assert(band_bytes<C::BM, C::WGN>() <= LdsOf<C>::BYTES, "the epilogue's bands");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LdsOf<C>::BYTES];
    gemm_plain<C::BM, C::BN, C::WGM, C::WGN, C::WGK, C::NSL, TA, TB, LinearEpi<PAIR, TA>>(g, g.first + blockIdx.x, smem);
}
template <int BM, bool TA, bool TB, bool PAIR>
__global__ void __launch_bounds__(512) k_linear_pipe(const LinearGemm g) {
    static_assert(band_bytes<BM, 4>() <= GemmLds<256, 256, 2>::BYTES, "the epilogue's bands");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[GemmLds<256, 256, 2>::BYTES];
    gemm_pipe<BM, TA, TB, LinearEpi<PAIR, TA>>(g, g.first + blockIdx.x, smem);
}

// Tiles for few tokens (k contiguous operands), tile numbers from 16 on.  The weights' bytes
// bound them: many copies in flight, STREAMS.
struct Wide64 { static constexpr int BM = 128, BN = 64, WGM = 4, WGN = 2, WGK = 1, NSL = 6; };
struct Wide32 { static constexpr int BM = 128, BN = 32, WGM = 4, WGN = 1, WGK = 1, NSL = 8; };
struct Wide128 { static constexpr int BM = 128, BN = 128, WGM = 4, WGN = 2, WGK = 1, NSL = 5; };
struct Quick32 { static constexpr int BM = 32, BN = 32, WGM = 2, WGN = 2, WGK = 2, NSL = 5; };
struct Quick64 { static constexpr int BM = 32, BN = 64, WGM = 2, WGN = 2, WGK = 2, NSL = 6; };
enum { WIDE64 = 16, WIDE32, WIDE128, QUICK32, QUICK64 };
template <class C, bool PAIR> __global__ void __launch_bounds__(threads_of<C>()) k_linear_stream(const LinearGemm g) {
    static_assert(band_bytes<C::BM, C::WGN>() <= LdsOf<C>::BYTES, "the epilogue's bands");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LdsOf<C>::BYTES];
    gemm_plain<C::BM, C::BN, C::WGM, C::WGN, C::WGK, C::NSL, false, false, LinearEpi<PAIR, false, true>>(
        g, g.first + blockIdx.x, smem);
}
// The product's form: operands k contiguous; A transposed; both transposed; A's rows paired.
enum { FORM_NN = 0, FORM_TN = 1, FORM_TT = 2, FORM_PAIRED = 3 };
template <int FORM> hipError_t linear_gemm(const LinearGemm& g, int tile, int splits, hipStream_t st);

}  // namespace mxq
