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
    int nt;                  // out is not read again soon
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

constexpr float LOG2_E = 1.44269504f;
// 1 / (1 + e^-z); 0 where e^-z passes binary32's range.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -LOG2_E));
}
// Phi(z) and, as .y, e^(-z^2 / 2).  Phi(-|z|) = e^(-z^2 / 2) R(|z|), R falling from 1/2 as 1 / |z|: t Q(t), t = 1 / (1 + c |z|), c
// and Q's seven coefficients fitted for the least relative error up to |z| = 13.2, beyond which the product is subnormal,
// weighted so that it grows as the exponential's own: 1.8e-7 + 2.4e-8 z^2 at most.  With the roundings to binary32 Phi(-|z|) is off
// by 8e-7 of its value up to 3, 3e-6 up to 8 and 1e-5 at 13, where a fit of the least absolute error (five coefficients) was off by
// 0.4% at 6 and 4% at 13, many steps of bf16.
__device__ __forceinline__ float2 normal(float z) {
    const float a = __builtin_fabsf(z), e = __builtin_amdgcn_exp2f(z * z * (-0.5f * LOG2_E));
    const float t = __builtin_amdgcn_rcpf(fmaf(a, 0.258962314f, 1.0f));
    float q = fmaf(t, -0.0764350050f, 0.245476727f);
    q = fmaf(t, q, -0.129486216f);
    q = fmaf(t, q, 0.182859706f);
    q = fmaf(t, q, 0.0665360478f);
    q = fmaf(t, q, 0.108047444f);
    q = fmaf(t, q, 0.103001208f) * t * e;
    return make_float2(z < 0.0f ? q : 1.0f - q, e);
}
constexpr float TANH_A = 1.59576912f, TANH_B = 0.044715f;  // 2 sqrt(2 / pi)
// act(z) and, D, act'(z).  The tanh form of the GELU is z sigmoid(2 u), u the
// tanh's argument, so that its lower tail keeps its precision.  Its slope p + z p (1 - p) 2 u' is p to the last bit beyond
// 16 of either sign, where p (1 - p) vanishes and z u' need not fit binary32: z and u' are taken there.
template <int ACT, bool D> __device__ __forceinline__ float2 activation(float z) {
    if constexpr (ACT == MXQ_ACT_RELU) {
        return make_float2(z <= 0.0f ? 0.0f : z, z <= 0.0f ? 0.0f : 1.0f);  // a NaN stays one
    } else if constexpr (ACT == MXQ_ACT_SILU) {
        const float p = sigmoid(z);
        return make_float2(z * p, D ? p * fmaf(z, 1.0f - p, 1.0f) : 0.0f);
    } else if constexpr (ACT == MXQ_ACT_GELU) {
        const float2 n = normal(z);
        return make_float2(z * n.x, D ? fmaf(z, 0.39894228f * n.y, n.x) : 0.0f);
    } else if constexpr (ACT == MXQ_ACT_GELU_TANH) {
        const float p = sigmoid(TANH_A * fmaf(TANH_B * z * z, z, z));
        const float c = __builtin_amdgcn_fmed3f(z, -16.0f, 16.0f);
        return make_float2(z * p, D ? fmaf(c * p * (1.0f - p), TANH_A * fmaf(3.0f * TANH_B * c, c, 1.0f), p) : 0.0f);
    } else {
        return make_float2(z, 1.0f);
    }
}
// f(integral_constant<int, act>), act being the same for every thread (KNOWN >= 0: it is that)
template <int KNOWN = -1, class F> __device__ __forceinline__ void with_act(int act, F f) {
    if constexpr (KNOWN >= 0) f(std::integral_constant<int, KNOWN>());
    else switch (act) {
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

// The epilogue works on the sums in registers, a lane's four consecutive m of a row
// n, then lays the tile out in LDS in the output's type, 16-byte chunks XOR-ed with the
// row, and stores whole rows of it.  (The same on chunks of 8 behind an LDS tile of binary32: 12 us of a 256 x 256 tile before its
// stores, most of them addresses, against 3.)
// (the XOR stays within the row: within runs of a power of two that its chunks divide into)
template <int RB> constexpr int tile_mask() { return ((RB / 16) & -(RB / 16)) < 16 ? ((RB / 16) & -(RB / 16)) - 1 : 15; }
template <int RB> __device__ __forceinline__ int tile_at(int row, int chunk) {
    return row * RB + ((chunk ^ (row & tile_mask<RB>())) << 4);
}
struct OutTile {
    uint8_t* p;       // of the tile's first element
    int64_t ld;
    int rows, chunks; // inside the matrix; chunks: 16 bytes
    uint32_t apart;   // PAIRS: bytes from a gate's chunk to its up's
};
// ROWS rows of an LDS tile to memory.  PAIRS: chunks alternate between the two halves of a row.  NT: not read again soon.
template <int ROWS, int RB, int NTH, bool PAIRS, bool NTS>
__device__ __forceinline__ void store_tile(const OutTile& o, const uint8_t* smem, int tid) {
    constexpr int CPR = RB / 16;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(o.p, 0, (int)EXTENT, 0x00020000);
#pragma unroll
    for (int k = 0; k < (ROWS * CPR + NTH - 1) / NTH; ++k) {
        const int c = tid + k * NTH, row = c / CPR, ch = c % CPR;
        if (ROWS * CPR % NTH != 0 && c >= ROWS * CPR) break;
        const v4u v = *(const v4u*)(smem + tile_at<RB>(row, ch));
        uint32_t off = __umul24((uint32_t)row, (uint32_t)o.ld) + (PAIRS ? (ch >> 1) * 16 + (ch & 1) * o.apart : ch * 16);
        off = row < o.rows && ch < o.chunks ? off : NOWHERE;
        __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, off, 0, NTS ? 2 : 0);
    }
}

// PLAIN: neither bias nor activation.  STREAM: see GemmBf16.  ACT >= 0: the activation.  GRAD: paired with dh (1) or
// without (0).  The large tiles' kernels know both: with all of them in one kernel its epilogue spilled.
template <bool PAIR, bool PLAIN, bool STREAM = false, int ACT = -1, int GRAD = -1> struct LinearEpi {
    using Args = LinearGemm;
    static constexpr bool PAIRED = PAIR, STREAMS = STREAM;
    template <int NT> static __device__ __forceinline__ float before(const LinearGemm&, uint32_t, int) { return 0.0f; }
    static __device__ __forceinline__ float after(const LinearGemm&) { return 0.0f; }
    // With a residual: its rows are copied to where the outputs go in LDS, lanes add their sums in place, and rows are
    // stored; binary32 in two passes where the tile's rows come in halves of 128.
    template <int ES, int BM, int BN, int WGM, int WGN, bool HALVES, int WGK>
    static __device__ __forceinline__ void add_and_store(const LinearGemm& g, const GemmTile& t,
                                                         v4f (&acc)[BM / WGM / 16][BN / WGN / 16], uint8_t* smem, int tid,
                                                         int rows, int cols) {
        constexpr int FM = BM / WGM / 16, FN = BN / WGN / 16, NT = 64 * WGM * WGN * WGK;
        constexpr int PASSES = HALVES && ES == 4 ? 2 : 1, FP = FN / PASSES, ROWS = BN / PASSES;
        constexpr int RB = BM * ES, CPR = RB / 16, PIECES = ROWS * RB / 1024;
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WGN, wn = wave % WGN;
        const bool on = WGK == 1 || wave < WGM * WGN;
        using PM = FragPlace<BM, WGM, HALVES>;
        using PN = FragPlace<BN, WGN, HALVES>;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int left = rows - p * ROWS;
            const int64_t n0 = t.n0 + p * ROWS;
            const v4u from = make_rsrc(g.residual + n0 * g.ldr + t.m0 * ES, EXTENT);
            if (p) __syncthreads();  // the first half has been read
#pragma unroll
            for (int k = 0; k < (PIECES + NT / 64 - 1) / (NT / 64); ++k) {
                const int piece = wave + k * (NT / 64);
                if (PIECES % (NT / 64) != 0 && piece >= PIECES) break;
                const int c = piece * 64 + lane, r = c / CPR, ch = c % CPR ^ (r & tile_mask<RB>());
                const uint32_t off = r < left && ch * (16 / ES) < cols ? __umul24((uint32_t)r, (uint32_t)g.ldr) + ch * 16 : NOWHERE;
                dma16(from, off, 0u, lds_addr(smem) + (uint32_t)piece * 1024u);
            }
            __builtin_amdgcn_s_waitcnt(wait_vm(0));
            __syncthreads();
            if (on)
#pragma unroll
            for (int j = p * FP; j < (p + 1) * FP; ++j)
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const int r = PN::base(wn) + (lane & 15) + PN::at(j, wn) - p * ROWS;
                    const int m = PM::base(wm) + 4 * (lane >> 4) + PM::at(i, wm);
                    if constexpr (ES == 4) {
                        v4f* at = (v4f*)(smem + tile_at<RB>(r, m >> 2));
                        *at = acc[i][j] + *at;
                    } else {
                        uint2* at = (uint2*)(smem + tile_at<RB>(r, m >> 3) + (m >> 2 & 1) * 8);
                        const uint2 v = *at;
                        *at = make_uint2(pack2(acc[i][j][0] + as_float(v.x << 16), acc[i][j][1] + as_float(v.x & 0xFFFF0000u)),
                                         pack2(acc[i][j][2] + as_float(v.y << 16), acc[i][j][3] + as_float(v.y & 0xFFFF0000u)));
                    }
                }
            __syncthreads();
            store_tile<ROWS, RB, NT, false, false>({g.out + n0 * g.ldo + t.m0 * ES, g.ldo, left, cols * ES / 16, 0u}, smem, tid);
        }
    }
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
        const int rows = (int)(g.N - t.n0 < BN ? g.N - t.n0 : BN), cols = (int)(m_end - t.m0 < BM ? m_end - t.m0 : BM);
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
                    const uint32_t off = col < rows && m < cols ? (uint32_t)(col * ld) + 4 * m : NOWHERE;
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, acc[i][j]), rsrc, off, 0, 0);
                }
            }
            return;
        }
        auto to_lds = [&]() __attribute__((always_inline)) {  // the sums, as bf16
            if (on)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const int m = wrow + PM::at(i, wm);
                    *(uint2*)(smem + tile_at<BM * 2>(wcol + PN::at(j, wn), m >> 3) + (m >> 2 & 1) * 8) =
                        make_uint2(pack2(acc[i][j][0], acc[i][j][1]), pack2(acc[i][j][2], acc[i][j][3]));
                }
        };
        if constexpr (PAIR) {
            static_assert(FM % 2 == 0, "fragments in twos");
            constexpr int F2 = FM / 2;
            const int64_t m0 = t.m0 / 2;
            const uint32_t apart = (uint32_t)g.pairs * 2;
            // Rows 0 to 7 of a fragment are gates, 8 to 15 their ups, in the upper half of the lanes.  Two fragments
            // change halves: the gates of one are in the lower lanes, of the other in the upper, and their ups in the
            // other register.  A lane's features, four for each two fragments, start at:
            auto feature = [&](int i) { return (PM::base(wm) + PM::at(2 * i, wm)) / 2 + (lane >> 5) * 8 + (lane >> 4 & 1) * 4; };
            const bool grad = GRAD < 0 ? g.dh != nullptr : GRAD == 1;
            uint2 dh[FN][F2];
            if (grad) {
                const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((uint8_t*)g.dh + t.n0 * g.ldh + m0 * 2, 0, (int)EXTENT, 0x00020000);
                if (on)
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int i = 0; i < F2; ++i) {
                        const int n = wcol + PN::at(j, wn), f = feature(i);
                        const uint32_t off = n < rows && 2 * f < cols ? __umul24((uint32_t)n, (uint32_t)g.ldh) + f * 2 : NOWHERE;
                        dh[j][i] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rsrc, off, 0, 0));
                    }
            }
            if (GRAD != 1 && g.z) {
                to_lds();
                __syncthreads();
                store_tile<BN, BM * 2, NT, true, true>({g.z + t.n0 * g.ldz + m0 * 2, g.ldz, rows, cols / 8, apart}, smem, tid);
                __syncthreads();
            }
            if (on)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < F2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const auto x = __builtin_amdgcn_permlane32_swap(as_uint(acc[2 * i][j][r]), as_uint(acc[2 * i + 1][j][r]),
                                                                        false, false);
                        acc[2 * i][j][r] = as_float(x[0]);
                        acc[2 * i + 1][j][r] = as_float(x[1]);
                    }
            if (grad) {  // out takes them in bf16, as k_act_back's, for the products that follow
                if (on)
                    with_act<ACT>(g.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
                        for (int j = 0; j < FN; ++j)
#pragma unroll
                            for (int i = 0; i < F2; ++i) {
                                const float d[4] = {as_float(dh[j][i].x << 16), as_float(dh[j][i].x & 0xFFFF0000u),
                                                    as_float(dh[j][i].y << 16), as_float(dh[j][i].y & 0xFFFF0000u)};
                                float gate[4], up[4];
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const float2 v = activation<decltype(a)::value, true>(acc[2 * i][j][r]);
                                    gate[r] = d[r] * acc[2 * i + 1][j][r] * v.y;
                                    up[r] = d[r] * v.x;
                                }
                                const int n = wcol + PN::at(j, wn), f = feature(i);
                                *(uint2*)(smem + tile_at<BM * 2>(n, f >> 3 << 1) + (f >> 2 & 1) * 8) =
                                    make_uint2(pack2(gate[0], gate[1]), pack2(gate[2], gate[3]));
                                *(uint2*)(smem + tile_at<BM * 2>(n, f >> 3 << 1 | 1) + (f >> 2 & 1) * 8) =
                                    make_uint2(pack2(up[0], up[1]), pack2(up[2], up[3]));
                            }
                    });
                __syncthreads();
                store_tile<BN, BM * 2, NT, true, false>({g.out + t.n0 * g.ldo + m0 * 2, g.ldo, rows, cols / 8, apart}, smem, tid);
                return;
            }
            if (GRAD != 1 && on)
                with_act<ACT>(g.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int i = 0; i < F2; ++i) {
                            float h[4];
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                h[r] = activation<decltype(a)::value, false>(acc[2 * i][j][r]).x * acc[2 * i + 1][j][r];
                            const int f = feature(i);
                            *(uint2*)(smem + tile_at<BM>(wcol + PN::at(j, wn), f >> 3) + (f >> 2 & 1) * 8) =
                                make_uint2(pack2(h[0], h[1]), pack2(h[2], h[3]));
                        }
                });
            __syncthreads();
            store_tile<BN, BM, NT, false, false>({g.out + t.n0 * g.ldo + m0 * 2, g.ldo, rows, cols / 16, 0u}, smem, tid);
        } else {
            if constexpr (!PLAIN) {
                if (g.bias && on) {
                    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((uint8_t*)(g.bias + t.m0), 0, (int)EXTENT, 0x00020000);
#pragma unroll
                    for (int i = 0; i < FM; ++i) {
                        const int m = wrow + PM::at(i, wm);
                        const v4f b = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rsrc, m < cols ? m * 4 : NOWHERE, 0, 0));
#pragma unroll
                        for (int j = 0; j < FN; ++j) acc[i][j] += b;
                        if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // registers for four loads, not for all
                    }
                }
                if (g.z) {
                    to_lds();
                    __syncthreads();
                    store_tile<BN, BM * 2, NT, false, true>({g.z + t.n0 * g.ldz + t.m0 * 2, g.ldz, rows, cols / 8, 0u}, smem, tid);
                    __syncthreads();
                }
                if (on && (ACT < 0 ? g.act != MXQ_ACT_NONE : ACT != MXQ_ACT_NONE))
                    with_act<ACT>(g.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
                        for (int j = 0; j < FN; ++j)
#pragma unroll
                            for (int i = 0; i < FM; ++i)
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    acc[i][j][r] = activation<decltype(a)::value, false>(acc[i][j][r]).x;
                                    if (r == 3 && i % 2) __builtin_amdgcn_sched_barrier(0);  // eight at a time: no spills
                                }
                    });
            }
            if (g.residual) {
                if (g.f32) add_and_store<4, BM, BN, WGM, WGN, HALVES, WGK>(g, t, acc, smem, tid, rows, cols);
                else add_and_store<2, BM, BN, WGM, WGN, HALVES, WGK>(g, t, acc, smem, tid, rows, cols);
                return;
            }
            if (!g.f32) {
                to_lds();
                __syncthreads();
                const OutTile o{g.out + t.n0 * g.ldo + t.m0 * 2, g.ldo, rows, cols / 8, 0u};
                if (g.nt) store_tile<BN, BM * 2, NT, false, true>(o, smem, tid);
                else store_tile<BN, BM * 2, NT, false, false>(o, smem, tid);
                return;
            }
            // binary32: in two passes where the tile's rows come in halves of 128
            constexpr int PASSES = HALVES ? 2 : 1, FP = FN / PASSES, ROWS = HALVES ? 128 : BN;
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                if (p) __syncthreads();  // the first half is stored
                if (on)
#pragma unroll
                    for (int j = p * FP; j < (p + 1) * FP; ++j)
#pragma unroll
                        for (int i = 0; i < FM; ++i)
                            *(v4f*)(smem + tile_at<BM * 4>(wcol + PN::at(j, wn) - p * ROWS, (wrow + PM::at(i, wm)) >> 2)) = acc[i][j];
                __syncthreads();
                const OutTile o{g.out + (t.n0 + p * ROWS) * g.ldo + t.m0 * 4, g.ldo, rows - p * ROWS, cols / 4, 0u};
                if (g.nt) store_tile<ROWS, BM * 4, NT, false, true>(o, smem, tid);
                else store_tile<ROWS, BM * 4, NT, false, false>(o, smem, tid);
            }
        }
    }
};
template <int BM, int BN, bool HALVES> constexpr int tile_bytes() {
    return BM * 4 * (HALVES ? 128 : BN) > BM * 2 * BN ? BM * 4 * (HALVES ? 128 : BN) : BM * 2 * BN;
}

// (Two waves per SIMD: without the bound the epilogue's activations took 260 registers on 128 x 128 tiles, and one
// block less fitted a CU.)
template <class C, bool TA, bool TB, bool PAIR>
__global__ void __launch_bounds__(threads_of<C>(), 2) k_linear_gemm(const LinearGemm g) {
    static_assert(tile_bytes<C::BM, C::BN, false>() <= LdsOf<C>::BYTES, "the epilogue's tile");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LdsOf<C>::BYTES];
    gemm_plain<C::BM, C::BN, C::WGM, C::WGN, C::WGK, C::NSL, TA, TB, LinearEpi<PAIR, TA>>(g, g.first + blockIdx.x, smem);
}
template <int BM, bool TA, bool TB, bool PAIR, int ACT, int GRAD>
__global__ void __launch_bounds__(512) k_linear_pipe(const LinearGemm g) {
    static_assert(tile_bytes<BM, 256, true>() <= GemmLds<256, 256, 2>::BYTES, "the epilogue's tile");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[GemmLds<256, 256, 2>::BYTES];
    gemm_pipe<BM, TA, TB, LinearEpi<PAIR, TA, false, ACT, GRAD>>(g, g.first + blockIdx.x, smem);
}

// Tiles for few tokens, tile numbers from 16 on.  The weights' bytes bound them: many copies in flight, STREAMS.
struct Wide64 { static constexpr int BM = 128, BN = 64, WGM = 4, WGN = 2, WGK = 1, NSL = 6; };
struct Wide32 { static constexpr int BM = 128, BN = 32, WGM = 4, WGN = 1, WGK = 1, NSL = 8; };
struct Wide128 { static constexpr int BM = 128, BN = 128, WGM = 4, WGN = 2, WGK = 1, NSL = 5; };
struct Quick32 { static constexpr int BM = 32, BN = 32, WGM = 1, WGN = 2, WGK = 2, NSL = 5; };
struct Quick64 { static constexpr int BM = 32, BN = 64, WGM = 1, WGN = 4, WGK = 2, NSL = 6; };
enum { WIDE64 = 16, WIDE32, WIDE128, QUICK32, QUICK64 };
template <class C, bool TA, bool PAIR> __global__ void __launch_bounds__(threads_of<C>()) k_linear_stream(const LinearGemm g) {
    static_assert(tile_bytes<C::BM, C::BN, false>() <= LdsOf<C>::BYTES, "the epilogue's tile");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LdsOf<C>::BYTES];
    gemm_plain<C::BM, C::BN, C::WGM, C::WGN, C::WGK, C::NSL, TA, false, LinearEpi<PAIR, TA, true>>(
        g, g.first + blockIdx.x, smem);
}
// Column sums of a matrix, 32 of them to a block: its threads take runs of 16 bytes of every G-th row, and their
// sums are joined in order.
struct ColumnSums {
    const uint8_t* p;        // bf16 or fp32 [rows][N]
    int64_t ld, rows, N;     // bytes
    int f32, add;
    float* out;              // float [N], added to what is there with add
};
template <int NT, class V> __device__ __forceinline__ void column_sums(const ColumnSums& b, uint32_t block, uint8_t* smem, V load) {
    constexpr int E = sizeof(load((const uint8_t*)nullptr).v) / 4, LANES = 32 / E, G = NT / LANES;
    float (*red)[32] = (float (*)[32])smem;  // [G]
    const int tid = threadIdx.x, l = tid % LANES, r0 = tid / LANES;
    const int64_t c = (int64_t)block * 32 + l * E;
    float s[E];
#pragma unroll
    for (int k = 0; k < E; ++k) s[k] = 0.0f;
    if (c < b.N)
#pragma unroll 8
        for (int64_t r = r0; r < b.rows; r += G) {
            const auto v = load(b.p + r * b.ld + c * (32 / E == 8 ? 4 : 2));
#pragma unroll
            for (int k = 0; k < E; ++k) s[k] += v.v[k];
        }
#pragma unroll
    for (int k = 0; k < E; ++k) red[r0][l * E + k] = s[k];
    __syncthreads();
    for (int n = G / 2; n >= 1; n >>= 1) {
        for (int k = tid; k < n * 32; k += NT) red[k >> 5][k & 31] += red[(k >> 5) + n][k & 31];
        __syncthreads();
    }
    const int64_t o = (int64_t)block * 32 + tid;
    if (tid < 32 && o < b.N) b.out[o] = b.add ? b.out[o] + red[0][tid] : red[0][tid];
}
struct Eight { float v[8]; };
struct Four { float v[4]; };
template <int NT> __device__ __forceinline__ void column_sums(const ColumnSums& b, uint32_t block, uint8_t* smem) {
    if (b.f32)
        column_sums<NT>(b, block, smem, [](const uint8_t* p) __attribute__((always_inline)) {
            const float4 v = *(const float4*)p;
            return Four{{v.x, v.y, v.z, v.w}};
        });
    else
        column_sums<NT>(b, block, smem, [](const uint8_t* p) __attribute__((always_inline)) {
            Eight e;
            unpack8(*(const uint4*)p, e.v);
            return e;
        });
}
template <int NT> constexpr int sums_bytes() { return NT / 4 * 32 * 4; }

// Both gradients' products, and the bias's sums, in one launch: `nb` blocks of sums, `n0` of the first product.
template <class X, class W> __global__ void __launch_bounds__(threads_of<X>(), 2)
k_linear_grads(const LinearGemm x, const LinearGemm w, const ColumnSums b, uint32_t nb, uint32_t n0, int w_first) {
    static_assert(threads_of<X>() == threads_of<W>(), "one block size");
    constexpr int BYTES = LdsOf<X>::BYTES > LdsOf<W>::BYTES ? LdsOf<X>::BYTES : LdsOf<W>::BYTES;
    static_assert(tile_bytes<X::BM, X::BN, false>() <= BYTES && tile_bytes<W::BM, W::BN, false>() <= BYTES &&
                  sums_bytes<threads_of<X>()>() <= BYTES, "the epilogue's tile");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[BYTES];
    if (blockIdx.x < nb) {
        column_sums<threads_of<X>()>(b, blockIdx.x, smem);
        return;
    }
    const uint32_t i = blockIdx.x - nb;
    if ((i < n0) != (w_first != 0))
        gemm_plain<X::BM, X::BN, X::WGM, X::WGN, X::WGK, X::NSL, true, false, LinearEpi<false, true>>(x, i < n0 ? i : i - n0, smem);
    else
        gemm_plain<W::BM, W::BN, W::WGM, W::WGN, W::WGK, W::NSL, true, true, LinearEpi<false, true>>(w, i < n0 ? i : i - n0, smem);
}
// The same on large tiles, BX and BW rows high; the sums go last, where CUs have nothing else to do.
template <int BX, int BW> __global__ void __launch_bounds__(512)
k_linear_grads_pipe(const LinearGemm x, const LinearGemm w, const ColumnSums b, uint32_t n0, uint32_t products, int w_first) {
    constexpr int BYTES = GemmLds<256, 256, 2>::BYTES;
    static_assert(tile_bytes<256, 256, true>() <= BYTES && sums_bytes<512>() <= BYTES, "the epilogue's tile");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[BYTES];
    const uint32_t i = blockIdx.x;
    if (i >= products)
        column_sums<512>(b, i - products, smem);
    else if ((i < n0) != (w_first != 0))
        gemm_pipe<BX, true, false, LinearEpi<false, true, false, 0, 0>>(x, i < n0 ? i : i - n0, smem);
    else
        gemm_pipe<BW, true, true, LinearEpi<false, true, false, 0, 0>>(w, i < n0 ? i : i - n0, smem);
}
hipError_t linear_grads(const LinearGemm& x, int x_tile, const LinearGemm& w, int w_tile, const ColumnSums& b, hipStream_t st);

// The product's form: operands k contiguous; A transposed; both transposed; A's rows paired.
enum { FORM_NN = 0, FORM_TN = 1, FORM_TT = 2, FORM_PAIRED = 3 };
template <int FORM> hipError_t linear_gemm(const LinearGemm& g, int tile, int splits, hipStream_t st);

}  // namespace mxq
