// loss_gemm.h - the bf16 matrix products of the vocabulary cross entropy on
// gfx950's v_mfma_f32_16x16x32_bf16, fp32 accumulation, with the loss's own
// epilogues.
//
// out[n][m] = sum_k A(m, k) B(n, k).  Each operand lies in memory either with
// k contiguous ([mn][k]) or transposed, with mn contiguous ([k][mn]); the
// latter is read from LDS by ds_read_b64_tr_b16, so that neither the
// projection, nor the hidden states, nor the logits' gradient is ever
// transposed in memory.
//
// Operand layout of the 16x16x32 MFMA: lane l supplies row l % 16, k = 8 (l /
// 16) .. +7.  Accumulator lane l, register r is A's row 4 (l / 16) + r and B's
// row l % 16: a lane holds one n and runs of four m.  With m the vocabulary
// and n the tokens a softmax over the vocabulary is a reduction inside lanes,
// and every output row is contiguous along m.
//
// Large products here run as fast as the card's power lets them, and on
// ordinary data the 16x16x32 instruction draws less for the same work than
// the 32x32x16: from registers alone 2037 against 1813 TFLOP/s (on zeros
// both reach 2460 to 2480).
#pragma once
#include "common.h"
#include "gemm_kernel.h"
#include "train_launch.h"

namespace mxq {

typedef short v4s __attribute__((ext_vector_type(4)));

constexpr int KT = 64;  // k per tile: 128 bytes of a row with k contiguous

enum { EPI_LSE = 0, EPI_G = 1, EPI_DX = 2, EPI_DW = 3 };

struct LossGemm {
    const uint8_t *A, *B;
    int64_t lda, ldb;      // bytes
    int64_t M, N, K;
    int64_t ntm, ntn;      // tiles
    uint32_t first;        // block of the product that this launch starts with
    int splits;            // of k; split s covers k tiles [s * per, ...)
    int64_t per;           // k tiles of a split
    // epilogues
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

// Bytes that no operand reaches: the offset of lanes with nothing to copy.
// A copy at or past the resource's extent writes zeros.
constexpr uint32_t NOWHERE = 0x80000000u;
constexpr int64_t EXTENT = 0x7FFFFFF0;

// One operand's k tiles into LDS.  A wave copies PER pieces of 1 KiB (piece i
// of wave w is piece w + i NW of the tile), lane L the 16 bytes at 16 L.
//  k contiguous: rows of 128 bytes, eight per piece, chunks swizzled as
//    lds_off<128>.
//  transposed: regions of RW = min(ROWS, 128) mn, each [64 k][RW]; the 32-byte
//    segments of a row are XOR-ed with f(k), so that the eight rows k whose
//    segment 32 lanes of a transposing read take (two runs of four, eight
//    apart) lie in distinct banks.
template <int ROWS, bool T, int NW>
struct LossLoader {
    static constexpr int PER = ROWS / 8 / NW;
    static constexpr int RW = ROWS < 128 ? ROWS : 128, RWB = RW * 2, RP = 1024 / RWB;  // T
    static constexpr int REGION = KT * RWB;
    static_assert(PER * NW * 8 == ROWS, "whole pieces per wave");
    v4u rsrc;
    uint64_t base;
    int64_t step;           // bytes from one k tile to the next
    uint32_t off[PER];
    int kpos;               // k contiguous: of the lane's chunk; transposed: of its row in piece 0
    static __device__ __forceinline__ int f(int k) {
        return (RW == 128 ? 2 * (k & 3) : 2 * ((k >> 1) & 1)) + ((k >> 3) & 1);
    }
    static __device__ __forceinline__ int piece_k(int wave, int i) { return ((wave + i * NW) * RP) % KT; }
    __device__ __forceinline__ void init(const uint8_t* p, int64_t ld, int64_t mn0, int64_t mn, int64_t k0, int wave,
                                         int lane) {
        const int64_t left = mn - mn0;
        if constexpr (!T) {
            base = (uint64_t)(p + mn0 * ld + k0 * 2);
            step = KT * 2;
            const int r = lane >> 3, c = lane & 7;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int row = (wave + i * NW) * 8 + r;
                off[i] = row < left ? (uint32_t)(row * ld + ((c ^ swz<128>(row)) << 4)) : NOWHERE;
            }
            kpos = 0;
        } else {
            base = (uint64_t)(p + k0 * ld + mn0 * 2);
            step = KT * ld;
            const int kr = lane / (RWB / 16), c = lane % (RWB / 16);
            kpos = kr;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int pc = wave + i * NW, reg = pc * RP / KT, k = (pc * RP) % KT + kr;
                const int seg = (c >> 1) ^ f(k);
                const int col = reg * RW + seg * 16 + (c & 1) * 8;
                off[i] = col < left ? (uint32_t)(k * ld + col * 2) : NOWHERE;
            }
        }
        rsrc = make_rsrc((const void*)base, EXTENT);
    }
    // k index (within the tile) that lane's copy i starts at
    __device__ __forceinline__ int k_of(int i, int wave, int lane) const {
        if constexpr (!T) return ((lane & 7) ^ swz<128>((wave + i * NW) * 8 + (lane >> 3))) * 8;
        else return piece_k(wave, i) + kpos;
    }
    // Copy i of the current tile; `left`: k that remain from the tile's first on.
    __device__ __forceinline__ void issue(int i, int left, uint32_t dst, int wave, int lane) const {
        uint32_t o = off[i];
        if (left < KT) o = k_of(i, wave, lane) < left ? o : NOWHERE;
        dma16(rsrc, o, 0u, dst + (uint32_t)(wave + i * NW) * 1024u);
    }
    __device__ __forceinline__ void advance(int n = 1) {
        base += (uint64_t)(step * n);
        rsrc[0] = (unsigned)base;
        rsrc[1] = (unsigned)(base >> 32) & 0xFFFFu;
    }
};

// The fragment (16 rows from row0, k = 32 ks .. +31) of an operand tile in LDS.
template <int ROWS, bool T>
__device__ __forceinline__ v8bf loss_frag(const uint8_t* s, int row0, int ks, int lane) {
    const int i = lane & 15, q = lane >> 4;
    if constexpr (!T) {
        return *reinterpret_cast<const v8bf*>(s + lds_off<128>(row0 + i, ks * 4 + q));
    } else {
        using L = LossLoader<ROWS, true, 1>;
        const int k = ks * 32 + 8 * q + (i >> 2);
        const int reg = row0 / L::RW, seg = (row0 % L::RW) / 16;
        const uint8_t* a = s + reg * L::REGION + k * L::RWB + ((seg ^ L::f(k)) << 5) + (i & 3) * 8;
        typedef __attribute__((address_space(3))) v4s* lp;
        struct { v4s lo, hi; } r;
        r.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)lds_addr(a));
        r.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)lds_addr(a + 4 * L::RWB));  // f(k + 4) = f(k)
        return __builtin_bit_cast(v8bf, r);
    }
}

// The tile and split of block b of a product.  Blocks go round-robin over the 8 XCDs:
// consecutive tiles are gathered onto one XCD, GM tile columns (n) at a time.
struct LossTile { int64_t m0, n0; int split; };
template <int BM, int BN>
__device__ __forceinline__ LossTile loss_tile(const LossGemm& g, uint32_t b) {
    // 32-bit: a product has fewer than 2^31 blocks
    const uint32_t ntm = (uint32_t)g.ntm, ntn = (uint32_t)g.ntn, tiles = ntm * ntn, nblk = tiles * (uint32_t)g.splits;
    if (nblk % 8 == 0) b = (b % 8) * (nblk / 8) + b / 8;
    const uint32_t split = b / tiles;
    b -= split * tiles;
    constexpr uint32_t GM = 4;
    const uint32_t grp = b / (GM * ntm), first = grp * GM;
    const uint32_t gs = ntn - first < GM ? ntn - first : GM;
    const uint32_t in = b - grp * GM * ntm, q = in / gs;
    return {uni64((int64_t)q * BM), uni64((int64_t)(first + in - q * gs) * BN),
            (int)__builtin_amdgcn_readfirstlane(split)};
}

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

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16;
}

// Where the fragments of wave w (of WG) lie in a tile of B rows: one block of
// rows per wave, or (HALVES, the pipelined loop) a block in the first 128 rows
// and one in the rest.
template <int B, int WG, bool HALVES> struct FragPlace {
    static constexpr int S = B / WG, S0 = 128 / WG, S1 = (B - 128) / WG, F0 = S0 / 16;
    static __device__ __forceinline__ int base(int w) { return w * (HALVES ? S0 : S); }
    // row of fragment i after the base
    static __device__ __forceinline__ int at(int i, int w) {
        return !HALVES || i < F0 ? 16 * i : 128 + w * (S1 - S0) + 16 * (i - F0);
    }
};

// Epilogues on the accumulators of a wave (of the first group of waves; the
// others of WGK pass its barriers and help to store).
template <int BM, int BN, int WGM, int WGN, int EPI, bool HALVES = false, int WGK = 1>
__device__ __forceinline__ void loss_epilogue(const LossGemm& g, const LossTile& t, float gscale,
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

template <int BM, int BN, int NSL, int WGK = 1> struct LossLds {
    static constexpr int SLOT = (BM + BN) * KT * 2;
    static constexpr int STAGE = BN * (BM * 2 + 16);
    static constexpr int BYTES = WGK * NSL * SLOT > STAGE ? WGK * NSL * SLOT : STAGE;
    static_assert(BYTES <= 160 * 1024, "LDS");
};

// The plain loop: a ring of NSL k tiles, one barrier per tile.  WGK > 1: that
// many groups of waves take the k tiles in turn, each with its own ring, and
// the first adds the others' sums at the end, in their order.
template <int BM, int BN, int WGM, int WGN, int WGK, int NSL, bool TA, bool TB, int EPI>
__device__ __forceinline__ void loss_gemm_plain(const LossGemm& g, uint32_t block, uint8_t* smem) {
    constexpr int NW = WGM * WGN, SM = BM / WGM, SN = BN / WGN, FM = SM / 16, FN = SN / 16;
    constexpr int SLOT = LossLds<BM, BN, NSL, WGK>::SLOT, A_B = BM * KT * 2;
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = WGK == 1 ? wid : wid % NW, kg = WGK == 1 ? 0 : wid / NW;
    const int wm = wave / WGN, wn = wave % WGN;
    const LossTile t = loss_tile<BM, BN>(g, block);
    const int64_t k0 = t.split * g.per * KT;
    const int64_t kend = k0 + g.per * KT < g.K ? k0 + g.per * KT : g.K;
    const int nk = (int)uni64(kend > k0 ? (kend - k0 + KT * WGK - 1) / (KT * WGK) : 0);
    float gscale = 1.0f;
    if constexpr (EPI == EPI_DW) gscale = *g.gscale;
    if constexpr (EPI == EPI_G) {
        gscale = g.own_scale ? largest_dloss<64 * NW * WGK>(g.dloss, g.targets, g.N, g.vocab) : *g.gscale;
        if (g.own_scale && block == 0 && tid == 0) *g.gscale = gscale;
    }
    LossLoader<BM, TA, NW> la;
    LossLoader<BN, TB, NW> lb;
    la.init(g.A, g.lda, t.m0, g.M, k0 + kg * KT, wave, lane);
    lb.init(g.B, g.ldb, t.n0, g.N, k0 + kg * KT, wave, lane);
    constexpr int COPIES = decltype(la)::PER + decltype(lb)::PER;
    uint8_t* ring = smem + kg * NSL * SLOT;
    const uint32_t lds = lds_addr(ring);
    int left = (int)uni64(kend - k0) - kg * KT;  // k from the next tile to copy on
    auto issue = [&](int kt) __attribute__((always_inline)) {  // tile kt; past the end: nothing is fetched
        const uint32_t dst = lds + (uint32_t)(kt % NSL) * SLOT;
#pragma unroll
        for (int i = 0; i < decltype(la)::PER; ++i) la.issue(i, left, dst, wave, lane);
#pragma unroll
        for (int i = 0; i < decltype(lb)::PER; ++i) lb.issue(i, left, dst + A_B, wave, lane);
        la.advance(WGK);
        lb.advance(WGK);
        left -= KT * WGK;
    };
    v4f acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < NSL - 1; ++s) issue(s);
    for (int kt = 0; kt < nk; ++kt) {
        if constexpr (NSL == 1) {
            if (kt) __syncthreads();  // tile kt - 1 is read
            issue(kt);
        }
        __builtin_amdgcn_s_waitcnt(wait_vm(NSL == 1 ? 0 : (NSL - 2) * COPIES));  // tile kt has landed ...
        __syncthreads();  // ... for every wave; tile kt - 1 is read
        if constexpr (NSL > 1) issue(kt + NSL - 1);
        const uint8_t* s = ring + (kt % NSL) * SLOT;
#pragma unroll
        for (int ks = 0; ks < KT / 32; ++ks) {
            v8bf a[FM], b[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) a[i] = loss_frag<BM, TA>(s, wm * SM + 16 * i, ks, lane);
#pragma unroll
            for (int j = 0; j < FN; ++j) b[j] = loss_frag<BN, TB>(s + A_B, wn * SN + 16 * j, ks, lane);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(0));  // no copy may land in what follows
    __syncthreads();
    if constexpr (WGK > 1) {
        static_assert((WGK - 1) * BM * BN * 4 <= LossLds<BM, BN, NSL, WGK>::BYTES, "LDS");
        float* sums = (float*)smem;  // [WGK - 1][wave][register][lane]
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (kg > 0) sums[((((kg - 1) * NW + wave) * FM + i) * FN + j) * 256 + r * 64 + lane] = acc[i][j][r];
        __syncthreads();
        if (kg == 0)
            for (int q = 0; q < WGK - 1; ++q)
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[i][j][r] += sums[(((q * NW + wave) * FM + i) * FN + j) * 256 + r * 64 + lane];
        __syncthreads();
    }
    loss_epilogue<BM, BN, WGM, WGN, EPI, false, WGK>(g, t, gscale, acc, smem, tid);
}

// Tiles of the plain loop: two blocks per CU on 128 x 128 and on 64 x 64, and
// one on 64 x 64 with two groups of waves, for launches of few blocks.
struct Mid { static constexpr int BM = 128, BN = 128, WGM = 2, WGN = 2, WGK = 1, NSL = 2; };
struct Tiny { static constexpr int BM = 64, BN = 64, WGM = 2, WGN = 2, WGK = 1, NSL = 4; };
struct Deep { static constexpr int BM = 64, BN = 64, WGM = 2, WGN = 2, WGK = 2, NSL = 4; };
// Mid for launches of one block per CU: three k tiles on their way instead of
// one.  128 tokens x 4096 x 32000 words forward 71 us against 85.
struct Lone { static constexpr int BM = 128, BN = 128, WGM = 2, WGN = 2, WGK = 1, NSL = 4; };
// dw of few tokens, where a tile's stores outweigh its products: three blocks
// per CU, each with one k tile in LDS at a time.  Bound by HBM: for 48 tokens x
// 4096 x 131072 the 1.07 GB of dw take 200 us, on Mid 280.
struct Flat { static constexpr int BM = 128, BN = 128, WGM = 2, WGN = 2, WGK = 1, NSL = 1; };
template <class C> constexpr int threads_of() { return 64 * C::WGM * C::WGN * C::WGK; }
template <class C> using LdsOf = LossLds<C::BM, C::BN, C::NSL, C::WGK>;

template <class C, bool TA, bool TB, int EPI>
__global__ void __launch_bounds__(threads_of<C>()) k_loss_gemm(const LossGemm g) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LdsOf<C>::BYTES];
    loss_gemm_plain<C::BM, C::BN, C::WGM, C::WGN, C::WGK, C::NSL, TA, TB, EPI>(g, g.first + blockIdx.x, smem);
}

// dx's and dw's products of a piece in one launch: both wait for g alone.
template <class X, class W>
__global__ void __launch_bounds__(threads_of<X>()) k_loss_grads(const LossGemm x, const LossGemm w, uint32_t nx) {
    static_assert(threads_of<X>() == threads_of<W>(), "one block size");
    constexpr int BYTES = LdsOf<X>::BYTES > LdsOf<W>::BYTES ? LdsOf<X>::BYTES : LdsOf<W>::BYTES;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[BYTES];
    if (blockIdx.x < nx)
        loss_gemm_plain<X::BM, X::BN, X::WGM, X::WGN, X::WGK, X::NSL, true, false, EPI_DX>(x, blockIdx.x, smem);
    else
        loss_gemm_plain<W::BM, W::BN, W::WGM, W::WGN, W::WGK, W::NSL, true, true, EPI_DW>(w, blockIdx.x - nx, smem);
}

// ---------------------------------------------------------------------------
// The pipelined loop for 256 x 256 tiles: 8 waves, two per SIMD, in two groups
// (the tile's upper and lower wave row) that run half a phase apart: while one
// group's MFMAs run, the other reads fragments and starts copies.
//
// A k tile of an operand is two halves of 128 mn, A0 A1 B0 B1 of 16 KiB each;
// a wave owns 64 rows of A and 32 of B in each half, and a k tile takes two
// phases of 32 MFMAs:
//     phase       0                       1
//     reads       a0 b0 b1 (k)            a1 (k)
//     multiplies  a0 b0, a0 b1            a1 b0, a1 b1
//     copies      A1 (k + 1)              A0 B0 B1 (k + 2)
// (With 192 rows of A the second half has 64, and the second phase 16 MFMAs.)
// Two slots of LDS hold a k tile each.  A group's reads have arrived before
// the barrier that ends its reading half of the phase, so the other group may
// refill what both have read one phase later.  Eight copies of a wave (seven)
// are in flight after each phase's own: a copy has three phases to land, and each
// phase waits for the halves that the next one reads.
//
// Measured at M = 16384, N = 8192, K = 4096 on one MI355X: 706 us without an
// epilogue (1557 TFLOP/s); with the copies left out and the same data 611; on
// zeros, which draw little power, 495 (0.89 of the peak at 2.4 GHz).  So the
// clock, held down by power to 1.6 - 1.75 GHz, bounds it more than any wait.
// Four phases of eight (32x32x16) MFMAs took 4% more than two of 16, the plain
// loop above 20% more; the 32x32x16 instruction in this loop 8%.
// ---------------------------------------------------------------------------
constexpr int HALF = 128 * KT * 2;

template <int ROWS, bool T>
struct HalfLoader {
    using L = LossLoader<ROWS, T, 8>;
    L h;
    int left;  // k from this half's next tile on
    __device__ __forceinline__ void init(const uint8_t* p, int64_t ld, int64_t mn0, int64_t mn, int64_t k0, int k, int wave,
                                         int lane) {
        h.init(p, ld, mn0, mn, k0, wave, lane);
        left = k;
    }
    __device__ __forceinline__ void copy(uint32_t dst, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < L::PER; ++i) h.issue(i, left, dst, wave, lane);
        h.advance();
        left -= KT;
    }
};

__device__ __forceinline__ void phase_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <int BM, bool TA, bool TB, int EPI>
__global__ void __launch_bounds__(512) k_loss_gemm_pipe(const LossGemm g) {
    constexpr int BN = 256, WGM = 2, WGN = 4;
    constexpr int A1 = BM - 128, F1 = A1 / 32;  // rows of A's second half; fragments of a wave in it
    static_assert(A1 == 128 || A1 == 64, "256 or 192 rows");
    constexpr int FLIGHT = 6 + A1 / 64;  // copies of a wave that stay in flight over a phase
    constexpr int SLOT = 4 * HALF, OA = 0, OB = 2 * HALF;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LossLds<256, BN, 2>::BYTES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const LossTile t = loss_tile<BM, BN>(g, g.first + blockIdx.x);
    const int64_t k0 = t.split * g.per * KT;
    const int64_t kend = k0 + g.per * KT < g.K ? k0 + g.per * KT : g.K;
    const int k = (int)uni64(kend > k0 ? kend - k0 : 0);
    const int nk = (k + KT - 1) / KT;
    HalfLoader<128, TA> a0;
    HalfLoader<A1, TA> a1;
    HalfLoader<128, TB> b0, b1;
    a0.init(g.A, g.lda, t.m0, g.M, k0, k, wave, lane);
    a1.init(g.A, g.lda, t.m0 + 128, g.M, k0, k, wave, lane);
    b0.init(g.B, g.ldb, t.n0, g.N, k0, k, wave, lane);
    b1.init(g.B, g.ldb, t.n0 + 128, g.N, k0, k, wave, lane);
    const uint32_t lds = lds_addr(smem);
    v4f acc[4 + F1][4];
#pragma unroll
    for (int i = 0; i < 4 + F1; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    b0.copy(lds + OB, wave, lane);
    a0.copy(lds + OA, wave, lane);
    b1.copy(lds + OB + HALF, wave, lane);
    a1.copy(lds + OA + HALF, wave, lane);
    b0.copy(lds + SLOT + OB, wave, lane);
    a0.copy(lds + SLOT + OA, wave, lane);
    b1.copy(lds + SLOT + OB + HALF, wave, lane);
    __builtin_amdgcn_s_waitcnt(wait_vm(FLIGHT));  // B0(0), A0(0), B1(0)
    phase_barrier();

    v8bf fa[4][2], fb[4][2];
    if (wm == 1) phase_barrier();  // the second group runs half a phase behind

    auto mfmas = [&](auto ha_) __attribute__((always_inline)) {
        constexpr int ha = decltype(ha_)::value;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        phase_barrier();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < (ha ? F1 : 4); ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[4 * ha + i][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i][s], fb[j][s], acc[4 * ha + i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        phase_barrier();
    };
    constexpr std::integral_constant<int, 0> I0;
    constexpr std::integral_constant<int, 1> I1;
    auto tile = [&](auto p_) __attribute__((always_inline)) {
        constexpr int P = decltype(p_)::value;
        const uint8_t* cur = smem + P * SLOT;
        const uint32_t lc = lds + P * SLOT, ln = lds + (1 - P) * SLOT;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i][s] = loss_frag<128, TA>(cur + OA, wm * 64 + 16 * i, s, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fb[j][s] = loss_frag<128, TB>(cur + OB + (j / 2) * HALF, wn * 32 + 16 * (j % 2), s, lane);
        }
        a1.copy(ln + OA + HALF, wave, lane);
        __builtin_amdgcn_s_waitcnt(wait_vm(FLIGHT));
        mfmas(I0);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < F1; ++i)
                fa[i][s] = loss_frag<A1, TA>(cur + OA + HALF, wm * (A1 / 2) + 16 * i, s, lane);
        b0.copy(lc + OB, wave, lane);
        a0.copy(lc + OA, wave, lane);
        b1.copy(lc + OB + HALF, wave, lane);
        __builtin_amdgcn_s_waitcnt(wait_vm(FLIGHT));
        mfmas(I1);
    };
    int kt = 0;
    for (; kt + 2 <= nk; kt += 2) {
        tile(I0);
        tile(I1);
    }
    if (kt < nk) tile(I0);
    if (wm == 0) phase_barrier();
    __builtin_amdgcn_s_waitcnt(wait_vm(0));  // no copy may land in what the epilogue stages
    __syncthreads();
    loss_epilogue<BM, BN, WGM, WGN, EPI, true>(g, t, EPI == EPI_G || EPI == EPI_DW ? *g.gscale : 1.0f, acc, smem, tid);
}

}  // namespace mxq
