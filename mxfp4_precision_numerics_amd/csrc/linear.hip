// linear.hip - linear layers with bias, activation and residual, gated layers, and
// the gradients of both, for gfx950.
//
//   linear  z = x w^T + bias, y = act(z) + residual
//           dz = dy act'(z), dx = dz w (+ add), dw (+)= dz^T x, dbias (+)= sum of dz's rows
//   gated   (gate, up) = x w^T, h = act(gate) up
//           dgate = dh up act'(gate), dup = dh act(gate), dx and dw as above
//
// The weights' bytes bound it up to some 200 tokens: 1 token x 4096 x 4096 8.8-9.3 us (a kernel alone; 8.3 at best), 48 x 4096 x
// 2 x 14336 42 us, 5.6 TB/s.  Above, the matrix units at the clock that their power leaves (1.6 to 1.9 GHz, the units busy
// for 0.70 to 0.78 of the cycles): 8192 x 14336 x 4096, fp32
// out and residual, 675-716 us (1340-1425 TFLOP/s), gated 8192 x 4096 x 2 x 14336 1.37-1.44 ms.  Gradients: dz is made
// in a pass of its own (bf16; of 235 million sums 195 us, 6.0 TB/s) where an activation asks for one, then both products, 2.9-3.1
// ms for that gated layer.
#include "gemm_plan.h"
#include "linear_gemm.h"

namespace mxq {
namespace {

// One to four tokens: the weights' bytes bound it.  A wave reads 512 k of each of R
// rows (paired: R / 2 of either matrix), a row's 1 KiB in one instruction, multiplies in
// binary32 and goes on NW x 512 k further; the lanes' sums are joined in a
// tree, the waves' in LDS in their order.  (Through the matrix units a wave would read 64
// bytes of each of 16 rows at a time.)
template <int T, int R, int NW, bool PAIR>
__global__ void __launch_bounds__(64 * NW) k_linear_rows(const LinearGemm g) {
    __shared__ float red[NW][T][R];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int PER = PAIR ? R / 2 : R;  // outputs
    static_assert(PER % 8 == 0, "whole chunks");
    const int64_t m0 = (int64_t)(g.first + blockIdx.x) * PER, width = PAIR ? g.pairs : g.M;
    constexpr int CPR = PER / 8;
    const int64_t n = tid / CPR, m = m0 + tid % CPR * 8;
    const bool mine = n < g.N && m < width;
    Beside beside{};
    if (mine) beside = load_beside<PAIR>(g, n, m);
    float acc[T][R];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[t][r] = 0.0f;
    for (int64_t k = wave * 512 + lane * 8; k < g.K; k += NW * 512) {
        uint4 w[R], x[T];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int64_t row = m0 + (PAIR ? r % PER : r);
            row = row < width ? row : width - 1;  // past the end: read and dropped
            w[r] = ld_nt16(g.A + (PAIR ? row + r / PER * g.pairs : row) * g.lda + k * 2);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) x[t] = *(const uint4*)(g.B + (t < g.N ? t : 0) * g.ldb + k * 2);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float xf[8];
            unpack8(x[t], xf);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float wf[8];
                unpack8(w[r], wf);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[t][r] = fmaf(xf[e], wf[e], acc[t][r]);
            }
        }
    }
    // a tree over the lanes that halves the rows as it goes: lane l ends with row l % R
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int half = R / 2; half > 0; half >>= 1) {
            const bool up = lane & half;
#pragma unroll
            for (int r = 0; r < half; ++r) {
                const float give = up ? acc[t][r] : acc[t][r + half], keep = up ? acc[t][r + half] : acc[t][r];
                acc[t][r] = keep + __shfl_xor(give, half, 64);
            }
        }
#pragma unroll
        for (int off = R; off < 64; off <<= 1) acc[t][0] += __shfl_xor(acc[t][0], off, 64);
        if (lane < R) red[wave][t][lane] = acc[t][0];
    }
    __syncthreads();
    if (!mine) return;
    auto sum8 = [&](int r0, float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = red[0][n][r0 + e];
#pragma unroll
            for (int w = 1; w < NW; ++w) v[e] += red[w][n][r0 + e];
        }
    };
    const int c = tid % CPR * 8;
    float v[8];
    sum8(c, v);
    if constexpr (PAIR) {
        float u[8];
        sum8(PER + c, u);
        finish_gated(g, n, m, v, u, beside);
    } else {
        finish_linear<false>(g, n, m, v, beside);
    }
}

// Join the splits' sums, in their order, and finish.  A thread takes a chunk.
template <bool PAIR, bool PLAIN> __device__ __forceinline__ void join_chunk(const LinearGemm& g, int64_t i) {
    const int64_t width = PAIR ? g.pairs : g.M, cpr = width / 8;
    if (i >= g.N * cpr) return;
    const int64_t n = i / cpr, ch = i - n * cpr, m = ch * 8;
    const Beside beside = load_beside<PAIR>(g, n, m);
    const float* p = g.part + n * g.M + (PAIR ? ch * 16 : m);
    auto sum8 = [&](const float* p, float (&v)[8]) {
        v4f lo = {0.0f, 0.0f, 0.0f, 0.0f}, hi = lo;
#pragma unroll 4
        for (int s = 0; s < g.splits; ++s) {
            lo += *(const v4f*)(p + s * g.N * g.M);
            hi += *(const v4f*)(p + s * g.N * g.M + 4);
        }
        *(v4f*)v = lo;
        *(v4f*)(v + 4) = hi;
    };
    float v[8];
    sum8(p, v);
    if constexpr (PAIR) {
        float u[8];
        sum8(p + 8, u);
        finish_gated(g, n, m, v, u, beside);
    } else {
        finish_linear<PLAIN>(g, n, m, v, beside);
    }
}
template <bool PAIR, bool PLAIN> __global__ void __launch_bounds__(256) k_linear_join(const LinearGemm g) {
    join_chunk<PAIR, PLAIN>(g, ((int64_t)g.first + blockIdx.x) * 256 + threadIdx.x);
}
// Two products' in one launch: nx blocks of x.
__global__ void __launch_bounds__(256) k_linear_join_two(const LinearGemm x, const LinearGemm w, uint32_t nx) {
    const bool is_x = blockIdx.x < nx;
    join_chunk<false, true>(is_x ? x : w, (int64_t)(is_x ? blockIdx.x : blockIdx.x - nx) * 256 + threadIdx.x);
}

// Gradients before the products.  A wave takes rows of 512 columns (8 a lane), a
// block every fourth row of a run of `rows`; the columns' sums (dbias) stay in
// registers, are joined over the block's waves and left per run.  dz is left in bf16, the matrix units' type:
// 32 bits would take two terms for each entry, twice the products and twice the bytes.  Gradients in bf16 are off by 2.35e-3
// (2-norm) with it, by 1.66e-3, their own rounding, without.
struct ActBack {
    const uint8_t *dy, *z;   // bf16 [T][N] (gated: z [T][2 N])
    uint8_t* dz;             // bf16 like z, or nullptr
    int64_t ld_dy, ld_z, ld_dz;
    int64_t T, N, rows;
    float* part;             // [runs][N] or nullptr
    int act;
};
template <bool GATED> __global__ void __launch_bounds__(256) k_act_back(const ActBack g) {
    __shared__ float red[3][8][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = ((int64_t)blockIdx.x * 64 + lane) * 8, t0 = blockIdx.y * g.rows;
    const int64_t t1 = t0 + g.rows < g.T ? t0 + g.rows : g.T;
    const bool in = c < g.N;
    float sum[8] = {};
    if (in)
        with_act(g.act, [&](auto a) {
            constexpr int ACT = decltype(a)::value;
#pragma unroll 4
            for (int64_t t = t0 + wave; t < t1; t += 4) {
                float d[8];
                if constexpr (GATED) {
                    float gate[8], up[8];
                    unpack8(ld_nt16(g.dy + t * g.ld_dy + c * 2), d);
                    unpack8(ld_nt16(g.z + t * g.ld_z + c * 2), gate);
                    unpack8(ld_nt16(g.z + t * g.ld_z + (c + g.N) * 2), up);
                    gated_gradient<ACT>(gate, up, d);
                    *(uint4*)(g.dz + t * g.ld_dz + c * 2) = pack8(gate);
                    *(uint4*)(g.dz + t * g.ld_dz + (c + g.N) * 2) = pack8(up);
                } else {
                    unpack8(*(const uint4*)(g.dy + t * g.ld_dy + c * 2), d);
                    if constexpr (ACT != MXQ_ACT_NONE) {
                        float z[8];
                        unpack8(ld_nt16(g.z + t * g.ld_z + c * 2), z);
#pragma unroll
                        for (int k = 0; k < 8; ++k) d[k] *= activation<ACT, true>(z[k]).y;
                        *(uint4*)(g.dz + t * g.ld_dz + c * 2) = pack8(d);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum[k] += d[k];
                }
            }
        });
    if (GATED || !g.part) return;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (wave) red[wave - 1][k][lane] = sum[k];
    __syncthreads();
    if (wave || !in) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = ((sum[k] + red[0][k][lane]) + red[1][k][lane]) + red[2][k][lane];
    float* o = g.part + blockIdx.y * g.N + c;
    *(float4*)o = make_float4(sum[0], sum[1], sum[2], sum[3]);
    *(float4*)(o + 4) = make_float4(sum[4], sum[5], sum[6], sum[7]);
}
__global__ void __launch_bounds__(256) k_column_sums(const ColumnSums b) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[sums_bytes<256>()];
    column_sums<256>(b, blockIdx.x, smem);
}

// No rows: a weights' gradient of zero.
__global__ void __launch_bounds__(256) k_zero_rows(uint8_t* __restrict__ p, int64_t rows, int64_t upr, int64_t ld) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * upr; i += (int64_t)gridDim.x * 256)
        *(uint4*)(p + i / upr * ld + i % upr * 16) = make_uint4(0u, 0u, 0u, 0u);
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Up to this many tokens a wave multiplies rows by itself (k_linear_rows).
constexpr int64_t FEW = 4;

// As TILES, for these products' epilogues, measured with K 512 and 2048 on whole and half rounds; of operands with k
// contiguous, and with one or both transposed.  (Far longer sums run at a lower clock, and binary32 outputs with a residual store
// for longer: 8192 x 14336 x 4096 with both takes 690 us where these say 612.)
constexpr TileCost LINEAR[2][NTILES] = {{{256, 256, 1, 0, 9.0, 0.80, 1.32},
                                         {Mid::BM, Mid::BN, 2, 0, 4.0, 0.73, 1.02},
                                         {Tiny::BM, Tiny::BN, 2, 0, 2.0, 0.26, 0.37},
                                         {Deep::BM, Deep::BN, 1, 0, 2.5, 0.17, 0.19},
                                         {192, 256, 1, 0, 7.0, 0.57, 1.06},
                                         {Lone::BM, Lone::BN, 1, 0, 3.5, 0.62, 0.67}},
                                        {{256, 256, 1, 0, 9.0, 0.75, 1.38},
                                         {Mid::BM, Mid::BN, 2, 0, 4.0, 0.72, 1.08},
                                         {Tiny::BM, Tiny::BN, 2, 0, 2.0, 0.29, 0.42},
                                         {Deep::BM, Deep::BN, 1, 0, 2.5, 0.16, 0.20},
                                         {192, 256, 1, 0, 7.5, 0.74, 1.12},
                                         {Lone::BM, Lone::BN, 1, 0, 3.5, 0.62, 0.67}}};
// A product's tiles: one launch, its sum cut in splits or not, or two along m or n, as many rows as fill whole
// rounds of 256 large tiles first.
struct Product { Choice a, b; int64_t first; bool along_m; double us; };
constexpr double LAUNCH_US = 2.5, JOIN_US = 4.0;
// A large product's copies come at 13.5 TB/s at most (256 tokens x 4096 x 14336, dx on 256 64 x 64 tiles, two k tiles
// at a time: 74 us for 940 MB, where 0.2 us a k tile would make it 45).
double product_time(bool transposed, int tile, int64_t M, int64_t N, int64_t K, int splits) {
    TileCost c = LINEAR[transposed][tile];
    const int64_t nk = ceil_div(ceil_div(K, KT), splits), slots = 256 * c.per_cu;
    const int64_t blocks = ceil_div(M, c.bm) * ceil_div(N, c.bn) * splits;
    if ((M + N) * K > (int64_t)12 << 20) {
        const double least = (double)((blocks < slots ? blocks : slots) * (c.bm + c.bn) * KT * 2) / 13.5e6;
        c.tk = c.tk > least ? c.tk : least;
        c.tk1 = c.tk1 > least ? c.tk1 : least;
    }
    return LAUNCH_US + tile_time(c, M, N, nk, splits, false) +
           (splits > 1 ? JOIN_US + (double)splits * (double)(M * N) * 8.0 / 4.5e6 : 0.0);
}
Product best_product(bool transposed, int64_t M, int64_t N, int64_t K, int most, unsigned among, bool cuts) {
    const int64_t nk = ceil_div(K, KT);
    auto one = [&](int64_t M, int64_t N, int most, double& us) {
        Choice best{MID, 1};
        us = INFINITY;
        for (int t = 0; t < NTILES; ++t) {
            if (!(among >> t & 1)) continue;
            const int64_t blocks = ceil_div(M, TILES[t].bm) * ceil_div(N, TILES[t].bn);
            if (t == LONE && blocks > 256) continue;
            for (int s = 1; s <= most && (s == 1 || (nk / s >= 8 && blocks * s <= 1024)); ++s) {
                const double u = product_time(transposed, t, M, N, K, s);
                if (u < us) { us = u; best = {t, s}; }
            }
        }
        return best;
    };
    Product p{};
    p.a = one(M, N, most, p.us);
    if (!cuts) return p;
    for (int t : {BIG, SLIM})
        for (bool along_m : {true, false}) {
            const int64_t all = along_m ? M : N, b = along_m ? TILES[t].bm : TILES[t].bn;
            const int64_t per = along_m ? ceil_div(N, TILES[t].bn) : ceil_div(M, TILES[t].bm);
            const int64_t first = ceil_div(all, b) * per / 256 * 256 / per * b;
            if (first < b || first >= all) continue;
            double rest_us;
            const Choice rest = along_m ? one(M - first, N, 1, rest_us) : one(M, N - first, 1, rest_us);
            const double us = rest_us + (along_m ? product_time(transposed, t, first, N, K, 1) : product_time(transposed, t, M, first, K, 1));
            if (us < p.us) p = {{t, 1}, rest, first, along_m, us};
        }
    return p;
}

// The forward product.  Up to 128 tokens the weights' bytes bound it, and the
// STREAMS tiles take it where they gain: a wide one where every CU has 128 rows of w or so to
// read (with the sum cut in `splits` where there are fewer rows), a quick one for short calls.  Times in us of
// one call among others, STREAMS / the best of the others (w cold):
//   24 tokens: 4096 x 28672 41.2 / 50.2, 8192 x 16384 47.2 / 59.2, 4096 x 8192 14.9 / 17.6, 1024 x 1024 5.7 / 7.0
//   48: 4096 x 28672 41.6 / 49.2, 8192 x 57344 paired 160 / 184, 1024 x 8192 8.0 / 8.4
//   100: 4096 x 28672 46.8 / 59.0, 8192 x 8192 34.7 / 41.9, 4096 x 16384 33.8 / 37.5
// and behind: 24: 8192 x 4096 20.2 / 18.4; 100: 4096 x 8192 23.7 / 24.5, 4096 x 4096 18.8 / 17.3.  (Up to 32 tokens QUICK32 is
// taken there all the same, and at any K: with few rows of w and a long K most CUs have no block.)
Product forward_product(int64_t T, int64_t H, int64_t M) {
    const bool large = M >= 24576 || (M >= 8192 && M * H >= (int64_t)44 << 20);
    const int64_t fills = T <= 32 ? 16384 : 32768;
    const int s = M < fills ? (int)(fills / M) : 1;
    if (T <= 128 && large) return {{T <= 32 ? WIDE32 : T <= 64 ? WIDE64 : WIDE128, s}};
    if (T <= 32) return {{QUICK32, M <= 4096 && H >= 6144 ? 2 : 1}};
    if (T <= 64 && H <= 2048 && M <= 8192) return {{QUICK64, 1}};
    return best_product(false, M, T, H, 16, ALL, true);
}
// Both gradients' products in one launch, M x Nx over Kx and M x Nw over Kw, on tiles with equal blocks to a CU: the
// blocks that take longer first, each slot taking the next one when its last one ends.
double together_time(const Choice& x, const Choice& w, int64_t M, int64_t Nx, int64_t Kx, int64_t Nw, int64_t Kw) {
    int64_t n[2];
    for (int i = 0; i < 2; ++i) {
        const Choice& c = i ? w : x;
        n[i] = ceil_div(M, TILES[c.tile].bm) * ceil_div(i ? Nw : Nx, TILES[c.tile].bn) * c.splits;
    }
    const int64_t slots = 256 * LINEAR[1][x.tile].per_cu, from = slots - 256;
    double full = (double)(n[0] + n[1] - from) / 256.0, us[2], join = 0.0;
    full = full < 0.0 ? 0.0 : full > 1.0 ? 1.0 : full;
    for (int i = 0; i < 2; ++i) {
        const Choice& c = i ? w : x;
        const TileCost& t = LINEAR[1][c.tile];
        us[i] = t.te + (t.tk1 + (t.tk - t.tk1) * full) * ceil_div(ceil_div(i ? Kw : Kx, KT), c.splits);
        if (c.splits > 1) join += (join == 0.0 ? JOIN_US : 0.0) + (double)c.splits * (double)(M * (i ? Nw : Nx)) * 8.0 / 9e6;
    }
    const int l = us[1] > us[0];
    // `late` slots end the long blocks one block later than the others
    int64_t late = n[l] % slots, left = n[1 - l];
    double t0 = us[l] * (n[l] / slots), t1 = t0 + (late ? us[l] : 0.0), end = t1;
    const double step = us[1 - l];
    if (left > 16 * slots) {
        t0 += (left / slots - 8) * step;
        t1 += (left / slots - 8) * step;
        left -= (left / slots - 8) * slots;
    }
    while (left > 0) {
        const bool first = t0 <= t1;
        double& t = first ? t0 : t1;
        left -= first ? slots - late : late;
        t += step;
        end = end > t ? end : t;
        if (!late) t1 = t0;
    }
    // two blocks on a CU run into each other: between these rounds and none at all.  (0.45, not 0.5: a fit to the sizes in
    // back_plan, a tenth less than their mean says; its cause was not looked for.)
    if (slots > 256) {
        double work = 0.0;
        for (int i = 0; i < 2; ++i) work += n[i] * (us[i] - 0.5 * LINEAR[1][(i ? w : x).tile].te) / slots;
        end = 0.45 * (end + work + LINEAR[1][x.tile].te);
    }
    return LAUNCH_US + end + join;
}
struct BackPlan {
    Product dx, dw;                         // each on its own
    Choice dx_one, dw_one;                  // both in one launch, where that takes less
    bool one;
    int64_t rows, runs;                     // of k_act_back
    int64_t pitch;                          // of dz
    int64_t dz, parts, dx_part, dw_part, bytes;  // offsets
};
// T > 0.  N: rows of w; runs of rows so that there are up to 1024 blocks, each wave with two rows at least.
BackPlan back_plan(int64_t T, int64_t H, int64_t N, int64_t inter, bool act) {
    BackPlan p{};
    const int64_t cols = ceil_div(inter ? inter : N, 512);
    p.rows = ceil_div(ceil_div(T, ceil_div(1024, cols)), 8) * 8;
    p.runs = ceil_div(T, p.rows);
    p.pitch = N * 2 + 256;  // off the powers of two
    p.dz = 0;
    p.parts = act ? up256(T * p.pitch) : 0;
    p.dx_part = p.parts + (inter ? 0 : up256(p.runs * N * 4));
    p.dx = best_product(true, H, T, N, 32, TRANSPOSED, true);
    p.dw = best_product(true, H, N, T, 16, TRANSPOSED, true);
    // dx of few tokens: as forward_product's (4096 x 14336, STREAMS / the others: 32 tokens 30.1 / 32.3 us, 64 31.2 /
    // 34.9, 128 35.4 / 49.2; behind on 4096 x 4096, 64: 15.2 / 12.8).
    const bool wide = T <= 128 && H <= 32768 && H * N >= (int64_t)44 << 20;
    if (wide) p.dx = {{T <= 32 ? WIDE32 : T <= 64 ? WIDE64 : WIDE128, (int)(32768 / H)}};
    // One launch for both: on small tiles, or on up to a few rounds of large ones.  Times in us of dx and dw, on
    // large tiles in one launch / the best otherwise: 2048 tokens x 4096 x 4096 110 / 132, 8192 x 1024 x 4096 130 / 154, 1024 x
    // 2048 x 8192 72 / 90; behind on 512 x 4096 x 4096, 49 / 44.  128 x 128 tiles for both, uncut: 2011 x 2880 x 1000 37 / 46.
    const Product x = best_product(true, H, T, N, 32, PLAIN, false), w = best_product(true, H, N, T, 16, PLAIN, false);
    const int64_t most = LAUNCH_THREADS / 512 / 4;
    auto blocks = [&](const Choice& q, int64_t n) { return ceil_div(H, TILES[q.tile].bm) * ceil_div(n, TILES[q.tile].bn) * q.splits; };
    double us = p.dx.us + p.dw.us;
    auto consider = [&](const Choice& x, const Choice& w) {
        const double t = together_time(x, w, H, T, N, N, T);
        if (t >= us) return;
        us = t;
        p.one = true;
        p.dx_one = x;
        p.dw_one = w;
    };
    if (!wide && blocks(x.a, T) < most && blocks(w.a, N) < most) {
        consider(x.a, w.a);
        const Choice mid{MID, 1};
        if (x.a.splits == 1 && w.a.splits == 1 && blocks(mid, T) >= 128 && blocks(mid, N) >= 128) consider(mid, mid);
        // estimates of small tiles are high; a call for one gradient alone goes by the sum of both as well
        if (x.us + w.us < p.dx.us + p.dw.us + 6.0) {
            p.dx = x;
            p.dw = w;
        }
    }
    const int64_t large = ceil_div(H, 256) * (ceil_div(T, 256) + ceil_div(N, 256));
    if (T >= 256 && large >= 64 && large <= 1024)
        for (int sx = 1; sx <= 4; ++sx)
            for (int sw = 1; sw <= 4; ++sw)
                for (int tiles = 0; tiles < 4; ++tiles)
                    if ((sx == 1 || N / KT / sx >= 8) && (sw == 1 || T / KT / sw >= 8))
                        consider({tiles & 1 ? SLIM : BIG, sx}, {tiles & 2 ? SLIM : BIG, sw});
    auto parts = [&](int a, int b) { const int s = a > b ? a : b; return s > 1 ? s : 0; };
    p.dw_part = p.dx_part + up256(parts(p.dx.a.splits, p.dx_one.splits) * T * H * 4);
    p.bytes = p.dw_part + up256(parts(p.dw.a.splits, p.dw_one.splits) * N * H * 4);
    return p;
}

int64_t join_blocks(const LinearGemm& g, bool paired) { return ceil_div(g.N * ((paired ? g.pairs : g.M) / 8), 256); }
template <int FORM> hipError_t product(LinearGemm g, const Product& p, void* part, hipStream_t st) {
    constexpr bool PAIRED = FORM == FORM_PAIRED, PLAIN_EPI = FORM == FORM_TN || FORM == FORM_TT;
    const Choice c = p.a;
    if (p.first) {
        LinearGemm a = g;
        (p.along_m ? a.M : a.N) = p.first;
        const hipError_t e = linear_gemm<FORM>(a, c.tile, 1, st);
        if (e != hipSuccess) return e;
        (p.along_m ? g.m_from : g.n_from) = p.first;
        return linear_gemm<FORM>(g, p.b.tile, 1, st);
    }
    g.part = c.splits > 1 ? (float*)part : nullptr;
    const hipError_t e = linear_gemm<FORM>(g, c.tile, c.splits, st);
    if (e != hipSuccess || c.splits == 1) return e;
    g.splits = c.splits;
    const int64_t all = join_blocks(g, PAIRED), most = LAUNCH_THREADS / 256;
    for (int64_t b0 = 0; b0 < all; b0 += most) {
        g.first = (uint32_t)b0;
        const unsigned nb = (unsigned)(all - b0 < most ? all - b0 : most);
        k_linear_join<PAIRED, PLAIN_EPI><<<nb, 256, 0, st>>>(g);
    }
    return hipGetLastError();
}
// dx's and dw's products (and dbias's sums) in one launch, and their joins in another.
hipError_t both(LinearGemm x, LinearGemm w, const BackPlan& p, const ColumnSums& b, uint8_t* ws, hipStream_t st) {
    for (int i = 0; i < 2; ++i) {
        LinearGemm& g = i ? w : x;
        const Choice c = i ? p.dw_one : p.dx_one;
        g.ntm = ceil_div(g.M, TILES[c.tile].bm);
        g.ntn = ceil_div(g.N, TILES[c.tile].bn);
        g.per = ceil_div(ceil_div(g.K, KT), c.splits);
        g.splits = c.splits;
        if (c.splits > 1) g.part = (float*)(ws + (i ? p.dw_part : p.dx_part));
    }
    const hipError_t e = linear_grads(x, p.dx_one.tile, w, p.dw_one.tile, b, st);
    if (e != hipSuccess) return e;
    const bool jx = x.splits > 1, jw = w.splits > 1;
    const int64_t nx = jx ? join_blocks(x, false) : 0, nw = jw ? join_blocks(w, false) : 0;
    if (nx + nw > 0) k_linear_join_two<<<(unsigned)(nx + nw), 256, 0, st>>>(x, w, (uint32_t)nx);
    return hipGetLastError();
}
// Few tokens.  R = 8 rows a wave (paired: 8 of either matrix), and waves until there are
// 4096 of them or a row has none left.  Times in us of one launch among others, 16 / 8 / 4 waves
// (inputs cold): 1 token x 7168 x 2 x 2048 12.6 / 15.4 / 15.0; 2 x 4096 x 4096 11.2 / 8.4 / 8.3, 2 x 14336 x 4096
// 22.2 / 19.7 / 20.0; 1 x 4096 x 2 x 14336 - / 44.2 / 39.7.
template <bool PAIR> hipError_t rows(LinearGemm& g, hipStream_t st) {
    constexpr int R = PAIR ? 16 : 8;
    const int64_t blocks = ceil_div(PAIR ? g.pairs : g.M, 8);
    const unsigned nb = (unsigned)blocks;
    g.first = 0;
    auto with = [&](auto t) {
        constexpr int T = decltype(t)::value;
        if (blocks >= 1024 || g.K <= 2048) k_linear_rows<T, R, 4, PAIR><<<nb, 256, 0, st>>>(g);
        else if (T > 1 || blocks >= 512 || g.K <= 4096) k_linear_rows<T, R, 8, PAIR><<<nb, 512, 0, st>>>(g);
        else if constexpr (T == 1) k_linear_rows<1, R, 16, PAIR><<<nb, 1024, 0, st>>>(g);
    };
    if (g.N == 1) with(std::integral_constant<int, 1>());
    else if (g.N == 2) with(std::integral_constant<int, 2>());
    else with(std::integral_constant<int, 4>());
    return hipGetLastError();
}
hipError_t forward(const LinearArgs& a, LinearGemm& g, hipStream_t st) {
    const bool pair = a.inter > 0;
    g.A = a.w; g.lda = a.ld_w;
    g.B = a.x; g.ldb = a.ld_x;
    g.pairs = a.inter;
    g.M = a.N;
    g.N = a.T; g.K = a.H;
    g.act = a.act;
    if (a.T <= FEW) return pair ? rows<true>(g, st) : rows<false>(g, st);
    const Product p = forward_product(a.T, a.H, g.M);
    return pair ? product<FORM_PAIRED>(g, p, a.ws + a.ws_part, st) : product<FORM_NN>(g, p, a.ws + a.ws_part, st);
}
int64_t forward_bytes(int64_t T, int64_t H, int64_t M) {
    const int splits = T > FEW ? forward_product(T, H, M).a.splits : 1;
    return splits > 1 ? up256(splits * T * M * 4) : 0;
}

}  // namespace

int64_t linear_bytes(int64_t T, int64_t H, int64_t N, int64_t inter, bool backward) {
    if (T == 0) return 0;
    const int64_t fwd = forward_bytes(T, H, N);
    if (!backward) return fwd;
    // recomputing a gated layer's sums uses the products' room before they do
    const BackPlan p = back_plan(T, H, N, inter, true);
    return p.bytes > p.dx_part + fwd ? p.bytes : p.dx_part + fwd;
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t st) {
    if (a.T == 0) return hipSuccess;
    LinearGemm g{};
    g.bias = a.bias;
    g.residual = a.residual; g.ldr = a.ld_r;
    g.out = a.out; g.ldo = a.ld_out; g.f32 = a.f32;
    g.z = a.z_out; g.ldz = a.ld_z;
    return forward(a, g, st);
}

hipError_t launch_linear_backward(const LinearArgs& a, hipStream_t st) {
    const int64_t es = a.f32 ? 4 : 2;
    if (a.T == 0) {
        if (!a.accumulate && a.dw) k_zero_rows<<<1024, 256, 0, st>>>(a.dw, a.N, a.H * es / 16, a.ld_dw);
        if (!a.accumulate && a.dbias) k_zero_rows<<<64, 256, 0, st>>>((uint8_t*)a.dbias, 1, a.N / 4, 0);
        return hipGetLastError();
    }
    const bool act = a.inter || a.act != MXQ_ACT_NONE;
    const BackPlan p = back_plan(a.T, a.H, a.N, a.inter, act);
    const bool one = p.one && a.dx && a.dw;
    const uint8_t* dz = act ? a.ws + p.dz : a.dy;
    const int64_t ld_dz = act ? p.pitch : a.ld_dy;
    if (a.inter && !a.z) {  // the sums again, their gradients in the epilogue
        LinearArgs f = a;
        f.ws_part = p.dx_part;
        LinearGemm g{};
        g.dh = a.dy; g.ldh = a.ld_dy;
        g.out = a.ws + p.dz; g.ldo = p.pitch;
        const hipError_t e = forward(f, g, st);
        if (e != hipSuccess) return e;
    } else if (act || (a.dbias && !one)) {
        ActBack b{a.dy, a.z, act ? a.ws + p.dz : nullptr, a.ld_dy, a.ld_z, p.pitch, a.T, a.inter ? a.inter : a.N, p.rows,
                  a.dbias ? (float*)(a.ws + p.parts) : nullptr, a.act};
        const dim3 grid((unsigned)ceil_div(b.N, 512), (unsigned)p.runs);
        if (a.inter) k_act_back<true><<<grid, 256, 0, st>>>(b);
        else k_act_back<false><<<grid, 256, 0, st>>>(b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // dbias: the sums of dy's rows, or of what k_act_back left of each run
    ColumnSums sums{};
    if (a.dbias) {
        const bool from_dy = !act && one;
        sums = {from_dy ? a.dy : a.ws + p.parts, from_dy ? a.ld_dy : a.N * 4, from_dy ? a.T : p.runs, a.N, !from_dy, a.accumulate,
                a.dbias};
    }
    LinearGemm x{}, w{};
    x.A = a.w; x.lda = a.ld_w; x.M = a.H;
    x.B = dz; x.ldb = ld_dz; x.N = a.T;
    x.K = a.N;
    x.out = a.dx; x.ldo = a.ld_dx;
    x.residual = a.residual; x.ldr = a.ld_r;
    w.A = a.x; w.lda = a.ld_x; w.M = a.H;
    w.B = dz; w.ldb = ld_dz; w.N = a.N;
    w.K = a.T;
    w.out = a.dw; w.ldo = a.ld_dw; w.f32 = a.f32; w.nt = 1;
    w.residual = a.accumulate ? a.dw : nullptr; w.ldr = a.ld_dw;
    if (one) return both(x, w, p, sums, a.ws, st);
    if (a.dbias) k_column_sums<<<(unsigned)ceil_div(a.N, 32), 256, 0, st>>>(sums);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.dx) e = product<FORM_TN>(x, p.dx, a.ws + p.dx_part, st);
    if (e == hipSuccess && a.dw) e = product<FORM_TT>(w, p.dw, a.ws + p.dw_part, st);
    return e;
}

}  // namespace mxq
