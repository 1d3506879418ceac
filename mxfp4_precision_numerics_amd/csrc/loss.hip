// loss.hip - softmax cross entropy of hidden states against a vocabulary
// projection, and its gradients, for gfx950: no logits in memory.
//
//   forward   z = x w^T tile by tile; each tile leaves a (max, sum of exp) per
//             token, a second launch joins them:  lse, loss = lse - z[target]
//   backward  per piece of the vocabulary:  g = (exp(z - lse) - onehot) dloss,
//             z computed again, g held in bf16;  dx += g w,  dw = g^T x
//
// The products are 2 T V H operations forward and 6 T V H backward, two more
// than with the logits kept, which would take T V values of workspace.
//
// g is rounded to bf16, the type that the matrix units multiply: 2^-8 of each
// entry at most.  The sums do not average that out (signal and rounding grow
// alike).  It shows where no entry of a token's g is near -1, which bf16 all but
// holds, that is, with few words: dx and dw are off by 1.94e-3 (2-norm, relative)
// for 300 tokens x 256 x 300 words, 1.83e-3 for 2051 x 1136 x 825, 1.71e-3 for 48 x
// 1024 x 4000, where g in binary32 gives 1.66e-3, the output's own rounding; for
// 2011 x 2880 x 50021 both are the same.  Where one entry outweighs the rest it
// is all of g's half step: dw of one token, 2696 x 1582, 3.8e-3 against 2.0e-3.
// g is relative to the largest |dloss|, so that a mean's common factor, applied to
// the binary32 sums, adds no rounding.
//
// 8192 tokens x 4096 x 131072 words, forward and gradients: 25.1 ms, 1402
// TFLOP/s over the four products (a library product of this size alone 1455 to
// 1492); 48 tokens forward 180 us, the projection read once at 6 TB/s.
#include "loss_gemm.h"

namespace mxq {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Large problems run 256 x 256 or 192 x 256 tiles with the pipelined loop, one
// block per CU; smaller ones the plain loop on tiles that reach more CUs sooner.

// Which tile: the one with the least estimated time in us, from fits to
// measurements of each tile over M 256 .. 16384, N 1 .. 16384, K 1 .. 16384
// on one MI355X: start and epilogue (of a round among others in the products with
// exponentials, EPI_LSE and EPI_G, and of any other round), time per k tile with
// one block on a CU, and with all its blocks (the clock falls as the large tiles
// fill the chip).
// Measured beside it (256 / 128 / 64 tiles):
// M 6000, N 200, K 1104: 25.6 / 16.2 / 12.3 us; 16384, 300, 2048: 40.5 / 32.7 /
// 40.9; 16384, 2011, 2880: 148 / 188 / 293.
struct TileCost { int bm, bn, per_cu; double te_exp, te, tk1, tk; };
enum { BIG, MID, TINY, DEEP, SLIM, LONE, NTILES };
constexpr TileCost TILES[NTILES] = {{256, 256, 1, 8.2, 11.0, 0.85, 1.35},
                                    {Mid::BM, Mid::BN, 2, 5.3, 3.2, 0.60, 1.00},
                                    {Tiny::BM, Tiny::BN, 2, 1.8, 1.8, 0.30, 0.42},
                                    {Deep::BM, Deep::BN, 1, 5.0, 5.0, 0.17, 0.21},
                                    {192, 256, 1, 7.5, 9.5, 0.68, 1.05},
                                    {Lone::BM, Lone::BN, 1, 3.2, 3.2, 0.48, 0.48}};
bool pipelined(int tile) { return tile == BIG || tile == SLIM; }
double tile_time(const TileCost& c, int64_t M, int64_t N, int64_t nk, int64_t splits, bool exps) {
    const int64_t blocks = ceil_div(M, c.bm) * ceil_div(N, c.bn) * splits;
    if (blocks <= 256) return c.te + (c.per_cu == 1 ? c.tk1 + (c.tk - c.tk1) * blocks / 256 : c.tk1) * nk;
    // whole rounds of the larger tiles; two small ones on a CU run into each other
    const int64_t slots = 256 * c.per_cu;
    const double rounds = c.bm > 64 || c.per_cu == 1 ? (double)ceil_div(blocks, slots) : (double)blocks / slots;
    return rounds <= 1.0 ? c.te + c.tk * nk : rounds * ((exps ? c.te_exp : c.te) + c.tk * nk);
}
struct Choice { int tile, splits; };
// most > 1: also how many ways to cut K, each of which writes and reads back
// M N binary32 sums (4.5 TB/s), a tile's share being at least eight k tiles.
// exps: of EPI_LSE or EPI_G; among: bits of the tiles; LONE is for products of two operands with k contiguous
// and one block per CU (on transposed ones it took 5-10% longer than MID).
constexpr unsigned ALL = (1u << NTILES) - 1, TRANSPOSED = ALL & ~(1u << LONE), PLAIN = 1u << MID | 1u << TINY;
Choice choose(int64_t M, int64_t N, int64_t K, int most, bool exps, unsigned among) {
    Choice best{MID, 1};
    double least = INFINITY;
    const int64_t nk = ceil_div(K > 0 ? K : 1, KT);
    for (int t = 0; t < NTILES; ++t) {
        if (!(among >> t & 1)) continue;
        if (t == LONE && ceil_div(M, Lone::BM) * ceil_div(N, Lone::BN) > 256) continue;
        for (int s = 1; s <= most && (s == 1 || nk / s >= 8); ++s) {
            const double us = tile_time(TILES[t], M, N, ceil_div(nk, s), s, exps) + (s - 1) * (double)(M * N) * 8.0 / 4.5e6;
            if (us < least) { least = us; best = {t, s}; }
        }
    }
    return best;
}

// The vocabulary in one launch, or cut in two: as many words as fill whole
// rounds of the 256-wide tiles, and the rest, less than a round, on smaller
// ones (`first` is all of it where one launch is estimated to be faster, 8 us
// being the second one's own cost).  Measured for 2011 tokens x 2880 x 50021
// words (6.1 rounds): forward 493 us in one, 453 + 27 us in two; 4000 x 4096 x
// 5000 forward and gradients 660 us against 608.
struct Cut { int64_t first; Choice a, b; double us; };
// v_is_m: the vocabulary is the product's m (else its n); other: its other size.
Cut cut(int64_t V, int64_t other, int64_t K, bool v_is_m) {
    const int64_t nk = ceil_div(K, KT);
    auto time = [&](int tile, int64_t v) {
        return v_is_m ? tile_time(TILES[tile], v, other, nk, 1, true) : tile_time(TILES[tile], other, v, nk, 1, false);
    };
    auto one = [&](int64_t v) { return v_is_m ? choose(v, other, K, 1, true, ALL) : choose(other, v, K, 1, false, TRANSPOSED); };
    Cut c{V, one(V), {0, 1}, 0.0};
    c.us = time(c.a.tile, V);
    for (int t : {BIG, SLIM}) {
        const int64_t bv = v_is_m ? TILES[t].bm : TILES[t].bn, bo = v_is_m ? TILES[t].bn : TILES[t].bm;
        const int64_t per = ceil_div(other, bo), rounds = ceil_div(V, bv) * per / 256;
        const int64_t first = per > 0 ? rounds * 256 / per * bv : V;
        if (first < bv || first >= V) continue;
        const Choice rest = one(V - first);
        const double two = time(t, first) + time(rest.tile, V - first) + 8.0;
        if (two < c.us) c = {first, {t, 1}, rest, two};
    }
    return c;
}

// A product's blocks, in more than one launch where they are too many for one.
template <class F> hipError_t launches(LossGemm& g, int threads, F go) {
    const int64_t all = g.ntm * g.ntn * g.splits, most = LAUNCH_THREADS / threads;
    for (int64_t b0 = 0; b0 < all; b0 += most) {
        g.first = (uint32_t)b0;
        go((unsigned)(all - b0 < most ? all - b0 : most));
    }
    return hipGetLastError();
}
template <bool TA, bool TB, int EPI> hipError_t gemm(LossGemm g, Choice c, hipStream_t st) {
    const TileCost& t = TILES[c.tile];
    g.ntm = ceil_div(g.M, t.bm);
    g.ntn = ceil_div(g.N, t.bn);
    g.per = ceil_div(ceil_div(g.K > 0 ? g.K : 1, KT), c.splits);
    g.splits = c.splits;
    const int nt = pipelined(c.tile) || c.tile == DEEP ? 512 : 256;
    static_assert(threads_of<Deep>() == 512 && threads_of<Mid>() == 256 && threads_of<Tiny>() == 256 &&
                  threads_of<Lone>() == 256, "threads of the tiles");
    return launches(g, nt, [&](unsigned nb) {
        if (c.tile == BIG) k_loss_gemm_pipe<256, TA, TB, EPI><<<nb, nt, 0, st>>>(g);
        else if (c.tile == SLIM) k_loss_gemm_pipe<192, TA, TB, EPI><<<nb, nt, 0, st>>>(g);
        else if (c.tile == MID) k_loss_gemm<Mid, TA, TB, EPI><<<nb, nt, 0, st>>>(g);
        else if (c.tile == TINY) k_loss_gemm<Tiny, TA, TB, EPI><<<nb, nt, 0, st>>>(g);
        else if (c.tile == DEEP) k_loss_gemm<Deep, TA, TB, EPI><<<nb, nt, 0, st>>>(g);
        else if constexpr (!TA) k_loss_gemm<Lone, TA, TB, EPI><<<nb, nt, 0, st>>>(g);
    });
}

// dw's cut; with dx on plain tiles a plain one too unless it costs more than the
// two in one launch save (200 tokens x 2048 x 32000: both gradients 144 us, 157
// in two launches with dw's best tile).
Cut cut_dw(int64_t V, int64_t H, int64_t T, const Choice* dx) {
    const Cut c = cut(V, H, T, false);
    if (!dx || !(PLAIN >> dx->tile & 1)) return c;
    const Choice p = choose(H, V, T, 1, false, PLAIN);
    const double us = tile_time(TILES[p.tile], H, V, ceil_div(T, KT), 1, false);
    return us < c.us + 12.0 ? Cut{V, p, {0, 1}, us} : c;
}

// dw of few tokens, on tiles of its own: up to 256 tokens, and enough tiles to
// outweigh what one launch with dx saves, if that is open.  Measured, both
// gradients, one launch / this one: 48 tokens x 4096 x 131072 (32768 tiles) 682
// / 613 us; 64 x 4096 x 32000 (8000) 168 / 158; 128 x 4096 x 32000 213 / 219;
// 64 x 2048 x 32000 (4000) 90 / 91.
bool flat_pays(const LossGemm& w, bool or_in_one) {
    const int64_t nk = ceil_div(w.K, KT);
    return nk <= 4 && ceil_div(w.M, Flat::BM) * ceil_div(w.N, Flat::BN) >= (or_in_one ? 4096 * nk : 1024);
}
hipError_t dw_flat(LossGemm w, hipStream_t st) {
    w.ntm = ceil_div(w.M, Flat::BM);
    w.ntn = ceil_div(w.N, Flat::BN);
    w.per = ceil_div(w.K, KT);
    w.splits = 1;
    return launches(w, threads_of<Flat>(), [&](unsigned nb) {
        k_loss_gemm<Flat, true, true, EPI_DW><<<nb, threads_of<Flat>(), 0, st>>>(w);
    });
}

// dx's and dw's products in one launch where their tiles share a block size
// (a launch costs the host 3 us, a gap on the device one).
bool one_launch(int x, int w) {
    return (x == DEEP && w == DEEP) || (PLAIN >> x & PLAIN >> w & 1);
}
// false: too many blocks
bool grads_in_one(const LossGemm& x, Choice cx, const LossGemm& w, Choice cw, hipStream_t st) {
    const bool deep = cx.tile == DEEP;
    LossGemm gx = x, gw = w;
    unsigned n[2];
    for (int i = 0; i < 2; ++i) {
        LossGemm& g = i ? gw : gx;
        const Choice c = i ? cw : cx;
        g.ntm = ceil_div(g.M, TILES[c.tile].bm);
        g.ntn = ceil_div(g.N, TILES[c.tile].bn);
        g.per = ceil_div(ceil_div(g.K > 0 ? g.K : 1, KT), c.splits);
        g.splits = c.splits;
        if (g.ntm * g.ntn * c.splits > LAUNCH_THREADS / 512 / 2) return false;  // both in one launch
        n[i] = (unsigned)(g.ntm * g.ntn * c.splits);
    }
    const unsigned nb = n[0] + n[1];
    if (deep) k_loss_grads<Deep, Deep><<<nb, threads_of<Deep>(), 0, st>>>(gx, gw, n[0]);
    else if (cx.tile == MID && cw.tile == MID) k_loss_grads<Mid, Mid><<<nb, threads_of<Mid>(), 0, st>>>(gx, gw, n[0]);
    else if (cx.tile == MID) k_loss_grads<Mid, Tiny><<<nb, threads_of<Mid>(), 0, st>>>(gx, gw, n[0]);
    else if (cw.tile == MID) k_loss_grads<Tiny, Mid><<<nb, threads_of<Mid>(), 0, st>>>(gx, gw, n[0]);
    else k_loss_grads<Tiny, Tiny><<<nb, threads_of<Tiny>(), 0, st>>>(gx, gw, n[0]);
    return true;
}

// Join the tiles' statistics: a block takes 8 tokens, 128 lanes for the tiles
// of each (64-byte pieces of the tiles' rows).
constexpr int JT = 8, JL = 128;
__device__ __forceinline__ float2 join(float2 a, float2 b) {  // (max, sum of exp relative to it)
    const float n = max_num(a.x, b.x), ref = n == -__builtin_inff() ? 0.0f : n;
    return make_float2(n, a.y * __expf(a.x - ref) + b.y * __expf(b.x - ref));
}
// T: of all tokens, a row of statistics; n: of this launch.
__global__ void __launch_bounds__(JT * JL) k_lse_join(const float2* __restrict__ part, int64_t ntm, int64_t T,
                                                      int64_t n, int64_t V, const float* __restrict__ zt,
                                                      const int64_t* __restrict__ targets, float* __restrict__ loss,
                                                      float* __restrict__ lse) {
    __shared__ float2 red[JT * JL / 64][JT];
    const int k = threadIdx.x % JT, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * JT + k;
    float2 a = make_float2(-__builtin_inff(), 0.0f);
    if (t < n)
#pragma unroll 4
        for (int64_t i = threadIdx.x / JT; i < ntm; i += JL) a = join(a, part[i * T + t]);
#pragma unroll
    for (int off = 32; off >= JT; off >>= 1)
        a = join(a, make_float2(__shfl_xor(a.x, off, 64), __shfl_xor(a.y, off, 64)));
    if ((threadIdx.x & 63) < JT) red[wave][k] = a;
    __syncthreads();
    if (threadIdx.x >= JT || t >= n) return;
    for (int w = 1; w < JT * JL / 64; ++w) a = join(a, red[w][k]);
    const float l = a.x + logf(a.y);
    const int64_t tg = targets[t];
    lse[t] = l;
    loss[t] = (uint64_t)tg < (uint64_t)V ? l - zt[t] : 0.0f;
}

__global__ void __launch_bounds__(1024) k_gscale(const float* __restrict__ dloss, const int64_t* __restrict__ targets,
                                                 int64_t T, int64_t V, float* __restrict__ out) {
    const float m = largest_dloss<1024>(dloss, targets, T, V);
    if (threadIdx.x == 0) *out = m;
}

// dx = gscale * the sum of the splits (`split` groups of four values apart), rounded once.  A thread takes 4.
__global__ void __launch_bounds__(256) k_dx_join(const float* __restrict__ part, int splits, int64_t split, int64_t T,
                                                 int64_t H,
                                                 const float* __restrict__ gscale, uint8_t* __restrict__ dx,
                                                 int64_t ld) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, upr = H / 4;
    if (i >= T * upr) return;
    const int64_t t = i / upr, u = i - t * upr;
    const v4f* q = (const v4f*)part + i;
    v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int p = 0; p < splits; ++p) s += q[p * split];
    const float gs = *gscale;
    *(uint2*)(dx + t * ld + u * 8) = make_uint2(pack_bf16(s[0] * gs, s[1] * gs), pack_bf16(s[2] * gs, s[3] * gs));
}

// No tokens: the projection's gradient is zero.
__global__ void __launch_bounds__(256) k_zero_rows(uint8_t* __restrict__ p, int64_t rows, int64_t upr, int64_t ld) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * upr; i += (int64_t)gridDim.x * 256)
        *(uint4*)(p + i / upr * ld + i % upr * 16) = make_uint4(0u, 0u, 0u, 0u);
}

constexpr int64_t OWN_SCALE = 1024;  // tokens; a block reads 12 bytes of each

// How the call is cut: equal pieces of the vocabulary whose g fits 512 MiB, or an
// eighth more where that saves a piece (3155 tokens x 264 x 85226: gradients 765
// us in one piece, 806 in two of which the second had 146 words), and
// the splits of dx's sum over it.
struct Plan {
    Cut lse;
    Choice dx;
    int64_t ntm;            // rows of statistics
    int64_t piece, pitch;   // vocabulary per piece; bytes per row of g
    int64_t parts, zt, gscale, g, dxs, bytes;  // offsets
};
Plan plan(int64_t T, int64_t H, int64_t V, bool backward) {
    Plan p{};
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    p.lse = cut(V, T, H, true);
    p.ntm = ceil_div(p.lse.first, TILES[p.lse.a.tile].bm) + ceil_div(V - p.lse.first, TILES[p.lse.b.tile].bm);
    p.parts = 0;
    p.zt = up(p.ntm * T * 8);
    p.bytes = p.zt + up(T * 4);
    if (!backward) return p;
    const int64_t fits = ((int64_t)256 << 20) / (T > 0 ? T : 1), most = (fits < 2048 ? 2048 : fits) * 9 / 8;
    p.piece = up(ceil_div(V, ceil_div(V, most)));
    p.pitch = p.piece * 2 + 256;  // off the powers of two: dx's product reads a column of lines 3% faster
    p.dx = choose(H, T, p.piece < V ? p.piece : V, 64, false, TRANSPOSED);
    p.gscale = 0;
    p.g = 256;
    p.dxs = p.g + up(T * p.pitch);
    const int64_t bwd = p.dxs + up(p.dx.splits * T * H * 4);
    p.bytes = bwd > p.bytes ? bwd : p.bytes;
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
    g.M = p.lse.first;
    hipError_t e = gemm<false, false, EPI_LSE>(g, p.lse.a, st);
    if (e == hipSuccess && p.lse.first < a.V) {
        LossGemm r = g;
        r.A = a.w + p.lse.first * a.ld_w; r.M = a.V - p.lse.first;
        r.m_first = p.lse.first;
        r.part = g.part + ceil_div(p.lse.first, TILES[p.lse.a.tile].bm) * a.T;
        e = gemm<false, false, EPI_LSE>(r, p.lse.b, st);
    }
    if (e != hipSuccess) return e;
    constexpr int64_t most = LAUNCH_THREADS / JL;  // tokens
    for (int64_t t0 = 0; t0 < a.T; t0 += most) {
        const int64_t n = a.T - t0 < most ? a.T - t0 : most;
        k_lse_join<<<(unsigned)ceil_div(n, JT), JT * JL, 0, st>>>(g.part + t0, p.ntm, a.T, n, a.V, g.zt + t0, a.targets + t0,
                                                                  a.loss + t0, a.lse + t0);
    }
    return hipGetLastError();
}

hipError_t launch_lce_backward(const LceArgs& a, hipStream_t st) {
    if (a.T == 0) {
        if (a.dw) k_zero_rows<<<1024, 256, 0, st>>>(a.dw, a.V, a.H / 8, a.ld_dw);
        return hipGetLastError();
    }
    const Plan p = plan(a.T, a.H, a.V, true);
    float* gscale = (float*)(a.ws + p.gscale);
    const Cut first = cut(p.piece < a.V ? p.piece : a.V, a.T, a.H, true);
    // one product's blocks find the largest |dloss| themselves where there are
    // few tokens and no other product needs it sooner
    const int own = a.T <= OWN_SCALE && !pipelined(first.a.tile) && first.first >= a.V;
    if (!own) k_gscale<<<1, 1024, 0, st>>>(a.dloss, a.targets, a.T, a.V, gscale);
    for (int64_t v0 = 0; v0 < a.V; v0 += p.piece) {
        const int64_t n = a.V - v0 < p.piece ? a.V - v0 : p.piece;
        LossGemm g{};
        g.A = a.w + v0 * a.ld_w; g.lda = a.ld_w; g.M = n;
        g.B = a.x; g.ldb = a.ld_x; g.N = a.T;
        g.K = a.H;
        g.m_first = v0; g.vocab = a.V;
        g.targets = a.targets; g.lse = a.lse_in; g.dloss = a.dloss; g.gscale = gscale; g.own_scale = own;
        g.out = a.ws + p.g; g.ldo = p.pitch;
        g.m_store = (n + 63) / 64 * 64;  // zeros to the end of the last k tile of dx's product
        const Cut c = cut(n, a.T, a.H, true);
        LossGemm r = g;
        if (c.first < n) {  // `first` is a multiple of 64
            g.M = g.m_store = c.first;
            r.A += c.first * a.ld_w; r.M -= c.first;
            r.m_first += c.first; r.m_store -= c.first;
            r.out += c.first * 2;
        }
        hipError_t e = gemm<false, false, EPI_G>(g, c.a, st);
        if (e == hipSuccess && c.first < n) e = gemm<false, false, EPI_G>(r, c.b, st);
        if (e != hipSuccess) return e;
        LossGemm x{}, w{};
        x.A = a.w + v0 * a.ld_w; x.lda = a.ld_w; x.M = a.H;
        x.B = a.ws + p.g; x.ldb = p.pitch; x.N = a.T;
        x.K = n;
        x.out = a.ws + p.dxs; x.ldo = a.H * 4;
        x.add = v0 > 0;
        w.A = a.x; w.lda = a.ld_x; w.M = a.H;
        w.B = a.ws + p.g; w.ldb = p.pitch; w.N = n;
        w.K = a.T;
        w.gscale = gscale;
        w.out = a.dw + v0 * a.ld_dw; w.ldo = a.ld_dw;
        const Cut cw = cut_dw(n, a.H, a.T, a.dx ? &p.dx : nullptr);
        const bool in_one = a.dx && a.dw && cw.first >= n && one_launch(p.dx.tile, cw.a.tile);
        const bool flat = a.dw && flat_pays(w, in_one);
        if (in_one && !flat && grads_in_one(x, p.dx, w, cw.a, st)) {
            e = hipGetLastError();
            if (e != hipSuccess) return e;
            continue;
        }
        if (a.dx) {
            e = gemm<true, false, EPI_DX>(x, p.dx, st);
            if (e != hipSuccess) return e;
        }
        if (flat) {
            e = dw_flat(w, st);
            if (e != hipSuccess) return e;
        } else if (a.dw) {
            LossGemm rest = w;
            if (cw.first < n) {
                w.N = cw.first;
                rest.B += cw.first * 2; rest.N -= cw.first;
                rest.out += cw.first * a.ld_dw;
            }
            e = gemm<true, true, EPI_DW>(w, cw.a, st);
            if (e == hipSuccess && cw.first < n) e = gemm<true, true, EPI_DW>(rest, cw.b, st);
            if (e != hipSuccess) return e;
        }
    }
    if (a.dx) {
        const int64_t upr = a.H / 4, most = LAUNCH_THREADS / upr / 256 * 256;  // tokens; the hidden size is below 2^22
        for (int64_t t0 = 0; t0 < a.T; t0 += most) {
            const int64_t n = a.T - t0 < most ? a.T - t0 : most;
            k_dx_join<<<(unsigned)ceil_div(n * upr, 256), 256, 0, st>>>((const float*)(a.ws + p.dxs) + t0 * a.H, p.dx.splits,
                                                                        a.T * upr, n, a.H, gscale, a.dx + t0 * a.ld_dx,
                                                                        a.ld_dx);
        }
    }
    return hipGetLastError();
}

}  // namespace mxq
