// gemm_plan.h - which tiles a product of bf16_gemm.h runs on, and its launches.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>

#include "bf16_gemm.h"
#include "train_launch.h"

namespace mxq {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Large problems run 256 x 256 or 192 x 256 tiles with the pipelined loop, one
// block per CU; smaller ones the plain loop on tiles that reach more CUs sooner.

// Which tile: the one with the least estimated time in us, from fits to
// measurements of each tile over M 256 .. 16384, N 1 .. 16384, K 1 .. 16384
// on one MI355X: start and epilogue (of a round among others in the products with
// exponentials, the cross entropy's logits, and of any other round), time per k tile with
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
inline bool pipelined(int tile) { return tile == BIG || tile == SLIM; }
inline double tile_time(const TileCost& c, int64_t M, int64_t N, int64_t nk, int64_t splits, bool exps) {
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
// exps: with exponentials in the epilogue; among: bits of the tiles; LONE is for products of two operands with k contiguous
// and one block per CU (on transposed ones it took 5-10% longer than MID).
constexpr unsigned ALL = (1u << NTILES) - 1, TRANSPOSED = ALL & ~(1u << LONE), PLAIN = 1u << MID | 1u << TINY;
inline Choice choose(int64_t M, int64_t N, int64_t K, int most, bool exps, unsigned among) {
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

// A product's blocks, in more than one launch where they are too many for one.
template <class G, class F> hipError_t launches(G& g, int threads, F go) {
    const int64_t all = g.ntm * g.ntn * g.splits, most = LAUNCH_THREADS / threads;
    for (int64_t b0 = 0; b0 < all; b0 += most) {
        g.first = (uint32_t)b0;
        go((unsigned)(all - b0 < most ? all - b0 : most));
    }
    return hipGetLastError();
}
// A product on the tiles of its choice: go(arguments, blocks, threads) for each launch.
template <class G, class F> hipError_t on_tiles(G g, Choice c, F go) {
    const TileCost& t = TILES[c.tile];
    g.ntm = ceil_div(g.M - g.m_from, t.bm);
    g.ntn = ceil_div(g.N - g.n_from, t.bn);
    g.per = ceil_div(ceil_div(g.K > 0 ? g.K : 1, KT), c.splits);
    g.splits = c.splits;
    const int nt = pipelined(c.tile) || c.tile == DEEP ? 512 : 256;
    static_assert(threads_of<Deep>() == 512 && threads_of<Mid>() == 256 && threads_of<Tiny>() == 256 &&
                  threads_of<Lone>() == 256, "threads of the tiles");
    return launches(g, nt, [&](unsigned nb) { go(g, nb, nt); });
}

}  // namespace mxq
