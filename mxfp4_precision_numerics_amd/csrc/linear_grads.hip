// linear_grads.hip - both gradients' products of a linear layer in one launch.
#include "gemm_plan.h"
#include "linear_gemm.h"

namespace mxq {

// Tiles and splits are set in x and w; the product whose blocks take longer goes first.
hipError_t linear_grads(const LinearGemm& x, int x_tile, const LinearGemm& w, int w_tile, const ColumnSums& b, hipStream_t st) {
    const uint32_t nx = (uint32_t)(x.ntm * x.ntn * x.splits), nw = (uint32_t)(w.ntm * w.ntn * w.splits);
    const uint32_t nb = b.out ? (uint32_t)ceil_div(b.N, 32) : 0u;
    const int w_first = TILES[w_tile].tk * w.per > TILES[x_tile].tk * x.per;
    const uint32_t n0 = w_first ? nw : nx, n = nb + nx + nw;
    if (pipelined(x_tile)) {
        auto go = [&](auto bx, auto bw) {
            k_linear_grads_pipe<decltype(bx)::value, decltype(bw)::value><<<n, 512, 0, st>>>(x, w, b, n0, nx + nw, w_first);
        };
        constexpr std::integral_constant<int, 256> big;
        constexpr std::integral_constant<int, 192> slim;
        if (x_tile == BIG) w_tile == BIG ? go(big, big) : go(big, slim);
        else w_tile == BIG ? go(slim, big) : go(slim, slim);
    } else if (x_tile == MID && w_tile == MID) k_linear_grads<Mid, Mid><<<n, threads_of<Mid>(), 0, st>>>(x, w, b, nb, n0, w_first);
    else if (x_tile == MID) k_linear_grads<Mid, Tiny><<<n, threads_of<Mid>(), 0, st>>>(x, w, b, nb, n0, w_first);
    else if (w_tile == MID) k_linear_grads<Tiny, Mid><<<n, threads_of<Mid>(), 0, st>>>(x, w, b, nb, n0, w_first);
    else k_linear_grads<Tiny, Tiny><<<n, threads_of<Tiny>(), 0, st>>>(x, w, b, nb, n0, w_first);
    return hipGetLastError();
}

}  // namespace mxq
