// linear_inst.hip - one form (MXQ_FORM) of the linear layers' products on every tile.
#include "gemm_plan.h"
#include "linear_gemm.h"

namespace mxq {

template <class F> void by_act(int act, F f) {
    if (act == MXQ_ACT_RELU) f(std::integral_constant<int, MXQ_ACT_RELU>());
    else if (act == MXQ_ACT_SILU) f(std::integral_constant<int, MXQ_ACT_SILU>());
    else if (act == MXQ_ACT_GELU) f(std::integral_constant<int, MXQ_ACT_GELU>());
    else if (act == MXQ_ACT_GELU_TANH) f(std::integral_constant<int, MXQ_ACT_GELU_TANH>());
    else f(std::integral_constant<int, MXQ_ACT_NONE>());
}

template <int FORM> hipError_t linear_gemm(const LinearGemm& g0, int tile, int splits, hipStream_t st) {
    constexpr bool TA = FORM == FORM_TN || FORM == FORM_TT, TB = FORM == FORM_TT, P = FORM == FORM_PAIRED;
    if constexpr (!TB) {
        auto stream = [&](auto c) {
            using C = decltype(c);
            LinearGemm g = g0;
            // as many rows to every CU
            const int64_t rounds = ceil_div(g.M * splits, 256 * C::BM);
            g.stride = ceil_div(ceil_div(g.M * splits, 256 * rounds), 16) * 16;
            if (g.stride > C::BM) g.stride = C::BM;
            g.ntm = ceil_div(g.M, g.stride);
            g.ntn = ceil_div(g.N, C::BN);
            g.per = ceil_div(ceil_div(g.K, KT), splits);
            g.splits = splits;
            return launches(g, threads_of<C>(), [&](unsigned nb) { k_linear_stream<C, TA, P><<<nb, threads_of<C>(), 0, st>>>(g); });
        };
        if (tile == WIDE64) return stream(Wide64());
        if (tile == WIDE32) return stream(Wide32());
        if (tile == WIDE128) return stream(Wide128());
        if constexpr (!TA) {
            if (tile == QUICK32) return stream(Quick32());
            if (tile == QUICK64) return stream(Quick64());
        }
    }
    return on_tiles(g0, Choice{tile, splits}, [&](const LinearGemm& g, unsigned nb, int nt) {
        auto pipe = [&](auto act, auto grad) {
            constexpr int ACT = decltype(act)::value, GRAD = decltype(grad)::value;
            if (tile == BIG) k_linear_pipe<256, TA, TB, P, ACT, GRAD><<<nb, nt, 0, st>>>(g);
            else k_linear_pipe<192, TA, TB, P, ACT, GRAD><<<nb, nt, 0, st>>>(g);
        };
        if (tile == BIG || tile == SLIM) {
            constexpr std::integral_constant<int, 0> no;
            constexpr std::integral_constant<int, 1> yes;
            // partial sums take no activation
            if constexpr (TA) pipe(no, no);
            else by_act(g.part ? (int)MXQ_ACT_NONE : g.act, [&](auto act) {
                if constexpr (P) {
                    if (g.dh) pipe(act, yes);
                    else pipe(act, no);
                } else {
                    pipe(act, no);
                }
            });
        } else if (tile == MID) k_linear_gemm<Mid, TA, TB, P><<<nb, nt, 0, st>>>(g);
        else if (tile == TINY) k_linear_gemm<Tiny, TA, TB, P><<<nb, nt, 0, st>>>(g);
        else if (tile == DEEP) k_linear_gemm<Deep, TA, TB, P><<<nb, nt, 0, st>>>(g);
        else if constexpr (!TA) k_linear_gemm<Lone, TA, TB, P><<<nb, nt, 0, st>>>(g);
    });
}
template hipError_t linear_gemm<MXQ_FORM>(const LinearGemm&, int, int, hipStream_t);

}  // namespace mxq
