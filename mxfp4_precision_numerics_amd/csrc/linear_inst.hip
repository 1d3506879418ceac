// linear_inst.hip - one form (MXQ_FORM) of the linear layers' products on every tile.
#include "gemm_plan.h"
#include "linear_gemm.h"

namespace mxq {

template <int FORM> hipError_t linear_gemm(const LinearGemm& g0, int tile, int splits, hipStream_t st) {
    constexpr bool TA = FORM == FORM_TN || FORM == FORM_TT, TB = FORM == FORM_TT, P = FORM == FORM_PAIRED;
    return on_tiles(g0, Choice{tile, splits}, [&](const LinearGemm& g, unsigned nb, int nt) {
        if (tile == BIG) k_linear_pipe<256, TA, TB, P><<<nb, nt, 0, st>>>(g);
        else if (tile == SLIM) k_linear_pipe<192, TA, TB, P><<<nb, nt, 0, st>>>(g);
        else if (tile == MID) k_linear_gemm<Mid, TA, TB, P><<<nb, nt, 0, st>>>(g);
        else if (tile == TINY) k_linear_gemm<Tiny, TA, TB, P><<<nb, nt, 0, st>>>(g);
        else if (tile == DEEP) k_linear_gemm<Deep, TA, TB, P><<<nb, nt, 0, st>>>(g);
        else if constexpr (!TA) k_linear_gemm<Lone, TA, TB, P><<<nb, nt, 0, st>>>(g);
    });
}
template hipError_t linear_gemm<MXQ_FORM>(const LinearGemm&, int, int, hipStream_t);

}  // namespace mxq
