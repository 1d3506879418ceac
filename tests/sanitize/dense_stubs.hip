// dense_stubs.hip - stand-ins for the launchers behind include/mxq_dense.h, for
// the sanitizer build of its host validation (dense_api.hip) on a machine
// without a GPU.  Test infrastructure: a call that passes validation reports
// no device, one without rows succeeds as the launchers do.
#include <hip/hip_runtime.h>

#include "../../mxfp4_precision_numerics_amd/csrc/dense_launch.h"

namespace mxq {

int64_t linear_bytes(int64_t T, int64_t H, int64_t N, int64_t, bool backward) {
    return T == 0 ? 0 : backward ? T * N * 2 + 256 : T * N <= 1 << 20 && H >= 16384 ? T * N * 8 : 0;
}
hipError_t launch_linear(const LinearArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_linear_backward(const LinearArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_adamw(const AdamwArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_grad_norm(const mxq_clip_tensor*, const int32_t*, int64_t, float*, double*, hipStream_t) {
    return hipErrorNoDevice;
}

}  // namespace mxq
