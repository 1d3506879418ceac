// train_stubs.hip - stand-ins for the launchers behind include/mxq_train.h, for
// the sanitizer build of its host validation (train_api.hip) on a machine
// without a GPU.  Test infrastructure: a call that passes validation reports
// no device.
#include <hip/hip_runtime.h>

#include "../../mxfp4_precision_numerics_amd/csrc/train_launch.h"

namespace mxq {

hipError_t launch_moe_topk(const void*, int, int64_t, int64_t, int64_t, int, int, int32_t*, float*, hipStream_t) {
    return hipErrorNoDevice;
}
hipError_t launch_moe_topk_backward(const void*, int, int64_t, int64_t, int64_t, const int32_t*, int, int,
                                    const float*, void*, int64_t, hipStream_t) {
    return hipErrorNoDevice;
}
int64_t moe_sort_bytes(int64_t n, int64_t G) { return n > 4096 ? n / 1024 * G * 4 : 0; }
hipError_t launch_moe_sort(const int32_t*, int64_t, int, int, int64_t*, int32_t*, int32_t*, void*, hipStream_t) {
    return hipErrorNoDevice;
}
hipError_t launch_moe_dispatch_mx(const void*, int, int64_t, int64_t, int64_t, const int32_t*, int, int, int64_t,
                                  uint8_t*, uint8_t*, hipStream_t) {
    return hipErrorNoDevice;
}
hipError_t launch_moe_combine(const void*, int, int64_t, int64_t, int64_t, const int32_t*, int64_t, int, const float*,
                              void*, int64_t, hipStream_t) {
    return hipErrorNoDevice;
}
hipError_t launch_moe_combine_backward(const void*, int, int64_t, int64_t, int64_t, const int32_t*, int, const float*,
                                       const void*, int64_t, int64_t, void*, int64_t, float*, hipStream_t) {
    return hipErrorNoDevice;
}
int64_t lce_bytes(int64_t T, int64_t, int64_t V, bool backward) { return (T + V) * (backward ? 8 : 4) + 256; }
hipError_t launch_lce(const LceArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_lce_backward(const LceArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_clip(const mxq_clip_tensor*, const int32_t*, int64_t, float, float*, double*, hipStream_t) {
    return hipErrorNoDevice;
}

}  // namespace mxq
