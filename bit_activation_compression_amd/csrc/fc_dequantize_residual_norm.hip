// Block norms of the all-gathered payload (include/fc/layer.h,
// fc_dequantize_residual_norm): the last step of the two-step all-reduce of
// "Flash Communication: Reducing Tensor Parallelization Bottleneck for Fast
// Large Language Model Inference" (Figure 5, right) with the residual update
// and the norms that follow it in the block (Figure 3). The kernel is in
// fc_norm.h.
#include "fc_norm.h"

namespace fc {
namespace {

template <int DT, int BITS>
hipError_t by_group(NormArgs a, int group, hipStream_t stream) {
    // groups counted in vectors of 8, or in pairs where they are not whole vectors
    const bool gen = group % kLaneElems != 0;
    const uint32_t d = (uint32_t)(gen ? group / 2 : group / kLaneElems);
    a.groups = a.H / group;
    a.gmagic = d == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + d - 1) / d);
    return gen ? launch_norm_any<DT, BITS, true>(a, stream) : launch_norm_any<DT, BITS, false>(a, stream);
}

}  // namespace

hipError_t launch_dequantize_residual_norm(const NormArgs &a, int dtype, int bits, int group,
                                           hipStream_t stream) {
    if (dtype == 0) return bits == 4 ? by_group<0, 4>(a, group, stream) : by_group<0, 8>(a, group, stream);
    return bits == 4 ? by_group<1, 4>(a, group, stream) : by_group<1, 8>(a, group, stream);
}

}  // namespace fc
