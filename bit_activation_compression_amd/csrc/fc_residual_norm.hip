// Block norms of a 16-bit block output (include/fc/layer.h, fc_residual_norm):
// the kernel is in fc_norm.h.
#include "fc_norm.h"

namespace fc {

hipError_t launch_residual_norm(const NormArgs &a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_norm_any<0, 0, false>(a, stream) : launch_norm_any<1, 0, false>(a, stream);
}

}  // namespace fc
