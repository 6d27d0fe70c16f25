// The gradient of a linear layer's input, dx = dy w (include/fc/train.h,
// fc_linear_input_grad): the weights [H][K] are read down their columns. The kernel
// is in fc_product.h.
#include "fc_product.h"

namespace fc {
namespace {

template <int DT>
hipError_t run(const ProductArgs &a, float *part, hipStream_t stream) {
    const SplitPlan plan = linear_plan(a.R, a.M, a.N, a.K);
    if (a.K % kChunk == 0 && a.N % kChunk == 0) return launch_split<DT, kRows, kCols, true>(a, plan, part, stream);
    return launch_split<DT, kRows, kCols, false>(a, plan, part, stream);
}

}  // namespace

hipError_t launch_linear_input_grad(const uint16_t *dy, const uint16_t *w, int dtype, int R, int T, int K,
                                    int H, const uint16_t *residual, uint16_t *dx, void *workspace,
                                    hipStream_t stream) {
    ProductArgs p = {};
    p.a = dy;
    p.b = w;
    p.R = R;
    p.M = T;
    p.N = K;
    p.K = H;
    p.e.residual = residual;
    p.e.y = dx;
    float *part = static_cast<float *>(workspace);
    return dtype == 0 ? run<0>(p, part, stream) : run<1>(p, part, stream);
}

}  // namespace fc
