// The linear layer with bias, activation, second factor and residual in the
// product's epilogue (include/fc/train.h, fc_linear_act); the kernel is in
// fc_product.h.
#include "fc_product.h"

namespace fc {
namespace {

template <int DT>
hipError_t run(const ProductArgs &a, hipStream_t stream) {
    if (a.K % kChunk == 0) return launch_tiles<DT, kRows, kRows, true, false>(a, stream);
    return launch_tiles<DT, kRows, kRows, false, false>(a, stream);
}

}  // namespace

hipError_t launch_linear_act(const uint16_t *a, const uint16_t *w, int dtype, int R, int T, int K, int H,
                             const LinearEpilogue &e, hipStream_t stream) {
    ProductArgs p = {};
    p.a = a;
    p.b = w;
    p.R = R;
    p.M = T;
    p.N = H;
    p.K = K;
    p.split = 1;
    p.split_k = K;
    p.e = e;
    return dtype == 0 ? run<0>(p, stream) : run<1>(p, stream);
}

}  // namespace fc
