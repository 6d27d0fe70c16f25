// The gradient of a linear layer's weights, dw = dy^T x, from the INT8 payload of x
// (include/fc/train.h, fc_linear_weight_grad): both operands are read down their
// columns, and the codes become 16-bit values on their way into LDS. The kernel is
// in fc_product.h.
#include "fc_product.h"

namespace fc {
namespace {

template <int DT>
hipError_t run(const ProductArgs &a, hipStream_t stream) {
    if (a.M % kChunk == 0) return launch_product<DT, kCols, kCodes, 128, 128, 2, 2, true, true>(a, stream);
    return launch_product<DT, kCols, kCodes, 128, 128, 2, 2, false, true>(a, stream);
}

// dw (+)= the sum of the splits' parts, in their order
__global__ __launch_bounds__(kBlockThreads) void join_kernel(const float *part, int split, uint64_t n, int accumulate, float *dw) {
    const uint64_t i = grid_index() * kBlockThreads + __builtin_amdgcn_workitem_id_x();
    if (i >= n) return;
    float s = part[i];
    for (int p = 1; p < split; ++p) s += part[(uint64_t)p * n + i];
    dw[i] = accumulate ? dw[i] + s : s;
}

}  // namespace

int weight_grad_splits(int R, int T, int K, int H) {
    return 1;
}

hipError_t launch_linear_weight_grad(const uint16_t *dy, const Payload &px, int group, int dtype, int R,
                                     int T, int K, int H, int accumulate, float *dw, float *part,
                                     hipStream_t stream) {
    ProductArgs p = {};
    p.a = dy;
    p.pb = px;
    p.group = group;
    p.R = R;
    p.M = H;
    p.N = K;
    p.K = T;
    p.split = weight_grad_splits(R, T, K, H);
    const int stages = (T - 1) / kStageK + 1;
    p.split_k = (stages + p.split - 1) / p.split * kStageK;
    p.split = (T - 1) / p.split_k + 1;   // no run is empty
    p.out = p.split > 1 ? part : dw;
    p.accumulate = p.split > 1 ? 0 : accumulate;
    hipError_t err = dtype == 0 ? run<0>(p, stream) : run<1>(p, stream);
    if (err != hipSuccess || p.split == 1) return err;
    const uint64_t n = (uint64_t)R * (uint64_t)H * (uint64_t)K;
    hipLaunchKernelGGL(join_kernel, grid_of_blocks((n + kBlockThreads - 1) / kBlockThreads), dim3(kBlockThreads), 0, stream,
                       part, p.split, n, accumulate, dw);
    return hipGetLastError();
}

}  // namespace fc
