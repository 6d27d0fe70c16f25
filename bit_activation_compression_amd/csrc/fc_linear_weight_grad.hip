// The gradient of a linear layer's weights, dw = dy^T x, from the INT8 payload of x
// (include/fc/train.h, fc_linear_weight_grad): both operands are read down their
// columns. The codes become 16-bit values on their way into LDS, or, where many rows of
// tiles would each do that again, in a launch of the dequantizer before the product.
// Sums over many tokens for few outputs are split, and joined in a fixed order. The
// kernel is in fc_product.h, the rules are in fc_product_dispatch.h.
#include "fc_launch.h"
#include "fc_product.h"

namespace fc {
namespace {

template <int DT>
hipError_t run(const ProductArgs &a, hipStream_t stream) {
    const bool direct = a.M % kChunk == 0;   // and columns are whole chunks: groups are
    if (a.b != nullptr) return launch_tiles<DT, kCols, kCols, true, true>(a, stream);   // the plan's H % 8 == 0
    return direct ? launch_tiles<DT, kCols, kCodes, true, true>(a, stream) : launch_tiles<DT, kCols, kCodes, false, true>(a, stream);
}

// dw (+)= the sum of the splits' parts, in their order
__global__ __launch_bounds__(kBlockThreads) void join_kernel(const float *part, int split, uint64_t n, int accumulate, float *dw) {
    const uint64_t i = grid_index() * kBlockThreads + __builtin_amdgcn_workitem_id_x();
    if (i >= n) return;
    float s = 0.0f;
    for (int p = 0; p < split; p += 8) {   // 8 loads in flight at a time
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = p + k < split ? part[(uint64_t)(p + k) * n + i] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k];
    }
    dw[i] = accumulate ? dw[i] + s : s;
}

}  // namespace

hipError_t launch_linear_weight_grad(const uint16_t *dy, const Payload &px, int group, int dtype, int R,
                                     int T, int K, int H, int accumulate, float *dw, void *workspace,
                                     hipStream_t stream) {
    const WeightGradPlan plan = weight_grad_plan(R, T, K, H);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *part = reinterpret_cast<float *>(ws + plan.value_bytes);
    ProductArgs p = {};
    p.a = dy;
    p.R = R;
    p.M = H;
    p.N = K;
    p.K = T;
    p.group = group;
    hipError_t err;
    if (plan.value_bytes != 0) {
        uint16_t *values = reinterpret_cast<uint16_t *>(ws);
        const uint64_t n = (uint64_t)R * (uint64_t)T * (uint64_t)K;
        const bool pow2 = (group & (group - 1)) == 0 && group <= 8192;
        err = pow2 ? launch_dequantize(px.codes, px.s, px.z, n, 8, group, dtype, values, stream)
                   : launch_dequantize_generic(px.codes, px.s, px.z, n, 8, group, dtype, nullptr, values, stream);
        if (err != hipSuccess) return err;
        p.b = values;
    } else {
        p.pb = px;
    }
    p.split = plan.split.split;
    p.split_k = plan.split.split_k;
    p.out = p.split > 1 ? part : dw;
    p.accumulate = p.split > 1 ? 0 : accumulate;
    err = dtype == 0 ? run<0>(p, stream) : run<1>(p, stream);
    if (err != hipSuccess || p.split == 1) return err;
    const uint64_t n = (uint64_t)R * (uint64_t)H * (uint64_t)K;
    hipLaunchKernelGGL(join_kernel, grid_of_blocks((n + kBlockThreads - 1) / kBlockThreads), dim3(kBlockThreads), 0, stream,
                       part, p.split, n, accumulate, dw);
    return hipGetLastError();
}

}  // namespace fc
