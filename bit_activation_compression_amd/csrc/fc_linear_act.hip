// The linear layer with bias, activation, second factor and residual in the
// product's epilogue (include/fc/train.h, fc_linear_act). The product of many tokens is
// in fc_product.h; the one of few tokens is here: it is bound by the weights' stream,
// and stages nothing in LDS.
#include "fc_product.h"

namespace fc {
namespace {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * kWave;
constexpr int kFewRows = 16;     // output channels of a workgroup
constexpr int kPiece = 64;       // k that a wave takes at a time: a line of each row
constexpr int kAhead = 4;        // pieces in flight

// 8 values at k of a row of K, zeros past its end.
__device__ __forceinline__ u32x4 row_values(const uint16_t *row, int k, int K) {
    if (k + kChunk <= K) return *reinterpret_cast<const u32x4_a2 *>(row + k);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
        if (k + i < K) w[i / 2] |= (uint32_t)row[k + i] << (16 * (i & 1));
    return u32x4{w[0], w[1], w[2], w[3]};
}

// A workgroup has 16 output channels of one rank, as the rows of the matrix
// instruction, and the tokens (up to 16) as its columns. Its waves take every eighth
// line of the rows' k, their sums meet in LDS in the order of the waves. One token,
// K = 8192, H = 7168 bf16: 27 us, 4.3 TB/s. Four waves or 16, two or eight lines in
// flight are as fast or up to 60% slower on some of eight shapes, loads past the caches
// 5 to 10% slower.
template <int DT>
__global__ __launch_bounds__(kFewThreads) void linear_few_kernel(const uint16_t *a, const uint16_t *w, int R, int T, int K, int H,
                                                                 LinearEpilogue e) {
    __shared__ f32x4 lds[kFewWaves][kWave];
    const uint32_t tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63u;
    const int wave = (int)__builtin_amdgcn_readfirstlane(tid >> 6);
    const uint64_t id = grid_index();
    const uint32_t groups = ((uint32_t)H + kFewRows - 1) / kFewRows;
    const uint64_t r = id / groups;
    if (r >= (uint64_t)R) return;
    const int h0 = (int)(id - r * groups) * kFewRows;
    const int h = h0 + (int)(lane & 15u), t = (int)(lane & 15u), g = (int)(lane >> 4) * kChunk;
    // channels and tokens that are not there read the last one's values: their results
    // are not stored
    const uint16_t *wr = w + (r * (uint32_t)H + (uint32_t)(h < H ? h : H - 1)) * (uint64_t)K;
    const uint16_t *ar = a + (r * (uint32_t)T + (uint32_t)(t < T ? t : T - 1)) * (uint64_t)K;
    f32x4 acc = {};
    const int whole = K / kPiece;
    for (int c = wave; c < whole; c += kFewWaves * kAhead) {
        u32x4 wv[kAhead][2], av[kAhead][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int p = c + u * kFewWaves < whole ? c + u * kFewWaves : c;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                wv[u][i] = *reinterpret_cast<const u32x4_a2 *>(wr + p * kPiece + i * kStepK + g);
                av[u][i] = *reinterpret_cast<const u32x4_a2 *>(ar + p * kPiece + i * kStepK + g);
            }
        }
        __builtin_amdgcn_sched_barrier(0);   // all of them in flight before the first use
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (c + u * kFewWaves >= whole) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) acc = mfma<DT>(wv[u][i], av[u][i], acc);
        }
    }
    if (whole * kPiece < K && wave == whole % kFewWaves) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = whole * kPiece + i * kStepK + g;
            acc = mfma<DT>(row_values(wr, k, K), row_values(ar, k, K), acc);
        }
    }
    lds[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) acc += lds[i][lane];
    const int n = h0 + (int)(lane >> 4) * 4, left = H - n;
    if (t >= T || left <= 0) return;
    float bias[4] = {}, v[4] = {acc.x, acc.y, acc.z, acc.w};
    if (e.bias != nullptr) widen4<DT>(e.bias + r * (uint32_t)H + (uint32_t)n, left, bias);
    finish4<DT>(e, (r * (uint32_t)T + (uint32_t)t) * (uint32_t)H + (uint32_t)n, left, bias, v);
}

template <int DT>
hipError_t run(const ProductArgs &a, float *part, hipStream_t stream) {
    if (a.M <= kFewTokens) {
        const uint64_t blocks = (uint64_t)a.R * (((uint32_t)a.N + kFewRows - 1) / kFewRows);
        hipLaunchKernelGGL((linear_few_kernel<DT>), grid_of_blocks(blocks), dim3(kFewThreads), 0, stream, a.a, a.b, a.R, a.M, a.K,
                           a.N, a.e);
        return hipGetLastError();
    }
    const SplitPlan plan = linear_plan(a.R, a.M, a.N, a.K);
    if (a.K % kChunk == 0) return launch_split<DT, kRows, kRows, true>(a, plan, part, stream);
    return launch_split<DT, kRows, kRows, false>(a, plan, part, stream);
}

}  // namespace

hipError_t launch_linear_act(const uint16_t *a, const uint16_t *w, int dtype, int R, int T, int K, int H,
                             const LinearEpilogue &e, void *workspace, hipStream_t stream) {
    ProductArgs p = {};
    p.a = a;
    p.b = w;
    p.R = R;
    p.M = T;
    p.N = H;
    p.K = K;
    p.e = e;
    float *part = static_cast<float *>(workspace);
    return dtype == 0 ? run<0>(p, part, stream) : run<1>(p, part, stream);
}

}  // namespace fc
