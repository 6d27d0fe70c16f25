// Linear layer on MXFP4 operands (include/fc/layer.h): y[r] = a[r] w[r]^T on
// the scaled matrix cores, v_mfma_scale_f32_16x16x128_f8f6f4 with both
// operands FP4: lane l holds row l % 16 of its operand at k = 32 (l / 16) +
// 0..31, 16 bytes of codes and one scale byte, which is one block of the format.
//
// The row operand is w (16 channels) and the column operand a (16 tokens), so
// a lane's four accumulators are 4 consecutive channels of one token.
#include "fc_launch.h"
#include "fc_mxfp4.h"

namespace fc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kFp4 = 4;   // operand format of the f8f6f4 instructions

__device__ __forceinline__ i32x8 operand(const u32x4 &v) {
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

__device__ __forceinline__ f32x4 mfma_mx(const u32x4 &w, const u32x4 &a, const f32x4 &c, uint32_t sw,
                                         uint32_t sa) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(a), c, kFp4, kFp4, 0,
                                                            (int)sw, 0, (int)sa);
}

template <int DT>
__device__ __forceinline__ uint16_t round1(float v) {
    if constexpr (DT == 1) return __builtin_bit_cast(uint16_t, (__bf16)as_f32(v));
    else return __builtin_bit_cast(uint16_t, (_Float16)as_f32(v));
}

template <int DT>
__global__ __launch_bounds__(kBlockThreads) void matmul_mxfp4_kernel(
    const uint8_t *__restrict__ ac, const uint8_t *__restrict__ as, const uint8_t *__restrict__ wc,
    const uint8_t *__restrict__ ws, int T, int Kp, int H, int tiles_t, int tiles_h,
    uint64_t tiles, uint16_t *__restrict__ y) {
    const int lane = lane_id();
    const uint64_t tile = wave_index();
    if (tile >= tiles) return;
    const uint32_t per_rank = (uint32_t)tiles_t * (uint32_t)tiles_h;
    const uint32_t r = (uint32_t)(tile / per_rank);
    const uint32_t i = (uint32_t)(tile - (uint64_t)r * per_rank);
    const int h0 = (int)(i / (uint32_t)tiles_t) * 16, t0 = (int)(i % (uint32_t)tiles_t) * 16;
    const int row = lane & 15, kb = lane >> 4;
    const int hr = h0 + row < H ? h0 + row : H - 1;
    const int tr = t0 + row < T ? t0 + row : T - 1;
    const uint64_t wrow = (uint64_t)r * (uint32_t)H + (uint32_t)hr, arow = (uint64_t)r * (uint32_t)T + (uint32_t)tr;
    const uint8_t *wcp = wc + wrow * (uint32_t)(Kp / 2) + kb * 16, *acp = ac + arow * (uint32_t)(Kp / 2) + kb * 16;
    const uint8_t *wsp = ws + wrow * (uint32_t)(Kp / 32) + kb, *asp = as + arow * (uint32_t)(Kp / 32) + kb;
    f32x4 acc = {};
    for (int k = 0; k < Kp / kMxStepElems; ++k) {
        acc = mfma_mx(*reinterpret_cast<const u32x4 *>(wcp + k * 64), *reinterpret_cast<const u32x4 *>(acp + k * 64),
                      acc, wsp[k * 4], asp[k * 4]);
    }
    const int t = t0 + row;
    if (t >= T) return;
    uint16_t *yr = y + ((uint64_t)r * (uint32_t)T + (uint32_t)t) * (uint32_t)H;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int h = h0 + 4 * kb + j;
        if (h < H) yr[h] = round1<DT>(acc[j]);
    }
}

}  // namespace

hipError_t launch_matmul_mxfp4(const uint8_t *a_codes, const uint8_t *a_scales,
                               const uint8_t *w_codes, const uint8_t *w_scales, int R, int T, int Kp,
                               int H, int dtype, uint16_t *y, hipStream_t stream) {
    const int tiles_t = (T + 15) / 16, tiles_h = (H + 15) / 16;
    const uint64_t tiles = (uint64_t)R * (uint64_t)tiles_t * (uint64_t)tiles_h;
    const unsigned blocks = (unsigned)((tiles + kWavesPerBlock - 1) / kWavesPerBlock);
    auto kernel = dtype == 0 ? matmul_mxfp4_kernel<0> : matmul_mxfp4_kernel<1>;
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kBlockThreads), 0, stream, a_codes, a_scales, w_codes,
                       w_scales, T, Kp, H, tiles_t, tiles_h, tiles, y);
    return hipGetLastError();
}

}  // namespace fc
