// Rows of 16-bit elements held in registers, 8 to a vector: loads and stores at
// the alignment of an element, and sums over the lanes and waves of a row.
#pragma once

#include "fc_device.h"

namespace fc {
namespace {

// vectors at the alignment of their elements
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

// Sum over rows of 16 lanes, the same bits in every lane of a row: butterflies
// in which both partners add the same pair.
__device__ __forceinline__ float row_sum(float v) {
    v += dpp<0xB1>(v);    // lane ^ 1
    v += dpp<0x4E>(v);    // lane ^ 2
    v += dpp<0x141>(v);   // 7 - i inside 8 lanes
    v += dpp<0x140>(v);   // 15 - i inside 16 lanes
    return v;
}

// Sum over the wave: the four rows' sums in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
    const int b = __builtin_bit_cast(int, row_sum(v));
    const float a0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
    const float a1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
    const float a2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
    const float a3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
    return (a0 + a1) + (a2 + a3);
}

// Sum over the workgroup's nw <= 16 waves, the same bits in every thread.
// `part` is this reduction's own LDS (one float per wave): no barrier is
// needed after it.
__device__ __forceinline__ float block_sum(float v, float *part, uint32_t nw) {
    v = wave_sum(v);
    if (nw > 1) {
        const uint32_t tid = __builtin_amdgcn_workitem_id_x(), i = tid & 15u;
        if ((tid & (kWave - 1)) == 0) part[tid / kWave] = v;
        __syncthreads();
        v = i < nw ? part[i] : 0.0f;
        v = row_sum(v);
    }
    return v;
}

template <int DT>
__device__ __forceinline__ float widen1(uint16_t b) {
    if constexpr (DT == 1) return __builtin_bit_cast(float, (uint32_t)b << 16);
    else return (float)__builtin_bit_cast(_Float16, b);
}

template <int DT>
__device__ __forceinline__ uint16_t narrow1(float v) {
    if constexpr (DT == 1) return __builtin_bit_cast(uint16_t, (__bf16)as_f32(v));
    else return __builtin_bit_cast(uint16_t, (_Float16)as_f32(v));
}

// The 8 elements from b of a row of H; of a row shorter than that, those it has.
__device__ __forceinline__ u32x4 load_row8(const uint16_t *row, int b, int H) {
    if (H >= kLaneElems) return *reinterpret_cast<const u32x4_a2 *>(row + b);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k)
        if (k < H) w[k / 2] |= (uint32_t)row[k] << (16 * (k & 1));
    return u32x4{w[0], w[1], w[2], w[3]};
}

// v[k] is element b + k; the lane's own are those from e to the row's end.
template <int DT>
__device__ __forceinline__ void store_row8(uint16_t *row, int e, int b, int H, const float (&v)[kLaneElems]) {
    if (e + kLaneElems <= H) {
        *reinterpret_cast<u32x4_a2 *>(row + e) = narrow8<DT>(v);
        return;
    }
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k)
        if (b + k >= e && b + k < H) row[b + k] = narrow1<DT>(v[k]);
}

// n / d by the reciprocal ceil(2^32 / d), exact while n * d < 2^32; 0 stands
// for d = 1, whose reciprocal does not fit.
__device__ __forceinline__ uint32_t group_of(uint32_t n, uint32_t magic) {
    return magic ? __umulhi(n, magic) : n;
}

// Sum over L = 2^llog lanes (L <= 64, aligned), the same bits in each of them.
__device__ __forceinline__ float lanes_sum(float v, int llog) {
    if (llog >= 1) v += dpp<0xB1>(v);
    if (llog >= 2) v += dpp<0x4E>(v);
    if (llog >= 3) v += dpp<0x141>(v);
    if (llog >= 4) v += dpp<0x140>(v);
    if (llog >= 5)   // lane ^ 16
        v += __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F));
    if (llog >= 6) {   // lane ^ 32
        const uint32_t b = __builtin_bit_cast(uint32_t, v);
        const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
        v = __builtin_bit_cast(float, (uint32_t)h[0]) + __builtin_bit_cast(float, (uint32_t)h[1]);
    }
    return v;
}

// 2^result lanes hold n vectors (n <= 64).
inline int lanes_log(int n) {
    int l = 0;
    while ((1 << l) < n) ++l;
    return l;
}

}  // namespace
}  // namespace fc
