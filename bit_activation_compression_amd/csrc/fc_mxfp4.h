// MXFP4 helpers shared by the quantizer and the product (include/fc/layer.h):
// 32 values of a row share a scale 2^E, stored as the byte E + 127 (255: NaN),
// and a value is an E2M1 code: sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6.
#pragma once

#include "fc_device.h"

namespace fc {

constexpr int kMxBlockElems = 32;   // values per scale
constexpr int kMxStepElems = 128;   // rows are padded to a multiple of this

// --- the scaled matrix cores (v_mfma_scale_f32_*_f8f6f4) ---
typedef int i32x8 __attribute__((ext_vector_type(8)));
constexpr int kFp4 = 4;                   // operand format
// a lane's 32 FP4 codes as the instruction's operand of up to 8 bits a value
__device__ __forceinline__ i32x8 mx_operand(const u32x4 &v) {
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}
// buffer resource word 3 for raw (untyped, unswizzled) 32-bit-addressed
// buffers on gfx9-family GPUs
constexpr int kRawBufferFlags = 0x00020000;
constexpr uint32_t kPast = 0xFFFFFFF0u;   // an offset past every resource

// 8 elements of 16 bits at the alignment of one (one global_load_dwordx4)
typedef u32x4 u32x4_u16 __attribute__((aligned(2)));

// Larger magnitude of each 16-bit half, as unsigned numbers (the order of the
// magnitudes, with infinities and then NaNs at the top).
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

__device__ __forceinline__ uint32_t abs_max8(const u32x4 &v) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    return pk_max(pk_max(v.x & kAbs, v.y & kAbs), pk_max(v.z & kAbs, v.w & kAbs));
}

// The scale byte of a block whose largest magnitude has the dtype's bits
// `top`: E + 127 = max(exponent field of its binary32 form - 2, 0). A bf16
// subnormal's field is 0 and floor(log2) - 2 lies below -127 as well; an fp16
// one is a normal binary32. A block with an infinity or a NaN: 255.
template <int DT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    uint32_t field;
    if constexpr (DT == 1) {
        field = top >> 7;
    } else {
        const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)top);
        field = __builtin_bit_cast(uint32_t, f) >> 23;
    }
    const uint32_t byte = field > 2 ? field - 2 : 0u;
    return top >= (DT == 1 ? 0x7F80u : 0x7C00u) ? 255u : byte;
}

// The binary32 number whose exponent field is the scale byte: 2^E, where the
// conversions below take only the field (byte 0 is 2^-127 to them).
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// Codes of 8 values (v_cvt_scalef32_pk_fp4_{bf16,f16}: x / 2^E rounded half to
// even to E2M1, saturating), element 2i in the low nibble of byte i.
template <int DT>
__device__ __forceinline__ uint32_t mx_encode8(const u32x4 &v, float scale) {
    // (named words: a bit cast of a vector's element takes its first word)
    const uint32_t w0 = v.x, w1 = v.y, w2 = v.z, w3 = v.w;
    uint32_t q = 0;
    if constexpr (DT == 1) {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w0), scale, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w1), scale, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w2), scale, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w3), scale, 3);
    } else {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w0), scale, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w1), scale, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w2), scale, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w3), scale, 3);
    }
    return q;
}

// 8 values from element e of a row of K, zeros past its end.
__device__ __forceinline__ u32x4 mx_load8(const uint16_t *row, uint32_t e, uint32_t K) {
    if (e + kLaneElems <= K) return *reinterpret_cast<const u32x4_u16 *>(row + e);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t k = 0; k < kLaneElems; ++k)
        if (e + k < K) w[k / 2] |= (uint32_t)row[e + k] << (16 * (k & 1));
    return u32x4{w[0], w[1], w[2], w[3]};
}

// The scale byte of the block that 4 neighbouring lanes hold, 8 values each.
template <int DT>
__device__ __forceinline__ uint32_t mx_block_scale(const u32x4 &v) {
    uint32_t m = abs_max8(v);
    m = pk_max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));   // lane ^ 1
    m = pk_max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));   // lane ^ 2
    return mx_scale_byte<DT>((m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16));
}

// Two binary32 sums rounded to the dtype, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t mx_round2(float a, float b) {
    const f32x2 pair = {as_f32(a), as_f32(b)};
    if constexpr (DT == 1) return __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, bf16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, f16x2));
}

}  // namespace fc
