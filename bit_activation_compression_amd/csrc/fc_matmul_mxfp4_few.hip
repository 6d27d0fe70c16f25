// Linear layer on MXFP4 weights for few tokens (include/fc/layer.h,
// fc_linear_mxfp4 and fc_matmul_mxfp4): the weights are read once, from HBM
// straight into the matrix cores' registers, and bound the call.
//
// A wave owns 16 channels and all tokens, in column blocks of 16
// (v_mfma_scale_f32_16x16x128_f8f6f4, both operands FP4: lane l holds row l %
// 16 of its operand at k = 32 (l / 16) + 0..31, 16 bytes of codes and one scale
// byte; its four accumulators are channels 4 (l / 16) + 0..3 of token l % 16).
// A step of k = 128 is 64 bytes of a row. Steps are loaded CH at a time, one
// such chunk ahead, so that a wave has up to 2 CH KiB of weights in flight.
// The scales of 4 steps of a row are one 16-byte load.
//
// Where the channels alone would leave the device empty (mxfp4_split_rounds), the
// SPLIT waves of a workgroup share 16 channels and take SPLIT runs of steps;
// the first adds the others' partial sums from LDS, in their order. (1 rank, 1
// token, K = 4096, H = 4096, bf16: 4.5 us, 9.1 unsplit; split over 8 waves 5.6.)
//
// The activations come as codes (from the cache: every wave reads all of
// them) or, where there are few, as 16-bit values that the workgroup
// quantizes into LDS while its first weights are on their way (4 ranks, 1 token,
// K = 2048, H = 8192, bf16: 8.8 us, 4.1 TB/s with the launch's ~2.5 us in it).
#include "fc_grid.h"
#include "fc_launch.h"
#include "fc_mxfp4.h"
#include "fc_mxfp4_dispatch.h"

namespace fc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStepBytes = 64;            // codes of a row in a step
constexpr int kStepScales = 4;
constexpr int kLdsPad = 16;               // spreads the token rows over the banks

struct FewArgs {
    const uint16_t *a;                    // 16-bit activations, or
    const uint8_t *ac, *as;               // their codes and scales
    const uint8_t *wc, *ws;
    uint16_t *y;
    int R, T, K, H;
    int steps;                            // Kp / 128
    int groups;                           // channel groups of a rank
};

__device__ __forceinline__ f32x4 mfma_mx(const u32x4 &w, const u32x4 &a, const f32x4 &c, uint32_t sw,
                                         uint32_t sa) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(w), mx_operand(a), c, kFp4, kFp4, 0, (int)sw, 0,
                                                            (int)sa);
}

__device__ __forceinline__ u32x4 buffer16(const __amdgpu_buffer_rsrc_t &r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// LDS: the quantized activations (T rows of codes, then T rows of scales), or
// the partial sums of split waves; sized at launch
extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];

constexpr int kWaves = 4;

// QUANT: quantize the 16-bit activations (T * Kp <= kMxfp4QuantizeMost)
template <int DT, int NT, int CH, int SPLIT, bool QUANT>
__global__ __launch_bounds__(kWaves *kWave) void matmul_mxfp4_few_kernel(const FewArgs p) {
    static_assert(CH % 4 == 0 && (!QUANT || NT == 1), "");
    constexpr int kUnits = kMxfp4QuantizeMost / (kWaves * kWave * kLaneElems);   // that a thread quantizes
    const uint32_t tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63u;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
    const uint32_t row = lane & 15u, kb = lane >> 4;
    const uint32_t code_row = (uint32_t)p.steps * kStepBytes, scale_row = (uint32_t)p.steps * kStepScales;
    constexpr uint32_t kGroup = kWaves / SPLIT * 16;     // channels of a workgroup
    const uint32_t bid = (uint32_t)grid_index();         // R * groups < 2^31
    const uint32_t r = bid / (uint32_t)p.groups;
    if (r >= (uint32_t)p.R) return;
    const uint32_t h0 = (bid - r * (uint32_t)p.groups) * kGroup + (SPLIT > 1 ? 0u : wave * 16u);
    // this wave's steps
    const uint32_t share = ((uint32_t)p.steps + SPLIT - 1) / SPLIT;
    const uint32_t s0 = SPLIT > 1 ? wave * share : 0u;
    const uint32_t s1 = s0 + share < (uint32_t)p.steps ? s0 + share : (uint32_t)p.steps;

    // resources over the operands' rows from the first needed one on; channels past H read as zeros
    const uint32_t rows = h0 < (uint32_t)p.H ? ((uint32_t)p.H - h0 < 16u ? (uint32_t)p.H - h0 : 16u) : 0u;
    const uint64_t w0 = (uint64_t)r * (uint32_t)p.H + (rows ? h0 : 0u);
    const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(p.wc + w0 * code_row), (short)0, (int)(rows * code_row), kRawBufferFlags);
    const __amdgpu_buffer_rsrc_t wsres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(p.ws + w0 * scale_row), (short)0, (int)(rows * scale_row), kRawBufferFlags);
    const uint64_t a0 = (uint64_t)r * (uint32_t)p.T;
    const __amdgpu_buffer_rsrc_t ares = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(p.ac + a0 * code_row), (short)0, QUANT ? 0 : (int)((uint32_t)p.T * code_row), kRawBufferFlags);
    const __amdgpu_buffer_rsrc_t asres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(p.as + a0 * scale_row), (short)0, QUANT ? 0 : (int)((uint32_t)p.T * scale_row), kRawBufferFlags);
    const uint32_t wo = row * code_row + kb * 16u, wso = row * scale_row;
    // with QUANT, lanes of tokens past T read the last one's row (their outputs are not stored)
    const uint32_t tok = !QUANT || row < (uint32_t)p.T ? row : (uint32_t)p.T - 1u;
    const uint32_t lds_row = code_row + kLdsPad;
    uint8_t *const lds_scales = few_lds + (uint32_t)p.T * lds_row;

    struct Chunk {
        u32x4 w[CH], ws[CH / 4];
        u32x4 a[QUANT ? 1 : CH][NT], as[QUANT ? 1 : CH / 4][NT];
    };
    auto load = [&](Chunk &c, uint32_t s) {
#pragma unroll
        for (uint32_t i = 0; i < CH; ++i) {
            const bool in = s + i < s1;
            if (i % 4 == 0) c.ws[i / 4] = buffer16(wsres, in ? wso + (s + i) * kStepScales : kPast);
            c.w[i] = buffer16(wres, in ? wo + (s + i) * kStepBytes : kPast);
            if constexpr (!QUANT) {
#pragma unroll
                for (uint32_t b = 0; b < NT; ++b) {
                    if (i % 4 == 0)
                        c.as[i / 4][b] = buffer16(asres, in ? wso + b * 16u * scale_row + (s + i) * kStepScales : kPast);
                    c.a[i][b] = buffer16(ares, in ? wo + b * 16u * code_row + (s + i) * kStepBytes : kPast);
                }
            }
        }
    };
    f32x4 acc[NT] = {};
    auto compute = [&](const Chunk &c, uint32_t s) {
#pragma unroll
        for (uint32_t i = 0; i < CH; ++i) {
            if (s + i >= s1) break;
            const uint32_t sw = c.ws[i / 4][i % 4] >> (8u * kb);
#pragma unroll
            for (uint32_t b = 0; b < NT; ++b) {
                u32x4 av;
                uint32_t sa;
                if constexpr (QUANT) {
                    av = *reinterpret_cast<const u32x4 *>(few_lds + tok * lds_row + (s + i) * kStepBytes + kb * 16u);
                    sa = lds_scales[tok * scale_row + (s + i) * kStepScales + kb];
                } else {
                    av = c.a[i][b];
                    sa = c.as[i / 4][b][i % 4] >> (8u * kb);
                }
                acc[b] = mfma_mx(c.w[i], av, acc[b], sw, sa);
            }
        }
    };

    Chunk c0, c1;
    if constexpr (QUANT) {
        // the activations first: loads complete in order
        const uint32_t per_row = (uint32_t)p.steps * (kMxStepElems / kLaneElems);
        const uint32_t units = (uint32_t)p.T * per_row;
        u32x4 v[kUnits];
#pragma unroll
        for (uint32_t u = 0; u < kUnits; ++u) {
            const uint32_t n = u * (kWaves * kWave) + tid;
            v[u] = u32x4{0, 0, 0, 0};
            if (n < units) {
                const uint32_t t = n / per_row, e = (n - t * per_row) * kLaneElems;
                v[u] = mx_load8(p.a + (a0 + t) * (uint32_t)p.K, e, (uint32_t)p.K);
            }
        }
        load(c0, s0);
        load(c1, s0 + CH);
#pragma unroll
        for (uint32_t u = 0; u < kUnits; ++u) {
            const uint32_t n = u * (kWaves * kWave) + tid;
            if (n - (tid & 3u) < units) {     // whole blocks of 4 lanes
                const uint32_t byte = mx_block_scale<DT>(v[u]);
                uint32_t q = mx_encode8<DT>(v[u], mx_scale(byte));
                if (byte == 255u) q = 0;
                const uint32_t t = n / per_row, i = n - t * per_row;
                *reinterpret_cast<uint32_t *>(few_lds + t * lds_row + i * 4u) = q;
                if ((tid & 3u) == 0) lds_scales[t * scale_row + i / 4u] = (uint8_t)byte;
            }
        }
        __syncthreads();
    } else {
        load(c0, s0);
        load(c1, s0 + CH);
    }
    for (uint32_t s = s0; s < s1; s += 2 * CH) {
        compute(c0, s);
        load(c0, s + 2 * CH);
        if (s + CH < s1) compute(c1, s + CH);
        load(c1, s + 3 * CH);
    }

    if constexpr (SPLIT > 1) {
        if constexpr (QUANT) __syncthreads();     // the activations' LDS is used again
        f32x4 *part = reinterpret_cast<f32x4 *>(few_lds);
        if (wave != 0) {
#pragma unroll
            for (uint32_t b = 0; b < NT; ++b) part[((wave - 1) * NT + b) * kWave + lane] = acc[b];
        }
        __syncthreads();
        if (wave != 0) return;
#pragma unroll
        for (uint32_t w = 0; w < SPLIT - 1; ++w)
#pragma unroll
            for (uint32_t b = 0; b < NT; ++b) {
                const f32x4 o = part[(w * NT + b) * kWave + lane];
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[b][k] += o[k];
            }
    }
    const uint32_t h = h0 + 4u * kb;
#pragma unroll
    for (uint32_t b = 0; b < NT; ++b) {
        const uint32_t t = b * 16u + row;
        if (t >= (uint32_t)p.T) continue;
        uint16_t *out = p.y + (a0 + t) * (uint32_t)p.H + h;
        const uint32_t lo = mx_round2<DT>(acc[b][0], acc[b][1]), hi = mx_round2<DT>(acc[b][2], acc[b][3]);
        if (h + 4u <= (uint32_t)p.H) {
            typedef u32x2 u32x2_u16 __attribute__((aligned(2)));
            *reinterpret_cast<u32x2_u16 *>(out) = u32x2{lo, hi};
        } else {
            if (h < (uint32_t)p.H) out[0] = (uint16_t)lo;
            if (h + 1u < (uint32_t)p.H) out[1] = (uint16_t)(lo >> 16);
            if (h + 2u < (uint32_t)p.H) out[2] = (uint16_t)hi;
        }
    }
}

template <int DT, int NT, int CH, int SPLIT, bool QUANT>
hipError_t launch(FewArgs p, int R, hipStream_t stream) {
    constexpr int group = kWaves / SPLIT * 16;
    p.groups = (p.H + group - 1) / group;
    const uint64_t blocks = (uint64_t)R * (uint64_t)p.groups;
    p.R = R;
    const size_t quant = QUANT ? (size_t)p.T * ((size_t)p.steps * (kStepBytes + kStepScales) + kLdsPad) : 0;
    const size_t parts = SPLIT > 1 ? (size_t)(SPLIT - 1) * NT * kWave * sizeof(f32x4) : 0;
    hipLaunchKernelGGL((matmul_mxfp4_few_kernel<DT, NT, CH, SPLIT, QUANT>), grid_of_blocks(blocks),
                       dim3(kWaves * kWave), quant > parts ? quant : parts, stream, p);
    return hipGetLastError();
}

template <int DT>
hipError_t by_tokens(const FewArgs &p, int R, hipStream_t stream) {
    if (p.T <= 16) return launch<DT, 1, 8, kWaves, false>(p, R, stream);
    if (p.T <= 32) return launch<DT, 2, 4, kWaves, false>(p, R, stream);
    return launch<DT, 4, 4, kWaves, false>(p, R, stream);
}

template <int DT>
hipError_t quantizing(const FewArgs &p, int R, hipStream_t stream) {
    const int cus = compute_units();
    if (cus <= 0) return hipErrorInvalidDevice;
    if (mxfp4_split_rounds(R, p.H, p.steps, cus) != 0) return launch<DT, 1, 8, kWaves, true>(p, R, stream);
    return launch<DT, 1, 8, 1, true>(p, R, stream);
}

}  // namespace

hipError_t launch_linear_mxfp4_few(const uint16_t *a, const uint8_t *w_codes, const uint8_t *w_scales,
                                   int R, int T, int K, int Kp, int H, int dtype, uint16_t *y,
                                   hipStream_t stream) {
    FewArgs p = {};
    p.a = a;
    p.wc = w_codes;
    p.ws = w_scales;
    p.y = y;
    p.T = T;
    p.K = K;
    p.H = H;
    p.steps = Kp / kMxStepElems;
    return dtype == 0 ? quantizing<0>(p, R, stream) : quantizing<1>(p, R, stream);
}

hipError_t launch_matmul_mxfp4_few(const uint8_t *a_codes, const uint8_t *a_scales,
                                   const uint8_t *w_codes, const uint8_t *w_scales, int R, int T, int Kp,
                                   int H, int dtype, uint16_t *y, hipStream_t stream) {
    FewArgs p = {};
    p.ac = a_codes;
    p.as = a_scales;
    p.wc = w_codes;
    p.ws = w_scales;
    p.y = y;
    p.T = T;
    p.H = H;
    p.steps = Kp / kMxStepElems;
    return dtype == 0 ? by_tokens<0>(p, R, stream) : by_tokens<1>(p, R, stream);
}

}  // namespace fc
