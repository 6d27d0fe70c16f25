// MXFP4 quantizer and dequantizer (include/fc/layer.h): HBM-bound, 2 bytes of
// activation and 17/32 of code and scale per value.
//
// A lane owns 8 consecutive values (16 bytes of activations, 4 of codes), a
// block of 32 is four neighbouring lanes: its largest magnitude is an
// unsigned maximum of the values' bits without their signs, two packed 16-bit
// halves at a time, and two DPP steps. The codes come from the hardware's
// scaled conversions, whose scale is a power of two, so the one rounding is
// the one to E2M1.
//
// Units of 8 values are numbered over the padded rows (Kp / 8 each); rows
// that need no padding are one flat run, and its 16-bit values are loaded and
// stored non-temporally: 8192 x 8192 bf16 quantized and dequantized in 51.9 us
// (6.5 TB/s) against 58.1 through the caches; 1, 2 and 4 units per lane 58.2 /
// 58.1 / 59.5. Rows of 8191, which are aligned to 2 bytes only, take 69.
#include "fc_grid.h"
#include "fc_launch.h"
#include "fc_mxfp4.h"

namespace fc {
namespace {

constexpr int kUnits = 2;   // units per lane

// Row and column of a unit: the workgroup's first unit by one 64-bit division
// of uniform values, the lane's from there.
struct Place {
    uint64_t row;
    uint32_t col;   // in values
};
__device__ __forceinline__ Place place(uint64_t first_row, uint32_t first_unit, uint32_t offset,
                                       uint32_t per_row) {
    const uint32_t u = first_unit + offset;
    const uint32_t r = u / per_row;
    return {first_row + r, (u - r * per_row) * kLaneElems};
}

template <int DT, bool FLAT>
__global__ __launch_bounds__(kBlockThreads) void quantize_mxfp4_kernel(
    const uint16_t *__restrict__ x, uint64_t units, int K, int per_row, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales) {
    const uint32_t tid = __builtin_amdgcn_workitem_id_x();
    const uint64_t base = grid_index() * (kBlockThreads * kUnits);
    uint64_t row0 = 0;
    uint32_t unit0 = 0;
    if constexpr (!FLAT) {
        row0 = base / (uint32_t)per_row;
        unit0 = (uint32_t)(base - row0 * (uint32_t)per_row);
    }
    u32x4 v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint32_t off = u * kBlockThreads + tid;
        v[u] = u32x4{0, 0, 0, 0};
        if (base + off < units) {
            if constexpr (FLAT) {
                v[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x + (base + off) * kLaneElems));
            } else {
                const Place p = place(row0, unit0, off, (uint32_t)per_row);
                v[u] = mx_load8(x + p.row * (uint64_t)K, p.col, (uint32_t)K);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint32_t off = u * kBlockThreads + tid;
        const uint32_t byte = mx_block_scale<DT>(v[u]);
        uint32_t q = mx_encode8<DT>(v[u], mx_scale(byte));
        if (byte == 255u) q = 0;
        if (base + off < units) {
            reinterpret_cast<uint32_t *>(codes)[base + off] = q;
            if ((tid & 3) == 0) scales[(base + off) / 4] = (uint8_t)byte;
        }
    }
}

template <int DT, bool FLAT>
__global__ __launch_bounds__(kBlockThreads) void dequantize_mxfp4_kernel(
    const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, uint64_t units, int K,
    int per_row, uint16_t *__restrict__ out) {
    const uint32_t tid = __builtin_amdgcn_workitem_id_x();
    const uint64_t base = grid_index() * (kBlockThreads * kUnits);
    uint64_t row0 = 0;
    uint32_t unit0 = 0;
    if constexpr (!FLAT) {
        row0 = base / (uint32_t)per_row;
        unit0 = (uint32_t)(base - row0 * (uint32_t)per_row);
    }
    uint32_t q[kUnits], byte[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint32_t off = u * kBlockThreads + tid;
        q[u] = 0;
        byte[u] = 0;
        if (base + off < units) {
            q[u] = reinterpret_cast<const uint32_t *>(codes)[base + off];
            byte[u] = scales[(base + off) / 4];
        }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint32_t off = u * kBlockThreads + tid;
        if (base + off >= units) continue;
        const float s = mx_scale(byte[u]);
        float f[kLaneElems];
        const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 0);
        const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 1);
        const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 2);
        const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 3);
        f[0] = p0.x; f[1] = p0.y; f[2] = p1.x; f[3] = p1.y;
        f[4] = p2.x; f[5] = p2.y; f[6] = p3.x; f[7] = p3.y;
        u32x4 w = narrow8<DT>(f);
        constexpr uint32_t kNan = DT == 1 ? 0x7FC07FC0u : 0x7E007E00u;
        if (byte[u] == 255u) w = u32x4{kNan, kNan, kNan, kNan};
        if constexpr (FLAT) {
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(out + (base + off) * kLaneElems));
        } else {
            const Place p = place(row0, unit0, off, (uint32_t)per_row);
            uint16_t *row = out + p.row * (uint64_t)K;
            if (p.col + kLaneElems <= (uint32_t)K) {
                *reinterpret_cast<u32x4_u16 *>(row + p.col) = w;
            } else {
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (uint32_t k = 0; k < kLaneElems; ++k)
                    if (p.col + k < (uint32_t)K) row[p.col + k] = (uint16_t)(ws[k / 2] >> (16 * (k & 1)));
            }
        }
    }
}

// Workgroups (a grid has fewer than 2^16 rows of 2^20 of them: 2^48 values).
bool grid_of(uint64_t units, dim3 *grid) {
    const uint64_t n = (units + kBlockThreads * kUnits - 1) / (kBlockThreads * kUnits);
    *grid = grid_of_blocks(n);
    return n <= uint64_t(65535) << kGridRow;
}

}  // namespace

hipError_t launch_quantize_mxfp4(const uint16_t *x, int dtype, uint64_t rows, int K, int Kp,
                                 uint8_t *codes, uint8_t *scales, hipStream_t stream) {
    const int per_row = Kp / kLaneElems;
    const uint64_t units = rows * (uint64_t)per_row;
    dim3 grid;
    if (!grid_of(units, &grid)) return hipErrorInvalidConfiguration;
#define FC_GO(DT, FLAT)                                                                              \
    hipLaunchKernelGGL((quantize_mxfp4_kernel<DT, FLAT>), grid, dim3(kBlockThreads), 0, stream, x, \
                       units, K, per_row, codes, scales)
    if (dtype == 0) {
        if (K == Kp) FC_GO(0, true);
        else FC_GO(0, false);
    } else {
        if (K == Kp) FC_GO(1, true);
        else FC_GO(1, false);
    }
#undef FC_GO
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, uint64_t rows, int K,
                                   int Kp, int dtype, uint16_t *out, hipStream_t stream) {
    const int per_row = Kp / kLaneElems;
    const uint64_t units = rows * (uint64_t)per_row;
    dim3 grid;
    if (!grid_of(units, &grid)) return hipErrorInvalidConfiguration;
#define FC_GO(DT, FLAT)                                                                            \
    hipLaunchKernelGGL((dequantize_mxfp4_kernel<DT, FLAT>), grid, dim3(kBlockThreads), 0, stream, \
                       codes, scales, units, K, per_row, out)
    if (dtype == 0) {
        if (K == Kp) FC_GO(0, true);
        else FC_GO(0, false);
    } else {
        if (K == Kp) FC_GO(1, true);
        else FC_GO(1, false);
    }
#undef FC_GO
    return hipGetLastError();
}

}  // namespace fc
