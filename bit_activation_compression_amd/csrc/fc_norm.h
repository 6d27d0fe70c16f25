// Block norms: the norm after a block, the gated and scaled residual update
// and the norm before the next block, one row (token) per workgroup.
//
//   n = w_post * x * rsqrt(mean(x^2) + eps)     (x itself without a post-norm)
//   h = res_scale * residual + out_scale * gate * n
//   y = w_pre * h * rsqrt(mean(h^2) + eps)
//
// The row stays in registers between its three uses, so each operand is read
// once and each output written once: HBM-bound, 8 bytes per element from a
// 16-bit block output, 6.5 from an INT4 payload. Everything between the loads
// and the two final roundings is binary32.
//
// A row is NT threads x V vectors of 8 elements (thread i holds vectors i, i +
// NT, ...), so a wave's load covers 1 KiB of consecutive elements. Rows need
// no alignment beyond an element's: the vectors are loaded and stored at
// 2-byte alignment (one global_load_dwordx4 all the same), and only a row's
// last vector, when H is not a multiple of 8, goes element by element.
#pragma once

#include "fc_device.h"
#include "fc_launch.h"

namespace fc {
namespace {

// vectors at the alignment of their elements
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

// Sum over the wave, the same in every lane: xor butterflies inside a row of
// 16 lanes (every lane adds the same pairs), then the four rows' sums in a
// fixed order.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xB1>(v);    // lane ^ 1
    v += dpp<0x4E>(v);    // lane ^ 2
    v += dpp<0x141>(v);   // 7 - i inside 8 lanes
    v += dpp<0x140>(v);   // 15 - i inside 16 lanes
    const int b = __builtin_bit_cast(int, v);
    const float a0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
    const float a1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
    const float a2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
    const float a3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
    return (a0 + a1) + (a2 + a3);
}

// Sum over the workgroup, the same bits in every thread. `part` is this
// reduction's own LDS (one float per wave): no barrier is needed after it.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float *part) {
    constexpr int NW = NT / kWave;
    v = wave_sum(v);
    if constexpr (NW > 1) {
        const uint32_t tid = __builtin_amdgcn_workitem_id_x();
        if ((tid & (kWave - 1)) == 0) part[tid / kWave] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) v += part[i];
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

// 8 elements from e of a row of H; zeros past its end.
__device__ __forceinline__ u32x4 load_row8(const uint16_t *row, int e, int H) {
    if (e + kLaneElems <= H) return *reinterpret_cast<const u32x4_a2 *>(row + e);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k)
        if (e + k < H) w[k / 2] |= (uint32_t)row[e + k] << (16 * (k & 1));
    return u32x4{w[0], w[1], w[2], w[3]};
}

template <int DT>
__device__ __forceinline__ void store_row8(uint16_t *row, int e, int H, const float (&v)[kLaneElems]) {
    if (e + kLaneElems <= H) {
        *reinterpret_cast<u32x4_a2 *>(row + e) = narrow8<DT>(v);
        return;
    }
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k)
        if (e + k < H) row[e + k] = narrow1<DT>(v[k]);
}

// n / d by the reciprocal ceil(2^32 / d), exact while n * d < 2^32; 0 stands
// for d = 1, whose reciprocal does not fit.
__device__ __forceinline__ uint32_t group_of(uint32_t n, uint32_t magic) {
    return magic ? __umulhi(n, magic) : n;
}

// SRC: 0 a 16-bit block output, 4 or 8 the payload of codes of that width.
// GEN (payload only): groups that are not a multiple of 8, which may end
// inside a vector (at a pair: groups are even); otherwise a vector lies in one
// group. A group's number is that of the vector (pair) over the vectors
// (pairs) of a group, both at most 2^15.
template <int DT, int SRC, bool GEN, int NT, int V>
__global__ __launch_bounds__(NT) void norm_kernel(const NormArgs a) {
    __shared__ float part[2][NT / kWave];
    const int tid = (int)__builtin_amdgcn_workitem_id_x();
    const uint64_t row = __builtin_amdgcn_workgroup_id_x();
    const int H = a.H;
    const uint16_t *res_row = a.residual + row * (uint64_t)H;

    // every operand of the row in flight before the first use; rows of more
    // than 32768 elements would not fit the registers that way, and load all
    // but x where they use it
    constexpr bool kEarly = V <= 4;
    float x[V][kLaneElems];
    u32x4 xr[V], rr[V], gr[V], wpost[V], wpre[V];
    uint32_t cw[V][SRC == 8 ? 2 : 1];
    uint32_t sz[V][GEN ? 4 : 1];   // scale in the low, zero in the high half
    const uint16_t *gate_row = nullptr;
    if (a.gate != nullptr)
        gate_row = a.gate + (uint64_t)((uint32_t)row / (uint32_t)a.gate_tokens) * (uint64_t)H;
    if constexpr (SRC != 0) {
        const uint8_t *crow = a.codes + row * (uint64_t)H * SRC / 8;
        const uint64_t g0 = row * (uint64_t)a.groups;
        const uint16_t *srow = a.s + g0, *zrow = a.z + g0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = tid + v * NT, e = i * kLaneElems;
#pragma unroll
            for (uint32_t &w : cw[v]) w = 0;
#pragma unroll
            for (uint32_t &w : sz[v]) w = 0;
            if (e + kLaneElems <= H) {
                if constexpr (SRC == 4) {
                    cw[v][0] = *reinterpret_cast<const u32_a1 *>(crow + e / 2);
                } else {
                    const u32x2 w = *reinterpret_cast<const u32x2_a1 *>(crow + e);
                    cw[v][0] = w.x;
                    cw[v][1] = w.y;
                }
            } else if constexpr (GEN) {
                // the row's last vector: whole pairs (H is even with a payload;
                // with groups of whole vectors it is a multiple of 8)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    if (e + 2 * p < H) {
                        if constexpr (SRC == 4) {
                            cw[v][0] |= (uint32_t)crow[e / 2 + p] << (8 * p);
                        } else {
                            cw[v][p / 2] |= ((uint32_t)crow[e + 2 * p] | (uint32_t)crow[e + 2 * p + 1] << 8)
                                            << (16 * (p & 1));
                        }
                    }
                }
            }
            if constexpr (GEN) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    if (e + 2 * p < H) {
                        const uint32_t g = group_of((uint32_t)(i * 4 + p), a.gmagic);
                        sz[v][p] = (uint32_t)srow[g] | (uint32_t)zrow[g] << 16;
                    }
                }
            } else if (e < H) {
                const uint32_t g = group_of((uint32_t)i, a.gmagic);
                sz[v][0] = (uint32_t)srow[g] | (uint32_t)zrow[g] << 16;
            }
        }
    } else {
        const uint16_t *xrow = a.x + row * (uint64_t)H;
#pragma unroll
        for (int v = 0; v < V; ++v) xr[v] = load_row8(xrow, (tid + v * NT) * kLaneElems, H);
    }
    auto elem = [&](int v) { return (tid + v * NT) * kLaneElems; };
    if constexpr (kEarly) {
#pragma unroll
        for (int v = 0; v < V; ++v) rr[v] = load_row8(res_row, elem(v), H);
        if (a.w_post != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) wpost[v] = load_row8(a.w_post, elem(v), H);
        }
        if (gate_row != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) gr[v] = load_row8(gate_row, elem(v), H);
        }
        if (a.w_pre != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) wpre[v] = load_row8(a.w_pre, elem(v), H);
        }
    }
    // operand vector v, loaded by now or here
    auto operand = [&](const u32x4 (&early)[V], const uint16_t *row_, int v) {
        if constexpr (kEarly) return early[v];
        else return load_row8(row_, elem(v), H);
    };

    // x; elements past the row's end are 0 (codes and scales of 0)
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if constexpr (SRC == 0) {
            widen8<DT>(xr[v], x[v]);
        } else {
            decode8<SRC>(cw[v], x[v]);
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) {
                const uint32_t m = sz[v][GEN ? k / 2 : 0];
                x[v][k] = __builtin_fmaf(x[v][k], half_bits_to_float((uint16_t)m),
                                         half_bits_to_float((uint16_t)(m >> 16)));
            }
        }
    }

    if (a.w_post != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) ss = __builtin_fmaf(x[v][k], x[v][k], ss);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(block_sum<NT>(ss, part[0]), a.inv_h, a.eps));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float w[kLaneElems];
            widen8<DT>(operand(wpost, a.w_post, v), w);
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) x[v][k] = x[v][k] * rstd * w[k];
        }
    }
    if (gate_row != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float g[kLaneElems];
            widen8<DT>(operand(gr, gate_row, v), g);
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) x[v][k] *= g[k];
        }
    }
    // h, in x's place
    uint16_t *hrow = a.h + row * (uint64_t)H;
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float r[kLaneElems];
        widen8<DT>(operand(rr, res_row, v), r);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) {
            x[v][k] = __builtin_fmaf(a.res_scale, r[k], a.out_scale * x[v][k]);
            ss = __builtin_fmaf(x[v][k], x[v][k], ss);
        }
        store_row8<DT>(hrow, elem(v), H, x[v]);
    }
    if (a.w_pre == nullptr) return;
    const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(block_sum<NT>(ss, part[1]), a.inv_h, a.eps));
    uint16_t *yrow = a.y + row * (uint64_t)H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[kLaneElems];
        widen8<DT>(operand(wpre, a.w_pre, v), w);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) w[k] *= x[v][k] * rstd;
        store_row8<DT>(yrow, elem(v), H, w);
    }
}

template <int DT, int SRC, bool GEN, int NT, int V>
hipError_t launch_norm_rows(const NormArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((norm_kernel<DT, SRC, GEN, NT, V>), dim3((unsigned)a.T), dim3(NT), 0, stream, a);
    return hipGetLastError();
}

template <int DT, int SRC, bool GEN>
hipError_t launch_norm_any(const NormArgs &a, hipStream_t stream) {
    const int nv = (a.H + kLaneElems - 1) / kLaneElems;   // vectors of a row
    if (nv <= 64) return launch_norm_rows<DT, SRC, GEN, 64, 1>(a, stream);
    if (nv <= 256) return launch_norm_rows<DT, SRC, GEN, 256, 1>(a, stream);
    if (nv <= 1024) return launch_norm_rows<DT, SRC, GEN, 1024, 1>(a, stream);
    if (nv <= 4096) return launch_norm_rows<DT, SRC, GEN, 1024, 4>(a, stream);
    return launch_norm_rows<DT, SRC, GEN, 1024, 8>(a, stream);
}

}  // namespace
}  // namespace fc
