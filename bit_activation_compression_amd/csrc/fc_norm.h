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
// A row is NT threads (whole waves, as many as it needs) x V vectors of 8
// elements (thread i holds vectors i, i + NT, ...), so a wave's load covers
// 1 KiB of consecutive elements. Rows need no alignment beyond an element's:
// vectors are loaded and stored at 2-byte alignment (one global_load_dwordx4
// all the same), and the last vector of a row that is no whole number of them
// loads the row's last 8 elements.
//
// Measured: 8192 rows of 4096 (fp16, post-norm) 48 us, 5.6 TB/s (on one set of
// buffers, part of which the Infinity Cache then holds, 39.4); 8192 rows of 8192 from
// an INT4 payload 76 us, 5.7 TB/s; 1777 rows of 5003 with a gate per token 18.3 us,
// 4.9 TB/s. One row is a launch and two reductions: 3.7 us. Non-temporal loads
// were slower, and so was shifting the vectors of a misaligned row to whole 16-byte
// ones (28 against 18.3 us). Non-temporal stores change nothing: 8192 x 8192 from an
// INT4 payload 75.8 against 76.0, 8192 x 8192 94.4 against 94.4, 65536 x 1024 92.7
// against 92.5, 4096 x 32768 213.8 against 212.3.
#pragma once

#include "fc_device.h"
#include "fc_grid.h"
#include "fc_launch.h"

namespace fc {
namespace {

constexpr int kNormThreads = 1024;   // most of a workgroup
constexpr uint64_t kManyElems = uint64_t(1) << 23;

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

// SRC: 0 a 16-bit block output, 4 or 8 the payload of codes of that width.
// GEN (payload only): groups that are not a multiple of 8, which may end
// inside a vector (at a pair: groups are even); otherwise a vector lies in one
// group. A group's number is that of the vector (pair) over the vectors
// (pairs) of a group, both at most 2^15.
template <int DT, int SRC, bool GEN, int V>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(const NormArgs a) {
    __shared__ float part[2][kNormThreads / kWave];
    const int NT = a.waves * kWave;
    const int tid = (int)__builtin_amdgcn_workitem_id_x();
    const uint64_t row = grid_index();
    if (row >= (uint64_t)a.T) return;
    const int H = a.H;
    // Vector v of the thread: its elements are those from elem(v), if any. All
    // loads take 8 whole ones, from begin(v): the row's last 8 where fewer (or
    // none) are left, and `own` zeroes what is not the thread's own.
    auto elem = [&](int v) { return (tid + v * NT) * kLaneElems; };
    const int last = H > kLaneElems ? H - kLaneElems : 0;
    auto begin = [&](int v) { return elem(v) < last ? elem(v) : last; };
    auto own = [&](int v, float (&x)[kLaneElems]) {
        if (elem(v) + kLaneElems <= H) return;
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k)
            if (begin(v) + k < elem(v) || begin(v) + k >= H) x[k] = 0.0f;
    };
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
    auto to_x = [&](int v) {
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
        own(v, x[v]);
    };
    if constexpr (SRC != 0) {
        const uint8_t *crow = a.codes + row * (uint64_t)H * SRC / 8;
        const uint64_t g0 = row * (uint64_t)a.groups;
        const uint16_t *srow = a.s + g0, *zrow = a.z + g0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int b = begin(v);
            if (!GEN || H >= kLaneElems) {
                if constexpr (SRC == 4) {
                    cw[v][0] = *reinterpret_cast<const u32_a1 *>(crow + b / 2);
                } else {
                    const u32x2 w = *reinterpret_cast<const u32x2_a1 *>(crow + b);
                    cw[v][0] = w.x;
                    cw[v][1] = w.y;
                }
            } else {
                for (uint32_t &w : cw[v]) w = 0;
#pragma unroll
                for (int k = 0; k < kLaneElems * SRC / 8; ++k)
                    if (k < H * SRC / 8) cw[v][k / 4] |= (uint32_t)crow[k] << (8 * (k & 3));
            }
            if constexpr (GEN) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const uint32_t pair = (uint32_t)(b / 2 + p);
                    const uint32_t g = group_of(pair < (uint32_t)H / 2 ? pair : 0u, a.gmagic);
                    sz[v][p] = (uint32_t)srow[g] | (uint32_t)zrow[g] << 16;
                }
            } else {
                const uint32_t g = group_of((uint32_t)b / kLaneElems, a.gmagic);
                sz[v][0] = (uint32_t)srow[g] | (uint32_t)zrow[g] << 16;
            }
            if constexpr (!kEarly) {
                to_x(v);   // one vector's codes and scales at a time
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } else {
        const uint16_t *xrow = a.x + row * (uint64_t)H;
#pragma unroll
        for (int v = 0; v < V; ++v) xr[v] = load_row8(xrow, begin(v), H);
    }
    if constexpr (kEarly) {
#pragma unroll
        for (int v = 0; v < V; ++v) rr[v] = load_row8(res_row, begin(v), H);
        if (a.w_post != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) wpost[v] = load_row8(a.w_post, begin(v), H);
        }
        if (gate_row != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) gr[v] = load_row8(gate_row, begin(v), H);
        }
        if (a.w_pre != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) wpre[v] = load_row8(a.w_pre, begin(v), H);
        }
    }
    // operand vector v, loaded by now or here
    auto operand = [&](const u32x4 (&early)[V], const uint16_t *row_, int v) {
        if constexpr (kEarly) return early[v];
        else return load_row8(row_, begin(v), H);
    };

    if constexpr (SRC == 0 || kEarly) {
#pragma unroll
        for (int v = 0; v < V; ++v) to_x(v);
    }

    if (a.w_post != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) ss = __builtin_fmaf(x[v][k], x[v][k], ss);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(block_sum(ss, part[0], (uint32_t)a.waves), a.inv_h, a.eps));
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
        }
        own(v, x[v]);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) ss = __builtin_fmaf(x[v][k], x[v][k], ss);
        store_row8<DT>(hrow, elem(v), begin(v), H, x[v]);
    }
    if (a.w_pre == nullptr) return;
    const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(block_sum(ss, part[1], (uint32_t)a.waves), a.inv_h, a.eps));
    uint16_t *yrow = a.y + row * (uint64_t)H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[kLaneElems];
        widen8<DT>(operand(wpre, a.w_pre, v), w);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) w[k] *= x[v][k] * rstd;
        store_row8<DT>(yrow, elem(v), begin(v), H, w);
    }
}

template <int DT, int SRC, bool GEN, int V>
hipError_t launch_norm_rows(NormArgs a, int nv, hipStream_t stream) {
    a.waves = (nv + V * kWave - 1) / (V * kWave);
    hipLaunchKernelGGL((norm_kernel<DT, SRC, GEN, V>), grid_of_blocks((uint64_t)a.T),
                       dim3((unsigned)(a.waves * kWave)), 0, stream, a);
    return hipGetLastError();
}

template <int DT, int SRC, bool GEN>
hipError_t launch_norm_any(NormArgs a, hipStream_t stream) {
    const int nv = (a.H + kLaneElems - 1) / kLaneElems;   // vectors of a row
    // Two vectors per thread once the device is full of rows, us with one / two (bf16,
    // in a graph on buffers that the caches do not hold): H = 8192, 512 / 1024 / 2048 /
    // 8192 rows 9.2 / 17.0 / 29.4 / 98.0 against 9.4 / 15.7 / 27.0 / 95.2; H = 4096, 512 /
    // 1024 / 8192 rows 6.0 / 9.1 / 48.2 against 6.1 / 9.4 / 48.4. Rows of at most a wave's
    // 64 vectors would leave half of it idle with two (30000 rows of 256: 23.6 against
    // 13.2 on one set of buffers).
    const bool few = nv <= kWave || (uint64_t)a.T * (uint64_t)a.H < kManyElems;
    if (nv <= kNormThreads && few) return launch_norm_rows<DT, SRC, GEN, 1>(a, nv, stream);
    if (nv <= 2 * kNormThreads) return launch_norm_rows<DT, SRC, GEN, 2>(a, nv, stream);
    if (nv <= 4 * kNormThreads) return launch_norm_rows<DT, SRC, GEN, 4>(a, nv, stream);
    return launch_norm_rows<DT, SRC, GEN, 8>(a, nv, stream);
}

}  // namespace
}  // namespace fc
