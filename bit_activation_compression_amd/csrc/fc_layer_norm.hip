// Layer and RMS norm (include/fc/train.h, fc_layer_norm):
//
//   m = mean(x) (0 for RMS), r = 1 / sqrt(mean((x - m)^2) + eps)
//   y = (x - m) * r * w + b
//
// and, on the way, the INT8 payload of x (what the stage-1 quantizer writes) for
// the backward pass. The row stays in registers between its uses: x is read once
// and y written once, 4 bytes per element and 1 + 4 / group for the payload, so
// the kernel is bound by memory. The variance is that of x - m (two sums over the
// row), which keeps its digits where the mean is large.
//
// Measured (rotating buffers): 8192 x 8192 bf16 49 us, 5.5 TB/s, with the payload 65,
// 5.2; 8192 x 4096 fp16 26, 5.1, with the payload 34.5, 4.9 (its vector instructions take about
// 70% of the issue slots there); 2048 x 16384 bf16 29, with the payload 36; one row of 8192 2.8.
//
// A row of more than 512 elements has a workgroup to itself, thread i holding the
// vectors of 8 elements i, i + threads, ... Shorter rows lie side by side in a wave,
// 2^llog lanes each, and meet no barrier.
#include "fc_grid.h"
#include "fc_launch_train.h"
#include "fc_rows.h"

namespace fc {
namespace {

constexpr int kRowThreads = 1024;   // most of a workgroup
constexpr int kTeamThreads = 256;   // of a workgroup of short rows

// min and max over 2^llog lanes (a group of the payload)
__device__ __forceinline__ void lanes_minmax_of(float &mn, float &mx, int llog) {
    switch (llog) {
    case 0: lanes_minmax<1>(mn, mx); break;
    case 1: lanes_minmax<2>(mn, mx); break;
    case 2: lanes_minmax<4>(mn, mx); break;
    case 3: lanes_minmax<8>(mn, mx); break;
    case 4: lanes_minmax<16>(mn, mx); break;
    case 5: lanes_minmax<32>(mn, mx); break;
    default: lanes_minmax<64>(mn, mx); break;
    }
}

// The INT8 codes of the vector from element e of a row, and its groups' scales and
// zeros. Groups are powers of two of at most 512: they lie in the lanes of a wave.
__device__ __forceinline__ void save8(const LayerNormArgs &a, uint64_t row, int e, const float (&x)[kLaneElems]) {
    const int glog = 31 - __builtin_clz((uint32_t)a.group);
    float mn, mx;
    minmax8(x, mn, mx);
    lanes_minmax_of(mn, mx, glog - 3);
    const GroupParams p = group_params<8>(mn, mx);
    uint32_t q[2];
    encode8<8>(x, p, q);
    if (e >= a.H) return;
    *reinterpret_cast<u32x2 *>(a.codes + row * (uint64_t)a.H + (uint32_t)e) = u32x2{q[0], q[1]};
    if ((e & (a.group - 1)) == 0) {
        const uint64_t g = row * (uint64_t)(a.H >> glog) + (uint32_t)(e >> glog);
        a.s[g] = p.s16;
        a.z[g] = p.z16;
    }
}

template <int DT, int V, bool TEAM>
__global__ __launch_bounds__(TEAM ? kTeamThreads : kRowThreads) void layer_norm_kernel(const LayerNormArgs a) {
    __shared__ float part[2][kRowThreads / kWave];
    const int thread = (int)__builtin_amdgcn_workitem_id_x();
    const int NT = TEAM ? 1 << a.llog : a.waves * kWave;   // of a row
    const int tid = TEAM ? thread & (NT - 1) : thread;
    uint64_t row = grid_index();
    if constexpr (TEAM) row = (row << (8 - a.llog)) + (uint32_t)(thread >> a.llog);   // 2^8 threads
    if (row >= (uint64_t)a.T) return;
    const int H = a.H;
    // As in the block norms: the vector's elements are those from elem(v), its
    // load takes 8 whole ones from begin(v), and own zeroes what is not its own.
    auto elem = [&](int v) { return (tid + v * NT) * kLaneElems; };
    const int last = H > kLaneElems ? H - kLaneElems : 0;
    auto begin = [&](int v) { return elem(v) < last ? elem(v) : last; };
    auto own = [&](int v, float (&x)[kLaneElems]) {
        if (elem(v) + kLaneElems <= H) return;
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k)
            if (begin(v) + k < elem(v) || begin(v) + k >= H) x[k] = 0.0f;
    };
    auto row_total = [&](float s, int i) {
        if constexpr (TEAM) return lanes_sum(s, a.llog);
        else return block_sum(s, part[i], (uint32_t)a.waves);
    };
    // w and b are in flight with x
    const uint16_t *xrow = a.x + row * (uint64_t)H;
    u32x4 xr[V], wr[V], br[V];
#pragma unroll
    for (int v = 0; v < V; ++v) xr[v] = load_row8(xrow, begin(v), H);
    if (a.w != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) wr[v] = load_row8(a.w, begin(v), H);
    }
    if (a.b != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) br[v] = load_row8(a.b, begin(v), H);
    }
    float x[V][kLaneElems];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        widen8<DT>(xr[v], x[v]);
        own(v, x[v]);
    }

    if (a.codes != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) save8(a, row, elem(v), x[v]);
    }

    if (!a.rms) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) s += x[v][k];
        const float mean = row_total(s, 0) * a.inv_h;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) x[v][k] -= mean;
            own(v, x[v]);
        }
        if (a.mean != nullptr && tid == 0) a.mean[row] = mean;
    }
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) ss = __builtin_fmaf(x[v][k], x[v][k], ss);
    const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(row_total(ss, 1), a.inv_h, a.eps));
    if (a.rstd != nullptr && tid == 0) a.rstd[row] = rstd;

    uint16_t *yrow = a.y + row * (uint64_t)H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float y[kLaneElems], w[kLaneElems], b[kLaneElems];
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) {
            y[k] = x[v][k] * rstd;
            w[k] = 1.0f;
            b[k] = 0.0f;
        }
        if (a.w != nullptr) {
            widen8<DT>(wr[v], w);
        }
        if (a.b != nullptr) {
            widen8<DT>(br[v], b);
        }
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) y[k] = __builtin_fmaf(y[k], w[k], b[k]);
        store_row8<DT>(yrow, elem(v), begin(v), H, y);
    }
}

// Rows of more than 4 vectors to a thread are read three times, from the L2 after the
// first.
template <int DT>
__global__ __launch_bounds__(kRowThreads) void layer_norm_long_kernel(const LayerNormArgs a) {
    __shared__ float part[2][kRowThreads / kWave];
    const int thread = (int)__builtin_amdgcn_workitem_id_x();
    const uint64_t row = grid_index();
    if (row >= (uint64_t)a.T) return;
    const int H = a.H, last = H - kLaneElems;
    const uint16_t *xrow = a.x + row * (uint64_t)H;
    // x - mean of the vector from e, zeros where it is not the vector's own
    auto vector = [&](int e, float mean, float (&x)[kLaneElems]) {
        const int b = e < last ? e : last;
        widen8<DT>(load_row8(xrow, b, H), x);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) x[k] = b + k < e ? 0.0f : x[k] - mean;
    };
    constexpr int kStep = kRowThreads * kLaneElems;
    float mean = 0.0f, s = 0.0f;
    if (!a.rms || a.codes != nullptr) {
        // whole turns: the lanes of a group exchange
        for (int e = thread * kLaneElems; e - thread * kLaneElems < H; e += kStep) {
            float x[kLaneElems] = {};
            if (e < H) vector(e, 0.0f, x);
            if (a.codes != nullptr) save8(a, row, e, x);
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) s += x[k];
        }
    }
    if (!a.rms) {
        mean = block_sum(s, part[0], kRowThreads / kWave) * a.inv_h;
        if (a.mean != nullptr && thread == 0) a.mean[row] = mean;
    }
    float ss = 0.0f;
    for (int e = thread * kLaneElems; e < H; e += kStep) {
        float x[kLaneElems];
        vector(e, mean, x);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) ss = __builtin_fmaf(x[k], x[k], ss);
    }
    const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(block_sum(ss, part[1], kRowThreads / kWave), a.inv_h, a.eps));
    if (a.rstd != nullptr && thread == 0) a.rstd[row] = rstd;
    for (int e = thread * kLaneElems; e < H; e += kStep) {
        const int b = e < last ? e : last;
        float x[kLaneElems], w[kLaneElems], bias[kLaneElems];
        vector(e, mean, x);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) {
            x[k] *= rstd;
            w[k] = 1.0f;
            bias[k] = 0.0f;
        }
        if (a.w != nullptr) widen8<DT>(load_row8(a.w, b, H), w);
        if (a.b != nullptr) widen8<DT>(load_row8(a.b, b, H), bias);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) x[k] = __builtin_fmaf(x[k], w[k], bias[k]);
        store_row8<DT>(a.y + row * (uint64_t)H, e, b, H, x);
    }
}

template <int DT, int V>
hipError_t launch_rows(LayerNormArgs a, int nv, hipStream_t stream) {
    a.waves = (nv + V * kWave - 1) / (V * kWave);
    hipLaunchKernelGGL((layer_norm_kernel<DT, V, false>), grid_of_blocks((uint64_t)a.T),
                       dim3((unsigned)(a.waves * kWave)), 0, stream, a);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_any(LayerNormArgs a, hipStream_t stream) {
    const int nv = (a.H + kLaneElems - 1) / kLaneElems;
    if (nv <= kWave) {
        a.llog = lanes_log(nv);
        const uint64_t rows = (uint64_t)kTeamThreads >> a.llog;
        hipLaunchKernelGGL((layer_norm_kernel<DT, 1, true>), grid_of_blocks(((uint64_t)a.T + rows - 1) / rows),
                           dim3(kTeamThreads), 0, stream, a);
        return hipGetLastError();
    }
    // two vectors per thread once the device is full of rows, as for the block norms
    const bool few = (uint64_t)a.T * (uint64_t)a.H < (uint64_t(1) << 23);
    if (nv <= kRowThreads && few) return launch_rows<DT, 1>(a, nv, stream);
    if (nv <= 2 * kRowThreads) return launch_rows<DT, 2>(a, nv, stream);
    if (nv <= 4 * kRowThreads) return launch_rows<DT, 4>(a, nv, stream);
    hipLaunchKernelGGL((layer_norm_long_kernel<DT>), grid_of_blocks((uint64_t)a.T), dim3(kRowThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs &a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_any<0>(a, stream) : launch_any<1>(a, stream);
}

}  // namespace fc
