// Backward pass of an activation from the INT8 payload of its input
// (include/fc/train.h, fc_activation_backward):
//
//   z = q * s + zero                         (binary32, not rounded to 16 bits)
//   dz = dy * mul * act'(z), dmul = dy * act(z), db = sum over tokens of dz
//
// A lane owns a vector of 8 columns and walks the rows of its workgroup's share, so
// that db needs no exchange until the share's end: the workgroup's rows meet in
// LDS, and a second launch adds the shares in a fixed order. Each operand is read
// once and each output written once: 5 bytes per element (8 with mul), bound by
// memory.
#include "fc_act.h"
#include "fc_grid.h"
#include "fc_launch_train.h"
#include "fc_rows.h"

namespace fc {
namespace {

constexpr int kShareThreads = 256;   // of a workgroup with a share of the rows
constexpr int kWholeThreads = 1024;  // of one that has all rows of its columns
constexpr int kBlocks = 2048;        // workgroups of shares that fill the device

template <int DT, int ACT, bool MUL, bool SUMS, int kThreads>
__global__ __launch_bounds__(kThreads) void activation_back_kernel(const ActBackArgs a) {
    __shared__ float lds[SUMS ? kThreads * kLaneElems : 1];
    const int thread = (int)__builtin_amdgcn_workitem_id_x();
    const int H = a.H, lanes = 1 << a.clog, rows = kThreads >> a.clog;
    const uint64_t id = grid_index();
    const uint64_t share = id / (uint32_t)a.blocks;         // of all ranks
    if (share >= (uint64_t)a.R * (uint32_t)a.parts) return;
    const uint32_t cb = (uint32_t)(id - share * (uint32_t)a.blocks);
    const uint32_t r = (uint32_t)(share / (uint32_t)a.parts), part = (uint32_t)(share - (uint64_t)r * (uint32_t)a.parts);
    const int lane = thread & (lanes - 1);
    const int e = ((int)(cb << a.clog) + lane) * kLaneElems;
    const int last = H > kLaneElems ? H - kLaneElems : 0, b = e < last ? e : last;
    const bool live = e < H;
    const int64_t first = (int64_t)part * a.chunk;
    const int64_t end = first + a.chunk < a.T ? first + a.chunk : a.T;
    float db[kLaneElems] = {};
    uint32_t g = 0;
    if constexpr (ACT != kActNone) g = group_of((uint32_t)b / kLaneElems, a.gmagic);
    if (live) {
        for (int64_t t = first + (thread >> a.clog); t < end; t += rows) {
            const uint64_t row = (uint64_t)r * (uint32_t)a.T + (uint64_t)t, at = row * (uint64_t)H;
            float dy[kLaneElems];
            widen8<DT>(load_row8(a.dy + at, b, H), dy);
            if constexpr (ACT != kActNone) {
                const uint64_t go = row * (uint64_t)a.groups + g;
                const u32x2 qz = *reinterpret_cast<const u32x2 *>(a.pz.codes + at + (uint32_t)b);
                const uint32_t wz[2] = {qz.x, qz.y};
                float z[kLaneElems], m[kLaneElems], dm[kLaneElems];
                dequant8<8>(wz, a.pz.s[go], a.pz.z[go], z);
                if constexpr (MUL) {
                    const u32x2 qm = *reinterpret_cast<const u32x2 *>(a.pm.codes + at + (uint32_t)b);
                    const uint32_t wm[2] = {qm.x, qm.y};
                    dequant8<8>(wm, a.pm.s[go], a.pm.z[go], m);
                }
#pragma unroll
                for (int k = 0; k < kLaneElems; ++k) {
                    float value, slope;
                    act_both<ACT>(z[k], value, slope);
                    dm[k] = dy[k] * value;
                    if constexpr (MUL) dy[k] *= m[k];
                    dy[k] *= slope;
                }
                *reinterpret_cast<u32x4 *>(a.dz + at + (uint32_t)b) = narrow8<DT>(dy);
                if constexpr (MUL) *reinterpret_cast<u32x4 *>(a.dmul + at + (uint32_t)b) = narrow8<DT>(dm);
            }
            if constexpr (SUMS) {
#pragma unroll
                for (int k = 0; k < kLaneElems; ++k) db[k] += dy[k];
            }
        }
    }
    if constexpr (SUMS) {
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) lds[thread * kLaneElems + k] = db[k];
        __syncthreads();
        float *out = (a.parts == 1 ? a.db + (uint64_t)r * (uint32_t)H : a.part + share * (uint64_t)H);
        const int width = lanes * kLaneElems;
        for (int c = thread; c < width; c += kThreads) {
            float s = 0.0f;
            for (int i = 0; i < rows; ++i) s += lds[i * width + c];
            const int ec = ((int)(cb << a.clog) + c / kLaneElems) * kLaneElems;
            const int col = (ec < last ? ec : last) + c % kLaneElems;
            if (col >= ec && col < H) out[col] = s;
        }
    }
}

// Rows up to which one workgroup sums all of them, 64 or more at a time, for 128
// columns: one launch and no workspace (100 rows of 3584 with db: 5.6 us against 8.5 in
// two launches).
constexpr int kWholeRows = 256;

// Lanes of a row's vectors, workgroups across a row, and shares of the rows: as many as
// fill the device, each of whole turns of the workgroup's rows.
void plan(int R, int T, int H, bool whole, int &clog, int &blocks, int &parts, int &chunk) {
    const int nv = (H + kLaneElems - 1) / kLaneElems;
    const int most = whole ? 16 : kWave;
    clog = lanes_log(nv < most ? nv : most);
    blocks = (nv + (1 << clog) - 1) >> clog;
    if (whole) {
        parts = 1;
        chunk = T;
        return;
    }
    const int rows = kShareThreads >> clog;
    const long long turns = ((long long)T + rows - 1) / rows;
    long long want = kBlocks / ((long long)R * blocks);
    want = want < 1 ? 1 : want > turns ? turns : want;
    const long long per = want > 0 ? (turns + want - 1) / want : 1;
    parts = turns > 0 ? (int)((turns + per - 1) / per) : 1;
    chunk = (int)(per * rows < T ? per * rows : T);
}

template <int DT, int ACT, bool MUL>
hipError_t launch_act(ActBackArgs a, hipStream_t stream) {
    const dim3 grid = grid_of_blocks((uint64_t)a.R * (uint64_t)a.parts * (uint64_t)a.blocks);
    if (a.db == nullptr)
        hipLaunchKernelGGL((activation_back_kernel<DT, ACT, MUL, false, kShareThreads>), grid, dim3(kShareThreads), 0, stream, a);
    else if (a.T <= kWholeRows)
        hipLaunchKernelGGL((activation_back_kernel<DT, ACT, MUL, true, kWholeThreads>), grid, dim3(kWholeThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((activation_back_kernel<DT, ACT, MUL, true, kShareThreads>), grid, dim3(kShareThreads), 0, stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.db == nullptr || a.parts == 1) return err;
    return launch_column_sum(a.part, a.R, a.parts, a.H, a.H, a.H, a.db, nullptr, stream);
}

template <int DT, bool MUL>
hipError_t by_act(const ActBackArgs &a, hipStream_t stream) {
    switch (a.act) {
    case kActRelu: return launch_act<DT, kActRelu, MUL>(a, stream);
    case kActSilu: return launch_act<DT, kActSilu, MUL>(a, stream);
    case kActGelu: return launch_act<DT, kActGelu, MUL>(a, stream);
    case kActGeluTanh: return launch_act<DT, kActGeluTanh, MUL>(a, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

int activation_parts(int R, int T, int H) {
    int clog, blocks, parts, chunk;
    plan(R, T, H, T <= kWholeRows, clog, blocks, parts, chunk);
    return parts;
}

hipError_t launch_activation_backward(const ActBackArgs &args, int dtype, hipStream_t stream) {
    ActBackArgs a = args;
    plan(a.R, a.T, a.H, a.db != nullptr && a.T <= kWholeRows, a.clog, a.blocks, a.parts, a.chunk);
    if (a.act == kActNone) {
        // dy's column sums alone
        return dtype == 0 ? launch_act<0, kActNone, false>(a, stream) : launch_act<1, kActNone, false>(a, stream);
    }
    const uint32_t d = (uint32_t)(a.group / kLaneElems);
    a.groups = a.H / a.group;
    a.gmagic = d == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + d - 1) / d);
    if (a.pm.codes != nullptr) return dtype == 0 ? by_act<0, true>(a, stream) : by_act<1, true>(a, stream);
    return dtype == 0 ? by_act<0, false>(a, stream) : by_act<1, false>(a, stream);
}

}  // namespace fc
