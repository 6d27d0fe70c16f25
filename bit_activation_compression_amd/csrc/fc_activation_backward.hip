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
// memory: 8192 x 7168 with mul 83 to 86 us, 5.5 TB/s; without 54, 5.5; GELU 57, with db 66, 4.5
// (5 of it the second launch); db alone 26, 4.4 (5).
#include "fc_act.h"
#include "fc_grid.h"
#include "fc_launch_train.h"
#include "fc_rows.h"

namespace fc {
namespace {

constexpr int kShareThreads = 256;   // of a workgroup with a share of the rows
constexpr int kWholeThreads = 1024;  // of one that has all rows of its columns
constexpr int kBlocks = 2048;        // workgroups of shares that fill the device
constexpr int kAhead = 2;            // rows of a lane in flight
constexpr int kFree = 16384;         // without sums (8192 x 7168, SiLU and mul, in turn: 89 us, with 2048 99)

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
    // share `part` has every parts-th turn of rows: the workgroups that run at a time
    // read neighbouring rows (8192 x 7168 with GELU and db 68 us, with shares of
    // consecutive rows 73)
    const int64_t first = (int64_t)part * rows, step = (int64_t)a.parts * rows, end = a.T;
    float db[kLaneElems] = {};
    uint32_t g = 0;
    if constexpr (ACT != kActNone) g = group_of((uint32_t)b / kLaneElems, a.gmagic);
    if (live) {
        // a row's operands, as loaded
        struct Row {
            u32x4 dy;
            u32x2 qz, qm;
            uint16_t zs, zz, ms, mz;
        };
        auto load = [&](int64_t t, Row &o) {
            const uint64_t row = (uint64_t)r * (uint32_t)a.T + (uint64_t)t, at = row * (uint64_t)H;
            if constexpr (ACT == kActNone) {
                o.dy = load_row8(a.dy + at, b, H);
            } else {
                // rows are whole vectors: groups are multiples of 8
                const uint64_t go = row * (uint64_t)a.groups + g;
                o.dy = *reinterpret_cast<const u32x4 *>(a.dy + at + (uint32_t)b);
                o.qz = *reinterpret_cast<const u32x2 *>(a.pz.codes + at + (uint32_t)b);
                o.zs = a.pz.s[go];
                o.zz = a.pz.z[go];
                if constexpr (MUL) {
                    o.qm = *reinterpret_cast<const u32x2 *>(a.pm.codes + at + (uint32_t)b);
                    o.ms = a.pm.s[go];
                    o.mz = a.pm.z[go];
                }
            }
        };
        auto finish = [&](int64_t t, const Row &o) {
            const uint64_t at = ((uint64_t)r * (uint32_t)a.T + (uint64_t)t) * (uint64_t)H;
            float dy[kLaneElems];
            widen8<DT>(o.dy, dy);
            if constexpr (ACT != kActNone) {
                const uint32_t wz[2] = {o.qz.x, o.qz.y};
                float z[kLaneElems], m[kLaneElems], dm[kLaneElems];
                dequant8<8>(wz, o.zs, o.zz, z);
                if constexpr (MUL) {
                    const uint32_t wm[2] = {o.qm.x, o.qm.y};
                    dequant8<8>(wm, o.ms, o.mz, m);
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
        };
        // kAhead rows in flight at a time
        int64_t t = first + (thread >> a.clog);
        for (; t + (kAhead - 1) * step < end; t += kAhead * step) {
            Row row[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) load(t + i * step, row[i]);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) finish(t + i * step, row[i]);
        }
        for (; t < end; t += step) {
            Row row;
            load(t, row);
            finish(t, row);
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
// columns: one launch and no workspace. Rows of 3584 with GELU and db: 100 of them 6.0 us,
// 256 10.3; 256 in shares and two launches 7.6.
constexpr int kWholeRows = 128;

// Lanes of a row's vectors, workgroups across a row, and shares of the rows' turns: as
// many as fill the device.
void plan(int R, int T, int H, bool whole, int fill, int &clog, int &blocks, int &parts) {
    const int nv = (H + kLaneElems - 1) / kLaneElems;
    const int most = whole ? 16 : kWave;
    clog = lanes_log(nv < most ? nv : most);
    blocks = (nv + (1 << clog) - 1) >> clog;
    const int rows = kShareThreads >> clog;
    const long long turns = ((long long)T + rows - 1) / rows;
    long long want = fill / ((long long)R * blocks);
    want = want < 1 ? 1 : want > turns ? turns : want;
    parts = whole ? 1 : (int)want;
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
    int clog, blocks, parts;
    plan(R, T, H, T <= kWholeRows, kBlocks, clog, blocks, parts);
    return parts;
}

hipError_t launch_activation_backward(const ActBackArgs &args, int dtype, hipStream_t stream) {
    ActBackArgs a = args;
    plan(a.R, a.T, a.H, a.db != nullptr && a.T <= kWholeRows, a.db != nullptr ? kBlocks : kFree, a.clog, a.blocks, a.parts);
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
