// Backward pass of the layer and RMS norm (include/fc/train.h,
// fc_layer_norm_backward), from the saved 16-bit x or from its INT8 payload:
//
//   n = (x - mean) * rstd, g = dy * w
//   dx = rstd * (g - mean_H(g) - n * mean_H(g * n)) + dres     (no mean_H(g) for RMS)
//   dw = sum over rows of dy * n,  db = sum over rows of dy
//
// A workgroup walks rows blockIdx, blockIdx + grid, ..., a vector of 8 elements to a
// thread (short rows lie side by side in a wave): the row stays in registers, as
// loaded, between its two uses, the next row's operands are in flight meanwhile, and
// each thread keeps its columns' sums of dw and db, which a second launch adds up over
// the workgroups in a fixed order. dy and x are read once and dx written once, 6 bytes
// per element (5 from a payload): bound by memory. Rows of more than 8192 elements are
// read twice, the second time mostly from the L2, and leave dw and db to a kernel that
// reads dy and x by columns.
#include "fc_grid.h"
#include "fc_launch_train.h"
#include "fc_rows.h"

namespace fc {
namespace {

constexpr int kRowThreads = 1024;       // most of a workgroup
constexpr int kTeamThreads = 256;       // of a workgroup of short rows
constexpr int kHeldElems = kRowThreads * kLaneElems;   // longest row that is held in registers
constexpr int kParts = 512;             // most workgroups whose sums are added up
constexpr int kColWaves = 4;            // of a column kernel's workgroup

// One vector of a row's operands, as loaded.
template <int SRC>
struct Loaded {
    u32x4 dy;
    u32x4 x;         // 16-bit x
    u32x2 q;         // or codes
    uint32_t sz;     // with scale (low half) and zero
};

template <int SRC>
__device__ __forceinline__ void load_vector(const LayerNormBackArgs &a, uint64_t row, int b, Loaded<SRC> &o) {
    const uint64_t at = row * (uint64_t)a.H;
    o.dy = load_row8(a.dy + at, b, a.H);
    if constexpr (SRC == 0) {
        o.x = load_row8(a.x + at, b, a.H);
    } else {
        // rows are whole vectors here: groups are multiples of 8
        o.q = *reinterpret_cast<const u32x2 *>(a.px.codes + at + (uint32_t)b);
        const uint64_t g = row * (uint64_t)a.groups + group_of((uint32_t)b / kLaneElems, a.gmagic);
        o.sz = (uint32_t)a.px.s[g] | (uint32_t)a.px.z[g] << 16;
    }
}

// n of the vector
template <int DT, int SRC>
__device__ __forceinline__ void normed(const Loaded<SRC> &o, float mean, float rstd, float (&n)[kLaneElems]) {
    if constexpr (SRC == 0) {
        widen8<DT>(o.x, n);
    } else {
        const uint32_t q[2] = {o.q.x, o.q.y};
        dequant8<8>(q, (uint16_t)o.sz, (uint16_t)(o.sz >> 16), n);
    }
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k) n[k] = (n[k] - mean) * rstd;
}

// g and n of a vector, and its dy, where `own` zeroes what is not the vector's
template <int DT, int SRC, class Own>
__device__ __forceinline__ void terms(const Loaded<SRC> &o, const u32x4 &wr, bool has_w, float mean, float rstd, Own &&own,
                                      float (&d)[kLaneElems], float (&g)[kLaneElems], float (&n)[kLaneElems]) {
    normed<DT, SRC>(o, mean, rstd, n);
    widen8<DT>(o.dy, d);
    own(d);
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k) g[k] = d[k];
    if (has_w) {
        float w[kLaneElems];
        widen8<DT>(wr, w);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) g[k] *= w[k];
    }
}

// Both sums of a row over the workgroup through one barrier. The two turns' places
// alternate: the next row's sums cannot reach a place that is still read.
__device__ __forceinline__ void row_sums(float &sg, float &sn, float *p, uint32_t thread, uint32_t nw) {
    sg = wave_sum(sg);
    sn = wave_sum(sn);
    const uint32_t i = thread & 15u;
    if ((thread & (kWave - 1)) == 0) {
        p[2 * (thread / kWave)] = sg;
        p[2 * (thread / kWave) + 1] = sn;
    }
    __syncthreads();
    sg = row_sum(i < nw ? p[2 * i] : 0.0f);
    sn = row_sum(i < nw ? p[2 * i + 1] : 0.0f);
}

template <int DT>
__device__ __forceinline__ void finish_row(const float (&g)[kLaneElems], const float (&n)[kLaneElems], float c1, float c2,
                                           float rstd, const u32x4 &res, bool has_res, uint16_t *drow, int e, int b, int H) {
    float d[kLaneElems];
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k) d[k] = (__builtin_fmaf(-n[k], c2, g[k]) - c1) * rstd;
    if (has_res) {
        float r[kLaneElems];
        widen8<DT>(res, r);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) d[k] += r[k];
    }
    store_row8<DT>(drow, e, b, H, d);
}

template <int DT, int SRC, bool TEAM, bool SUMS>
__global__ __launch_bounds__(TEAM ? kTeamThreads : kRowThreads) void layer_norm_back_kernel(const LayerNormBackArgs a) {
    constexpr int kPart = TEAM ? kTeamThreads * kLaneElems * 2 : 2 * 2 * (kRowThreads / kWave);
    __shared__ float lds[kPart];
    const int thread = (int)__builtin_amdgcn_workitem_id_x();
    const int NT = TEAM ? 1 << a.llog : a.waves * kWave;
    const int tid = TEAM ? thread & (NT - 1) : thread;
    const int H = a.H;
    // the vector's elements are those from e; its load takes 8 whole ones from b
    const int e = tid * kLaneElems, last = H > kLaneElems ? H - kLaneElems : 0, b = e < last ? e : last;
    auto own = [&](float (&x)[kLaneElems]) {
        if (e + kLaneElems <= H) return;
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k)
            if (b + k < e || b + k >= H) x[k] = 0.0f;
    };
    const uint64_t block = __builtin_amdgcn_workgroup_id_x(), grid = (uint32_t)a.grid;
    const uint64_t step = TEAM ? grid << (8 - a.llog) : grid;
    uint64_t row = TEAM ? (block << (8 - a.llog)) + (uint32_t)(thread >> a.llog) : block;
    const bool has_w = a.w != nullptr, has_res = a.dres != nullptr;
    u32x4 wr = {};
    if (has_w) wr = load_row8(a.w, b, H);
    float dw[kLaneElems] = {}, db[kLaneElems] = {};
    Loaded<SRC> cur, nxt;
    u32x4 res = {}, nres = {};
    float mean = 0.0f, rstd = 0.0f, nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](uint64_t r, Loaded<SRC> &o, u32x4 &d, float &m, float &s) {
        load_vector<SRC>(a, r, b, o);
        if (a.mean != nullptr) m = a.mean[r];
        s = a.rstd[r];
        if (has_res) d = load_row8(a.dres + r * (uint64_t)H, b, H);
    };
    if (row < (uint64_t)a.T) fetch(row, cur, res, mean, rstd);
    for (int turn = 0; row < (uint64_t)a.T; row += step, turn ^= 1) {
        if (row + step < (uint64_t)a.T) fetch(row + step, nxt, nres, nmean, nrstd);
        float d[kLaneElems], g[kLaneElems], n[kLaneElems];
        terms<DT, SRC>(cur, wr, has_w, mean, rstd, own, d, g, n);
        float sg = 0.0f, sn = 0.0f;
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) {
            if constexpr (SUMS) {
                dw[k] = __builtin_fmaf(d[k], n[k], dw[k]);
                db[k] += d[k];
            }
            sg += g[k];
            sn = __builtin_fmaf(g[k], n[k], sn);
        }
        if constexpr (TEAM) {
            sg = lanes_sum(sg, a.llog);
            sn = lanes_sum(sn, a.llog);
        } else {
            row_sums(sg, sn, lds + turn * 2 * (kRowThreads / kWave), (uint32_t)thread, (uint32_t)a.waves);
        }
        finish_row<DT>(g, n, a.mean != nullptr ? sg * a.inv_h : 0.0f, sn * a.inv_h, rstd, res, has_res,
                       a.dx + row * (uint64_t)H, e, b, H);
        cur = nxt;
        res = nres;
        mean = nmean;
        rstd = nrstd;
    }
    if constexpr (SUMS) {
        float *pw = a.part + block * (uint64_t)(2 * H), *pb = pw + H;
        if constexpr (TEAM) {
            // the workgroup's rows: [team][dw, db][NT * 8], then a column to a thread
            float *mine = lds + thread / NT * (2 * NT * kLaneElems) + tid * kLaneElems;
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) {
                mine[k] = dw[k];
                mine[NT * kLaneElems + k] = db[k];
            }
            __syncthreads();
            const int width = NT * kLaneElems, teams = kTeamThreads / NT;
            for (int c = thread; c < 2 * width; c += kTeamThreads) {
                float s = 0.0f;
                for (int t = 0; t < teams; ++t) s += lds[t * 2 * width + c];
                const int j = c < width ? c : c - width;   // place of the vector's element
                const int ej = j / kLaneElems * kLaneElems, bj = ej < last ? ej : last;
                const int col = bj + j % kLaneElems;
                if (col >= ej && col < H) (c < width ? pw : pb)[col] = s;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) {
                if (b + k >= e && b + k < H) {
                    pw[b + k] = dw[k];
                    pb[b + k] = db[k];
                }
            }
        }
    }
}

// dx of rows that are not held: the row is read for its sums, and again for dx.
template <int DT, int SRC>
__global__ __launch_bounds__(kRowThreads) void layer_norm_back_long_kernel(const LayerNormBackArgs a) {
    __shared__ float lds[2][2 * (kRowThreads / kWave)];
    const int thread = (int)__builtin_amdgcn_workitem_id_x();
    const int H = a.H, last = H - kLaneElems;
    const bool has_w = a.w != nullptr, has_res = a.dres != nullptr;
    int turn = 0;
    for (uint64_t row = __builtin_amdgcn_workgroup_id_x(); row < (uint64_t)a.T; row += (uint32_t)a.grid, turn ^= 1) {
        const float mean = a.mean != nullptr ? a.mean[row] : 0.0f, rstd = a.rstd[row];
        auto vector = [&](int e, float (&d)[kLaneElems], float (&g)[kLaneElems], float (&n)[kLaneElems]) {
            const int b = e < last ? e : last;
            Loaded<SRC> o;
            load_vector<SRC>(a, row, b, o);
            u32x4 wr = {};
            if (has_w) wr = load_row8(a.w, b, H);
            auto own = [&](float (&x)[kLaneElems]) {
#pragma unroll
                for (int k = 0; k < kLaneElems; ++k)
                    if (b + k < e) x[k] = 0.0f;
            };
            terms<DT, SRC>(o, wr, has_w, mean, rstd, own, d, g, n);
        };
        float sg = 0.0f, sn = 0.0f;
        for (int e = thread * kLaneElems; e < H; e += kRowThreads * kLaneElems) {
            float d[kLaneElems], g[kLaneElems], n[kLaneElems];
            vector(e, d, g, n);
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) {
                sg += g[k];
                sn = __builtin_fmaf(g[k], n[k], sn);
            }
        }
        row_sums(sg, sn, lds[turn], (uint32_t)thread, kRowThreads / kWave);
        const float c1 = a.mean != nullptr ? sg * a.inv_h : 0.0f, c2 = sn * a.inv_h;
        for (int e = thread * kLaneElems; e < H; e += kRowThreads * kLaneElems) {
            const int b = e < last ? e : last;
            float d[kLaneElems], g[kLaneElems], n[kLaneElems];
            vector(e, d, g, n);
            u32x4 res = {};
            if (has_res) res = load_row8(a.dres + row * (uint64_t)H, b, H);
            finish_row<DT>(g, n, c1, c2, rstd, res, has_res, a.dx + row * (uint64_t)H, e, b, H);
        }
    }
}

// dw and db of long rows: a wave owns 512 columns, the workgroup's waves take
// every fourth row of blockIdx.y's share, and their sums meet in LDS.
template <int DT, int SRC>
__global__ __launch_bounds__(kColWaves * kWave) void layer_norm_columns_kernel(const LayerNormBackArgs a) {
    __shared__ float lds[kColWaves][2][kWave * kLaneElems];
    const int thread = (int)__builtin_amdgcn_workitem_id_x(), lane = thread & (kWave - 1), wave = thread / kWave;
    const int H = a.H, last = H - kLaneElems;   // H > kHeldElems
    const int e = ((int)__builtin_amdgcn_workgroup_id_x() * kWave + lane) * kLaneElems, b = e < last ? e : last;
    const uint32_t part = __builtin_amdgcn_workgroup_id_y(), parts = (uint32_t)a.grid;
    float dw[kLaneElems] = {}, db[kLaneElems] = {};
    for (uint64_t row = (uint64_t)part * kColWaves + (uint32_t)wave; row < (uint64_t)a.T; row += (uint64_t)parts * kColWaves) {
        Loaded<SRC> o;
        const uint64_t at = row * (uint64_t)H;
        o.dy = load_row8(a.dy + at, b, H);
        if constexpr (SRC == 0) {
            o.x = load_row8(a.x + at, b, H);
        } else {
            o.q = *reinterpret_cast<const u32x2 *>(a.px.codes + at + (uint32_t)b);
            const uint64_t g = row * (uint64_t)a.groups + group_of((uint32_t)b / kLaneElems, a.gmagic);
            o.sz = (uint32_t)a.px.s[g] | (uint32_t)a.px.z[g] << 16;
        }
        float n[kLaneElems], d[kLaneElems];
        normed<DT, SRC>(o, a.mean != nullptr ? a.mean[row] : 0.0f, a.rstd[row], n);
        widen8<DT>(o.dy, d);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) {
            dw[k] = __builtin_fmaf(d[k], n[k], dw[k]);
            db[k] += d[k];
        }
    }
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k) {
        lds[wave][0][lane * kLaneElems + k] = dw[k];
        lds[wave][1][lane * kLaneElems + k] = db[k];
    }
    __syncthreads();
    float *out = a.part + (uint64_t)part * (uint64_t)(2 * H);
    for (int c = thread; c < 2 * kWave * kLaneElems; c += kColWaves * kWave) {
        const int which = c / (kWave * kLaneElems), j = c % (kWave * kLaneElems);
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kColWaves; ++w) s += lds[w][which][j];
        const int ej = ((int)__builtin_amdgcn_workgroup_id_x() * kWave + j / kLaneElems) * kLaneElems;
        const int col = (ej < last ? ej : last) + j % kLaneElems;
        if (col >= ej && col < H) out[which * (uint64_t)H + (uint32_t)col] = s;
    }
}

template <int DT, int SRC, bool TEAM, bool SUMS>
hipError_t launch_kernel(LayerNormBackArgs a, unsigned grid, unsigned threads, hipStream_t stream) {
    a.grid = (int)grid;
    hipLaunchKernelGGL((layer_norm_back_kernel<DT, SRC, TEAM, SUMS>), dim3(grid), dim3(threads), 0, stream, a);
    return hipGetLastError();
}

template <int DT, int SRC>
hipError_t launch_any(LayerNormBackArgs a, hipStream_t stream) {
    const int nv = (a.H + kLaneElems - 1) / kLaneElems;
    const bool sums = a.dw != nullptr || a.db != nullptr;
    const unsigned parts = (unsigned)layer_norm_parts(a.T, a.H);
    hipError_t err;
    if (nv <= kWave) {
        a.llog = lanes_log(nv);
        err = sums ? launch_kernel<DT, SRC, true, true>(a, parts, kTeamThreads, stream)
                   : launch_kernel<DT, SRC, true, false>(a, parts, kTeamThreads, stream);
    } else if (a.H <= kHeldElems) {
        a.waves = (nv + kWave - 1) / kWave;
        err = sums ? launch_kernel<DT, SRC, false, true>(a, parts, (unsigned)(a.waves * kWave), stream)
                   : launch_kernel<DT, SRC, false, false>(a, parts, (unsigned)(a.waves * kWave), stream);
    } else {
        a.grid = a.T < 2 * kParts ? a.T : 2 * kParts;
        hipLaunchKernelGGL((layer_norm_back_long_kernel<DT, SRC>), dim3((unsigned)a.grid), dim3(kRowThreads), 0, stream, a);
        err = hipGetLastError();
    }
    if (err != hipSuccess || !sums) return err;
    if (!layer_norm_sums_in_rows(a.H)) {
        a.grid = (int)parts;
        hipLaunchKernelGGL((layer_norm_columns_kernel<DT, SRC>), dim3((unsigned)((nv + kWave - 1) / kWave), parts),
                           dim3(kColWaves * kWave), 0, stream, a);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    // columns [0, H) are dw, [H, 2H) db
    const float *from = a.dw != nullptr ? a.part : a.part + a.H;
    const int cols = a.dw != nullptr && a.db != nullptr ? 2 * a.H : a.H;
    return launch_column_sum(from, 1, (int)parts, 2 * a.H, cols, a.dw != nullptr ? a.H : 0, a.dw, a.db, stream);
}

}  // namespace

bool layer_norm_sums_in_rows(int H) { return H <= kHeldElems; }

// Workgroups whose sums are added up, at most kParts: one per row (or set of short
// rows) for few of them.
int layer_norm_parts(int T, int H) {
    if (!layer_norm_sums_in_rows(H)) {
        const int n = (T - 1) / kColWaves + 1;
        return n < 64 ? n : 64;
    }
    const int nv = (H + kLaneElems - 1) / kLaneElems;
    const int rows = nv <= kWave ? kTeamThreads >> lanes_log(nv) : 1;
    const int n = (int)(((long long)T + rows - 1) / rows);
    return n < kParts ? n : kParts;
}

hipError_t launch_layer_norm_backward(const LayerNormBackArgs &args, int dtype, hipStream_t stream) {
    LayerNormBackArgs a = args;
    if (a.px.codes == nullptr)
        return dtype == 0 ? launch_any<0, 0>(a, stream) : launch_any<1, 0>(a, stream);
    const uint32_t d = (uint32_t)(a.group / kLaneElems);
    a.groups = a.H / a.group;
    a.gmagic = d == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + d - 1) / d);
    return dtype == 0 ? launch_any<0, 8>(a, stream) : launch_any<1, 8>(a, stream);
}

}  // namespace fc
