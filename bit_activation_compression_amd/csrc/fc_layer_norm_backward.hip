// Backward pass of the layer and RMS norm (include/fc/train.h,
// fc_layer_norm_backward), from the saved 16-bit x or from its INT8 payload:
//
//   n = (x - mean) * rstd, g = dy * w
//   dx = rstd * (g - mean_H(g) - n * mean_H(g * n)) + dres     (no mean_H(g) for RMS)
//   dw = sum over rows of dy * n,  db = sum over rows of dy
//
// A workgroup of up to 16 waves walks the rows, a vector of 8 elements to a thread, as
// many rows side by side as fit it: the row stays in registers, as
// loaded, between its two uses, the next row's operands are in flight meanwhile, and
// each thread keeps its columns' sums of dw and db, which a second launch adds up over
// the workgroups in a fixed order. dy and x are read once and dx written once, 6 bytes
// per element (5 from a payload): bound by memory. Rows of more than 8192 elements are
// read twice, the second time mostly from the L2, and leave dw and db to a kernel that
// reads dy and x by columns.
//
// Measured (rotating buffers that no cache holds, the second launch with it): 8192 x 8192 bf16
// from a payload 82 us, 4.1 TB/s, with dres 95, 5.0; from x 84, 4.8, with dres 108, without dw
// and db 78; 8192 x 4096 fp16 49 and 50; 1777 x 5003 from x, its rows aligned to 2 bytes, 27,
// without dw and db 19; 4096 x 1024 13, without 7; 2048 x 16384 (read twice) 80, without 50, from
// a payload 75. Vector instructions take half of the issue slots, and no unit is full: a
// compute unit has one workgroup, whose waves meet once a row.
#include "fc_grid.h"
#include "fc_launch_train.h"
#include "fc_rows.h"

namespace fc {
namespace {

constexpr int kRowThreads = 1024;       // most of a workgroup
constexpr int kHeldElems = kRowThreads * kLaneElems;   // longest row that is held in registers
constexpr int kParts = 256;             // most workgroups whose sums are added up
constexpr int kLongGrid = 1024;         // most workgroups of rows that are read twice
constexpr int kColWaves = 4;            // of a column kernel's workgroup

typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// One vector of a row's operands, as loaded.
template <int SRC>
struct Loaded {
    u32x4 dy;
    u32x4 x;         // 16-bit x
    u32x2 q;         // or codes
    uint16_t s, z;   // with scale and zero
};

// 8 elements of a row from b; WHOLE: the row has as many.
template <bool WHOLE>
__device__ __forceinline__ u32x4 load8(const uint16_t *row, int b, int H) {
    if constexpr (WHOLE) return *reinterpret_cast<const u32x4_a2 *>(row + b);
    else return load_row8(row, b, H);
}

template <int SRC, bool WHOLE>
__device__ __forceinline__ void load_vector(const LayerNormBackArgs &a, uint64_t row, int b, Loaded<SRC> &o) {
    const uint64_t at = row * (uint64_t)a.H;
    o.dy = load8<WHOLE>(a.dy + at, b, a.H);
    if constexpr (SRC == 0) {
        o.x = load8<WHOLE>(a.x + at, b, a.H);
    } else {
        // rows are whole vectors here: groups are multiples of 8
        o.q = *reinterpret_cast<const u32x2 *>(a.px.codes + at + (uint32_t)b);
        const uint64_t g = row * (uint64_t)a.groups + group_of((uint32_t)b / kLaneElems, a.gmagic);
        o.s = a.px.s[g];
        o.z = a.px.z[g];
    }
}

// n of the vector: (x - mean) * rstd of 16-bit x, the difference first, so that n keeps its
// digits where the mean is far above the deviations. Codes take one fma, of q * s and of
// z - mean, which is in a group's range too (each code is a subnormal half: a code and its
// position scaled by 2^-24, as in dequant8).
template <int DT, int SRC>
__device__ __forceinline__ void normed(const Loaded<SRC> &o, float mean, float rstd, float (&n)[kLaneElems]) {
    if constexpr (SRC == 0) {
        widen8<DT>(o.x, n);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) n[k] = (n[k] - mean) * rstd;
    } else {
        const float sc = half_bits_to_float(o.s) * rstd * 16777216.0f;
        const float c = (half_bits_to_float(o.z) - mean) * rstd;
        const uint32_t w[2] = {o.q.x, o.q.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f16x2 even = __builtin_bit_cast(f16x2, w[j] & 0x00FF00FFu);
            const f16x2 odd = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w[j], w[j], 0x0C030C01u));
            n[4 * j] = __builtin_fmaf((float)even.x, sc, c);
            n[4 * j + 1] = __builtin_fmaf((float)odd.x, sc, c);
            n[4 * j + 2] = __builtin_fmaf((float)even.y, sc, c);
            n[4 * j + 3] = __builtin_fmaf((float)odd.y, sc, c);
        }
    }
}

// A copy in registers of its own. The next row's loads then land in the variable's
// registers; the compiler would rather copy those once they have landed, and wait for
// them (and for the stores before them) at the end of each row.
__device__ __forceinline__ float moved(float v) {
    float r;
    asm volatile("v_mov_b32 %0, %1" : "=v"(r) : "v"(v));
    return r;
}
__device__ __forceinline__ u32x4 moved(const u32x4 &v) {
    uint32_t r[4];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("v_mov_b32 %0, %1" : "=v"(r[i]) : "v"(w[i]));
    return u32x4{r[0], r[1], r[2], r[3]};
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

// Both sums of a row over its waves, nw from `first`, through one barrier. The two turns' places
// alternate: the next row's sums cannot reach a place that is still read.
__device__ __forceinline__ void row_sums(float &sg, float &sn, float *p, uint32_t thread, uint32_t first, uint32_t nw) {
    sg = wave_sum(sg);
    sn = wave_sum(sn);
    const uint32_t i = thread & 15u;
    if ((thread & (kWave - 1)) == 0) {
        p[2 * (thread / kWave)] = sg;
        p[2 * (thread / kWave) + 1] = sn;
    }
    __syncthreads();
    sg = row_sum(i < nw ? p[2 * (first + i)] : 0.0f);
    sn = row_sum(i < nw ? p[2 * (first + i) + 1] : 0.0f);
}

template <int DT>
__device__ __forceinline__ void finish_row(const float (&g)[kLaneElems], const float (&n)[kLaneElems], float c1, float c2,
                                           float rstd, const u32x4 &res, bool has_res, uint16_t *drow, int e, int b, int H) {
    float d[kLaneElems];
    const float cn = -c2 * rstd, cg = -c1 * rstd;
#pragma unroll
    for (int k = 0; k < kLaneElems; ++k) d[k] = __builtin_fmaf(g[k], rstd, __builtin_fmaf(n[k], cn, cg));
    if (has_res) {
        float r[kLaneElems];
        widen8<DT>(res, r);
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) d[k] += r[k];
    }
    store_row8<DT>(drow, e, b, H, d);
}

// WAVES: a row is a.waves whole waves, else 2^llog lanes. The workgroup has a.teams
// rows at a time; what they sum meets in LDS at the end.
template <int DT, int SRC, bool WAVES, bool SUMS>
__global__ __launch_bounds__(kRowThreads) void layer_norm_back_kernel(const LayerNormBackArgs a) {
    extern __shared__ float lds[];   // [teams][dw, db][NT * 8]
    __shared__ float sums[2][2 * (kRowThreads / kWave)];
    const int thread = (int)__builtin_amdgcn_workitem_id_x();
    const int NT = WAVES ? a.waves * kWave : 1 << a.llog;
    const int team = WAVES ? (int)__builtin_amdgcn_readfirstlane((uint32_t)thread / kWave) / a.waves : thread >> a.llog;
    const int tid = thread - team * NT;
    const int H = a.H;
    // the vector's elements are those from e; its load takes 8 whole ones from b
    const int e = tid * kLaneElems, last = H > kLaneElems ? H - kLaneElems : 0, b = e < last ? e : last;
    auto own = [&](float (&x)[kLaneElems]) {
        if (e + kLaneElems <= H) return;
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k)
            if (b + k < e || b + k >= H) x[k] = 0.0f;
    };
    const uint64_t block = __builtin_amdgcn_workgroup_id_x(), step = (uint64_t)(uint32_t)a.grid * (uint32_t)a.teams;
    const bool has_w = a.w != nullptr, has_res = a.dres != nullptr;
    u32x4 wr = {};
    if (has_w) wr = load8<WAVES>(a.w, b, H);
    float dw[kLaneElems] = {}, db[kLaneElems] = {};
    // the operands of the team's next row, in flight while this one is summed and stored
    Loaded<SRC> in = {};
    u32x4 res = {};
    float mean = 0.0f, rstd = 0.0f;
    auto fetch = [&](uint64_t r) {
        if (r >= (uint64_t)a.T) return;
        load_vector<SRC, WAVES>(a, r, b, in);
        if (a.mean != nullptr) mean = a.mean[r];
        rstd = a.rstd[r];
        if (has_res) res = load8<WAVES>(a.dres + r * (uint64_t)H, b, H);
    };
    uint64_t row = block * (uint32_t)a.teams + (uint32_t)team;
    fetch(row);
    int turn = 0;
    // as many turns for every team: they meet
    for (uint64_t base = block * (uint32_t)a.teams; base < (uint64_t)a.T; base += step, row += step, turn ^= 1) {
        const bool live = row < (uint64_t)a.T;
        float d[kLaneElems], g[kLaneElems], n[kLaneElems];
        float sg = 0.0f, sn = 0.0f;
        const float rs = moved(rstd);
        const u32x4 rv = moved(res);
        if (live) {
            terms<DT, SRC>(in, wr, has_w, mean, rstd, own, d, g, n);
            fetch(row + step);
#pragma unroll
            for (int k = 0; k < kLaneElems; ++k) {
                if constexpr (SUMS) {
                    dw[k] = __builtin_fmaf(d[k], n[k], dw[k]);
                    db[k] += d[k];
                }
                sg += g[k];
                sn = __builtin_fmaf(g[k], n[k], sn);
            }
        }
        if constexpr (WAVES) row_sums(sg, sn, sums[turn], (uint32_t)thread, (uint32_t)(team * a.waves), (uint32_t)a.waves);
        if (live) {
            if constexpr (!WAVES) {
                sg = lanes_sum(sg, a.llog);
                sn = lanes_sum(sn, a.llog);
            }
            finish_row<DT>(g, n, a.mean != nullptr ? sg * a.inv_h : 0.0f, sn * a.inv_h, rs, rv, has_res,
                           a.dx + row * (uint64_t)H, e, b, H);
        }
    }
    if constexpr (SUMS) {
        // one workgroup writes the gradients themselves
        float *pw = a.grid == 1 ? a.dw : a.part + block * (uint64_t)(2 * H), *pb = a.grid == 1 ? a.db : pw + H;
        if (a.teams == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float *out = h == 0 ? pw : pb;
                const float (&v)[kLaneElems] = h == 0 ? dw : db;
                if (out == nullptr) continue;
                if (e + kLaneElems <= H) {
                    *reinterpret_cast<f32x4_a4 *>(out + e) = f32x4_a4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4_a4 *>(out + e + 4) = f32x4_a4{v[4], v[5], v[6], v[7]};
                } else {
#pragma unroll
                    for (int k = 0; k < kLaneElems; ++k)
                        if (b + k >= e && b + k < H) out[b + k] = v[k];
                }
            }
            return;
        }
        const int width = NT * kLaneElems;
        float *mine = lds + team * (2 * width) + tid * kLaneElems;
#pragma unroll
        for (int k = 0; k < kLaneElems; ++k) {
            mine[k] = dw[k];
            mine[width + k] = db[k];
        }
        __syncthreads();
        for (int c = thread; c < 2 * width; c += a.teams * NT) {
            float s = 0.0f;
            for (int t = 0; t < a.teams; ++t) s += lds[t * 2 * width + c];
            const int j = c < width ? c : c - width;   // place of the vector's element
            const int ej = j / kLaneElems * kLaneElems, bj = ej < last ? ej : last;
            const int col = bj + j % kLaneElems;
            float *out = c < width ? pw : pb;
            if (out != nullptr && col >= ej && col < H) out[col] = s;
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
            load_vector<SRC, true>(a, row, b, o);
            u32x4 wr = {};
            if (has_w) wr = load8<true>(a.w, b, H);
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
        row_sums(sg, sn, lds[turn], (uint32_t)thread, 0, kRowThreads / kWave);
        const float c1 = a.mean != nullptr ? sg * a.inv_h : 0.0f, c2 = sn * a.inv_h;
        for (int e = thread * kLaneElems; e < H; e += kRowThreads * kLaneElems) {
            const int b = e < last ? e : last;
            float d[kLaneElems], g[kLaneElems], n[kLaneElems];
            vector(e, d, g, n);
            u32x4 res = {};
            if (has_res) res = load8<true>(a.dres + row * (uint64_t)H, b, H);
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
        load_vector<SRC, false>(a, row, b, o);
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

// Lanes (a power of two) or whole waves of a row, and rows that a workgroup has at a
// time.
struct RowPlan {
    bool waves;
    int count, teams;
};
RowPlan row_plan(int H) {
    const int nv = (H + kLaneElems - 1) / kLaneElems;
    if (nv <= kWave) return {false, lanes_log(nv), kRowThreads >> lanes_log(nv)};
    const int waves = (nv + kWave - 1) / kWave;
    return {true, waves, kRowThreads / kWave / waves};
}

template <int DT, int SRC, bool WAVES, bool SUMS>
hipError_t launch_kernel(LayerNormBackArgs a, const RowPlan &p, unsigned grid, hipStream_t stream) {
    a.grid = (int)grid;
    a.waves = a.llog = p.count;
    a.teams = p.teams;
    const unsigned row = WAVES ? (unsigned)(p.count * kWave) : 1u << p.count, threads = row * (unsigned)p.teams;
    const unsigned lds = SUMS && p.teams > 1 ? threads * kLaneElems * 2 * (unsigned)sizeof(float) : 0;
    hipLaunchKernelGGL((layer_norm_back_kernel<DT, SRC, WAVES, SUMS>), dim3(grid), dim3(threads), lds, stream, a);
    return hipGetLastError();
}

template <int DT, int SRC>
hipError_t launch_any(LayerNormBackArgs a, hipStream_t stream) {
    const int nv = (a.H + kLaneElems - 1) / kLaneElems;
    const bool sums = a.dw != nullptr || a.db != nullptr;
    const unsigned parts = (unsigned)layer_norm_parts(a.T, a.H);
    hipError_t err;
    if (a.H <= kHeldElems) {
        const RowPlan p = row_plan(a.H);
        if (sums)
            err = p.waves ? launch_kernel<DT, SRC, true, true>(a, p, parts, stream)
                          : launch_kernel<DT, SRC, false, true>(a, p, parts, stream);
        else
            err = p.waves ? launch_kernel<DT, SRC, true, false>(a, p, parts, stream)
                          : launch_kernel<DT, SRC, false, false>(a, p, parts, stream);
        if (parts == 1) return err;
    } else {
        a.grid = a.T < kLongGrid ? a.T : kLongGrid;
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

// Workgroups whose sums are added up: one for each compute unit (16 waves: the registers
// hold 20), fewer where there are fewer rows. Two where they fit are slower for the sums of
// twice the workgroups, us at 256 and at 512: 4096 x 1024 13 and 17, 8192 x 4096 50 and 58, 1777
// x 5003 27 and 33, 8192 x 5120 54 and 59, 8192 x 6144 64 and 71, 8192 x 8192 84 and 92. Without
// dw and db they are level but at rows of 10 waves: 1777 x 5003 19.5 and 17.1, 8192 x 5120 53 and
// 48.
int layer_norm_parts(int T, int H) {
    if (!layer_norm_sums_in_rows(H)) {
        const int n = (T - 1) / kColWaves + 1;
        return n < 64 ? n : 64;
    }
    const int n = (T - 1) / row_plan(H).teams + 1;
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
