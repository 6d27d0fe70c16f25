// C ABI of the training operators (declared in include/fc/train.h): argument
// checks, workspaces and launches, and the two kernels that several of them share.
// Every check happens before anything is enqueued.
#include "fc/train.h"
#include "fc_device.h"
#include "fc_grid.h"
#include "fc_launch.h"
#include "fc_launch_train.h"
#include "fc_product_dispatch.h"
#include "fc_validate_train.h"

namespace fc {
namespace {

constexpr int kSumWaves = 16, kSumCols = 16, kSumRows = kSumWaves * (kWave / kSumCols);

// A workgroup sums 16 columns of one rank: each 16 lanes take every 64th row, and their
// sums meet in LDS, in a fixed order. The rows are the workgroups' sums of an earlier
// launch, mostly still in the L2 or the Infinity Cache: this is bound by latency, and
// has as many loads in flight as there are rows.
__global__ __launch_bounds__(kSumWaves * kWave) void column_sum_kernel(const float *part, int parts, int stride, int cols,
                                                                       int split, int blocks, uint64_t total,
                                                                       float *out, float *out2) {
    __shared__ float lds[kSumRows][kSumCols];
    const uint32_t thread = __builtin_amdgcn_workitem_id_x(), lane = thread % kSumCols, first = thread / kSumCols;
    const uint64_t id = grid_index();
    if (id >= total) return;
    const uint64_t r = id / (uint32_t)blocks;
    const int c = (int)(id - r * (uint32_t)blocks) * kSumCols + (int)lane;
    float s = 0.0f;
    if (c < cols) {
        const float *p = part + r * (uint64_t)parts * (uint32_t)stride + (uint32_t)c;
        for (uint32_t i = first; i < (uint32_t)parts; i += kSumRows * 4) {
            float v[4];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                const uint32_t row = i + k * kSumRows;
                v[k] = row < (uint32_t)parts ? p[(uint64_t)row * (uint32_t)stride] : 0.0f;
            }
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
    }
    lds[first][lane] = s;
    __syncthreads();
    if (thread >= kWave) return;
    // 4 lanes to a column, 16 rows each
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumRows / 4; ++i) s += lds[first * (kSumRows / 4) + i][lane];
    s += __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, s), 0x401F));   // lane ^ 16
    const uint32_t bits = __builtin_bit_cast(uint32_t, s);
    const auto halves = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);                     // lane ^ 32
    s = __builtin_bit_cast(float, (uint32_t)halves[0]) + __builtin_bit_cast(float, (uint32_t)halves[1]);
    if (thread >= kSumCols || c >= cols) return;
    if (c < split) out[r * (uint32_t)split + (uint32_t)c] = s;
    else out2[r * (uint32_t)(cols - split) + (uint32_t)(c - split)] = s;
}

__global__ __launch_bounds__(kBlockThreads) void fill_zero_kernel(float *out, uint64_t n) {
    const uint64_t i = grid_index() * kBlockThreads + __builtin_amdgcn_workitem_id_x();
    if (i < n) out[i] = 0.0f;
}

}  // namespace

hipError_t launch_column_sum(const float *part, int R, int parts, int stride, int cols, int split, float *out,
                             float *out2, hipStream_t stream) {
    const int blocks = (cols + kSumCols - 1) / kSumCols;
    const uint64_t total = (uint64_t)R * (uint64_t)blocks;
    hipLaunchKernelGGL(column_sum_kernel, grid_of_blocks(total), dim3(kSumWaves * kWave), 0, stream, part, parts, stride,
                       cols, split, blocks, total, out, out2);
    return hipGetLastError();
}

hipError_t launch_fill_zero(float *out, uint64_t n, hipStream_t stream) {
    hipLaunchKernelGGL(fill_zero_kernel, grid_of_blocks((n + kBlockThreads - 1) / kBlockThreads), dim3(kBlockThreads), 0,
                       stream, out, n);
    return hipGetLastError();
}

}  // namespace fc

namespace {

using namespace fc::validate;

fc_status from_hip(hipError_t e) { return e == hipSuccess ? FC_OK : FC_ERR_LAUNCH; }
const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }
uint16_t *u16(void *p) { return static_cast<uint16_t *>(p); }
float *f32(void *p) { return static_cast<float *>(p); }
hipStream_t stream_of(void *s) { return static_cast<hipStream_t>(s); }

// Zeros where a gradient is a sum over no tokens.
fc_status zero(float *out, size_t n, hipStream_t stream) {
    if (out == nullptr) return FC_OK;
    if (!aligned(out)) return FC_ERR_ALIGN;
    return from_hip(fc::launch_fill_zero(out, n, stream));
}

}  // namespace

extern "C" {

fc_status fc_layer_norm(const void *x, fc_dtype dt, int T, int H, const void *w, const void *b,
                        float eps, int rms, void *y, float *mean, float *rstd, uint8_t *codes,
                        uint16_t *s, uint16_t *z, int group, void *stream) {
    if (T < 0 || H < 1 || H > FC_TRAIN_MAX_NORM_H) return FC_ERR_SHAPE;
    if (codes != nullptr && (!group_ok(group) || H % group != 0)) return FC_ERR_SHAPE;
    if (!dtype_ok(dt)) return FC_ERR_DTYPE;
    if (!finite(eps) || eps < FLT_MIN) return FC_ERR_VALUE;
    if (T == 0) return FC_OK;
    const size_t n = elems(1, T, H), row = (size_t)H * 2;
    if ((codes == nullptr) != (s == nullptr) || (codes == nullptr) != (z == nullptr)) return FC_ERR_NULL;
    if (rms != 0 && mean != nullptr) return FC_ERR_VALUE;
    const Span xs = {x, n * 2}, ys = {y, n * 2}, ws = {w, row}, bs = {b, row}, ms = {mean, (size_t)T * 4},
               rs = {rstd, (size_t)T * 4};
    const size_t meta = codes != nullptr ? n / (size_t)group * 2 : 0;
    const Span cs = {codes, n}, ss = {s, meta}, zs = {z, meta};
    fc_status st = check_spans({xs, ys}, {ws, bs, ms, rs, cs, ss, zs});
    if (st != FC_OK) return st;
    st = check_overlap({ys, ms, rs, cs, ss, zs}, {xs, ws, bs});
    if (st != FC_OK) return st;
    fc::LayerNormArgs a = {};
    a.x = u16(x);
    a.w = u16(w);
    a.b = u16(b);
    a.y = u16(y);
    a.mean = mean;
    a.rstd = rstd;
    a.rms = rms != 0;
    a.eps = eps;
    a.inv_h = 1.0f / (float)H;
    a.T = T;
    a.H = H;
    a.group = group;
    // groups that do not lie in the lanes of a wave: a launch of the quantizer's own
    const bool fused = codes != nullptr && pow2_in_range(group) && group <= 512;
    if (fused) {
        a.codes = codes;
        a.s = s;
        a.z = z;
    } else if (codes != nullptr) {
        st = fc_quantize_groups(x, dt, 1, T, H, 8, group, codes, s, z, stream);
        if (st != FC_OK) return st;
    }
    return from_hip(fc::launch_layer_norm(a, (int)dt, stream_of(stream)));
}

size_t fc_layer_norm_backward_workspace_bytes(int T, int H) {
    if (T < 1 || H < 1 || H > FC_TRAIN_MAX_NORM_H) return 0;
    return (size_t)fc::layer_norm_parts(T, H) * 2 * (size_t)H * 4;
}

fc_status fc_layer_norm_backward(const void *dy, const void *x, const uint8_t *codes,
                                 const uint16_t *s, const uint16_t *z, int group, fc_dtype dt,
                                 int T, int H, const float *mean, const float *rstd, const void *w,
                                 const void *dres, void *dx, float *dw, float *db, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    if (T < 0 || H < 1 || H > FC_TRAIN_MAX_NORM_H) return FC_ERR_SHAPE;
    const bool saved = codes != nullptr;
    if (saved && !payload_group_ok(H, group)) return FC_ERR_SHAPE;
    if (!dtype_ok(dt)) return FC_ERR_DTYPE;
    if (T == 0) {
        if (overlap({dw, (size_t)H * 4}, {db, (size_t)H * 4})) return FC_ERR_OVERLAP;
        if (!optional_aligned({dw, db})) return FC_ERR_ALIGN;
        const fc_status st = zero(dw, (size_t)H, stream_of(stream));
        return st != FC_OK ? st : zero(db, (size_t)H, stream_of(stream));
    }
    if (saved == (x != nullptr)) return FC_ERR_NULL;   // one of the two
    if (saved && (s == nullptr || z == nullptr)) return FC_ERR_NULL;
    const bool sums = dw != nullptr || db != nullptr;
    if (sums && workspace == nullptr) return FC_ERR_NULL;
    const size_t n = elems(1, T, H), row = (size_t)H, meta = saved ? n / (size_t)group * 2 : 0;
    const size_t need = sums ? fc_layer_norm_backward_workspace_bytes(T, H) : 0;
    const Span dys = {dy, n * 2}, xs = {x, n * 2}, cs = {codes, n}, ss = {s, meta}, zs = {z, meta},
               ms = {mean, (size_t)T * 4}, rs = {rstd, (size_t)T * 4}, ws = {w, row * 2}, res = {dres, n * 2},
               dxs = {dx, n * 2}, dws = {dw, row * 4}, dbs = {db, row * 4}, wk = {workspace, need};
    fc_status st = check_spans({dys, rs, dxs}, {xs, cs, ss, zs, ms, ws, res, dws, dbs, wk});
    if (st != FC_OK) return st;
    if (workspace_bytes < need) return FC_ERR_WORKSPACE;
    // the columns of long rows are summed by a second kernel, which reads dy again
    const bool in_place = dx == dy && (!sums || fc::layer_norm_sums_in_rows(H));
    st = check_overlap({dxs}, {in_place ? Span{nullptr, 0} : dys, dx == dres ? Span{nullptr, 0} : res});
    if (st != FC_OK) return st;
    st = check_overlap({dxs, dws, dbs, wk}, {xs, cs, ss, zs, ms, rs, ws});
    if (st != FC_OK) return st;
    st = check_overlap({dws, dbs, wk}, {dys, res});
    if (st != FC_OK) return st;
    fc::LayerNormBackArgs a = {};
    a.dy = u16(dy);
    a.x = u16(x);
    a.px = {codes, s, z};
    a.group = group;
    a.mean = mean;
    a.rstd = rstd;
    a.w = u16(w);
    a.dres = u16(dres);
    a.dx = u16(dx);
    a.dw = dw;
    a.db = db;
    a.part = f32(workspace);
    a.inv_h = 1.0f / (float)H;
    a.T = T;
    a.H = H;
    return from_hip(fc::launch_layer_norm_backward(a, (int)dt, stream_of(stream)));
}

size_t fc_activation_backward_workspace_bytes(int R, int T, int H) {
    if (R < 1 || T < 1 || H < 1 || H > kProductMaxSize || !elems_ok(R, T, H)) return 0;
    const int parts = fc::activation_parts(R, T, H);
    return parts > 1 ? elems(R, parts, H) * 4 : 0;
}

fc_status fc_activation_backward(const void *dy, const uint8_t *codes, const uint16_t *s,
                                 const uint16_t *z, const uint8_t *mul_codes,
                                 const uint16_t *mul_s, const uint16_t *mul_z, int group,
                                 fc_dtype dt, int R, int T, int H, fc_act act, void *dz,
                                 void *dmul, float *db, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    if (R < 1 || T < 0 || H < 1 || H > kProductMaxSize || !elems_ok(R, T, H)) return FC_ERR_SHAPE;
    if (act < FC_ACT_NONE || act > FC_ACT_GELU_TANH) return FC_ERR_VALUE;
    const bool none = act == FC_ACT_NONE, mul = mul_codes != nullptr;
    if (!none && !payload_group_ok(H, group)) return FC_ERR_SHAPE;
    if (!dtype_ok(dt)) return FC_ERR_DTYPE;
    if (T == 0) return zero(db, elems(R, 1, H), stream_of(stream));
    if (none && (codes != nullptr || mul || dz != nullptr || dmul != nullptr)) return FC_ERR_VALUE;
    if (none && db == nullptr) return FC_ERR_NULL;
    if (!none && (codes == nullptr || s == nullptr || z == nullptr || dz == nullptr)) return FC_ERR_NULL;
    if (mul != (dmul != nullptr) || (mul && (mul_s == nullptr || mul_z == nullptr))) return FC_ERR_NULL;
    const size_t n = elems(R, T, H), meta = none ? 0 : n / (size_t)group * 2;
    const size_t need = db != nullptr ? fc_activation_backward_workspace_bytes(R, T, H) : 0;
    if (need != 0 && workspace == nullptr) return FC_ERR_NULL;
    const Span dys = {dy, n * 2}, cs = {codes, n}, ss = {s, meta}, zs = {z, meta}, mc = {mul_codes, n},
               ms = {mul_s, meta}, mz = {mul_z, meta}, dzs = {dz, n * 2}, dms = {dmul, n * 2},
               dbs = {db, elems(R, 1, H) * 4}, wk = {workspace, need};
    fc_status st = check_spans({dys}, {cs, ss, zs, mc, ms, mz, dzs, dms, dbs, wk});
    if (st != FC_OK) return st;
    if (workspace_bytes < need) return FC_ERR_WORKSPACE;
    st = check_overlap({dzs}, {dz == dy ? Span{nullptr, 0} : dys});
    if (st != FC_OK) return st;
    st = check_overlap({dzs, dms, dbs, wk}, {cs, ss, zs, mc, ms, mz});
    if (st != FC_OK) return st;
    st = check_overlap({dms, dbs, wk}, {dys});
    if (st != FC_OK) return st;
    fc::ActBackArgs a = {};
    a.dy = u16(dy);
    a.pz = {codes, s, z};
    if (mul) a.pm = {mul_codes, mul_s, mul_z};
    a.group = group;
    a.act = (int)act;
    a.dz = u16(dz);
    a.dmul = u16(dmul);
    a.db = db;
    a.part = f32(workspace);
    a.R = R;
    a.T = T;
    a.H = H;
    return from_hip(fc::launch_activation_backward(a, (int)dt, stream_of(stream)));
}

size_t fc_linear_act_workspace_bytes(int R, int T, int K, int H) {
    if (check_product(R, T, K, H) != FC_OK || T <= fc::kFewTokens) return 0;
    const int split = fc::linear_plan(R, T, H, K).split;
    return split > 1 ? (size_t)split * elems(R, T, H) * 4 : 0;
}

size_t fc_linear_input_grad_workspace_bytes(int R, int T, int K, int H) {
    if (check_product(R, T, K, H) != FC_OK || T == 0) return 0;
    const int split = fc::linear_plan(R, T, K, H).split;
    return split > 1 ? (size_t)split * elems(R, T, K) * 4 : 0;
}

fc_status fc_linear_act(const void *a, const void *w, fc_dtype dt, int R, int T, int K, int H,
                        const void *bias, fc_act act, const void *mul, const void *residual,
                        void *y, void *z_out, void *workspace, size_t workspace_bytes,
                        void *stream) {
    fc_status st = check_product(R, T, K, H);
    if (st != FC_OK) return st;
    if (act < FC_ACT_NONE || act > FC_ACT_GELU_TANH) return FC_ERR_VALUE;
    if (!dtype_ok(dt)) return FC_ERR_DTYPE;
    if (T == 0) return FC_OK;
    const size_t n = elems(R, T, H) * 2;
    const Span as = {a, elems(R, T, K) * 2}, ws = {w, elems(R, H, K) * 2}, bs = {bias, elems(R, 1, H) * 2},
               ms = {mul, n}, rs = {residual, n}, ys = {y, n}, zs = {z_out, n};
    const size_t need = fc_linear_act_workspace_bytes(R, T, K, H);
    if (need != 0 && workspace == nullptr) return FC_ERR_NULL;
    const Span wk = {workspace, need};
    st = check_spans({as, ws, ys}, {bs, ms, rs, zs, wk});
    if (st != FC_OK) return st;
    if (workspace_bytes < need) return FC_ERR_WORKSPACE;
    st = check_overlap({ys, zs, wk}, {as, ws, bs, ms});
    if (st != FC_OK) return st;
    if ((y != residual && overlap(ys, rs)) || overlap(zs, rs) || overlap(wk, rs)) return FC_ERR_OVERLAP;
    fc::LinearEpilogue e = {};
    e.bias = u16(bias);
    e.mul = u16(mul);
    e.residual = u16(residual);
    e.y = u16(y);
    e.z = u16(z_out);
    e.act = (int)act;
    return from_hip(fc::launch_linear_act(u16(a), u16(w), (int)dt, R, T, K, H, e, workspace, stream_of(stream)));
}

fc_status fc_linear_input_grad(const void *dy, const void *w, fc_dtype dt, int R, int T, int K,
                               int H, const void *residual, void *dx, void *workspace,
                               size_t workspace_bytes, void *stream) {
    fc_status st = check_product(R, T, K, H);
    if (st != FC_OK) return st;
    if (!dtype_ok(dt)) return FC_ERR_DTYPE;
    if (T == 0) return FC_OK;
    const size_t n = elems(R, T, K) * 2;
    const Span ds = {dy, elems(R, T, H) * 2}, ws = {w, elems(R, H, K) * 2}, rs = {residual, n}, xs = {dx, n};
    const size_t need = fc_linear_input_grad_workspace_bytes(R, T, K, H);
    if (need != 0 && workspace == nullptr) return FC_ERR_NULL;
    const Span wk = {workspace, need};
    st = check_spans({ds, ws, xs}, {rs, wk});
    if (st != FC_OK) return st;
    if (workspace_bytes < need) return FC_ERR_WORKSPACE;
    st = check_overlap({xs, wk}, {ds, ws});
    if (st != FC_OK) return st;
    if ((dx != residual && overlap(xs, rs)) || overlap(wk, rs)) return FC_ERR_OVERLAP;
    return from_hip(fc::launch_linear_input_grad(u16(dy), u16(w), (int)dt, R, T, K, H, u16(residual), u16(dx),
                                                 workspace, stream_of(stream)));
}

size_t fc_linear_weight_grad_workspace_bytes(int R, int T, int K, int H) {
    if (check_product(R, T, K, H) != FC_OK || T == 0 || K > FC_TRAIN_MAX_ROW) return 0;
    const fc::WeightGradPlan plan = fc::weight_grad_plan(R, T, K, H);
    return plan.value_bytes + plan.part_bytes;
}

fc_status fc_linear_weight_grad(const void *dy, const uint8_t *codes, const uint16_t *s,
                                const uint16_t *z, int group, fc_dtype dt, int R, int T, int K,
                                int H, int accumulate, float *dw, void *workspace,
                                size_t workspace_bytes, void *stream) {
    fc_status st = check_product(R, T, K, H);
    if (st != FC_OK) return st;
    if (!payload_group_ok(K, group)) return FC_ERR_SHAPE;
    if (!dtype_ok(dt)) return FC_ERR_DTYPE;
    const size_t nw = elems(R, H, K);
    if (T == 0) {
        if (dw == nullptr) return FC_ERR_NULL;
        return accumulate ? FC_OK : zero(dw, nw, stream_of(stream));
    }
    const size_t need = fc_linear_weight_grad_workspace_bytes(R, T, K, H);
    if (need != 0 && workspace == nullptr) return FC_ERR_NULL;
    const size_t n = elems(R, T, K), meta = n / (size_t)group * 2;
    const Span ds = {dy, elems(R, T, H) * 2}, cs = {codes, n}, ss = {s, meta}, zs = {z, meta}, ws = {dw, nw * 4},
               wk = {workspace, need};
    st = check_spans({ds, cs, ss, zs, ws}, {wk});
    if (st != FC_OK) return st;
    if (workspace_bytes < need) return FC_ERR_WORKSPACE;
    st = check_overlap({ws, wk}, {ds, cs, ss, zs});
    if (st != FC_OK) return st;
    return from_hip(fc::launch_linear_weight_grad(u16(dy), {codes, s, z}, group, (int)dt, R, T, K, H, accumulate, dw,
                                                  workspace, stream_of(stream)));
}

}  // extern "C"
