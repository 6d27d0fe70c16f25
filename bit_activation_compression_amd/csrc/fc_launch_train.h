// Internal launchers of the training operators (include/fc/train.h). Arguments
// are validated by the C ABI layer before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fc {

// An INT8 payload of rows of H values in groups of `group` (a multiple of 8).
struct Payload {
    const uint8_t *codes;
    const uint16_t *s, *z;
};

// Layer (or RMS) norm of T rows of H; w, b, mean and rstd may be NULL. codes
// (with s, z; a power of two group in [8, 512]): the INT8 payload of x.
struct LayerNormArgs {
    const uint16_t *x, *w, *b;
    uint16_t *y;
    float *mean, *rstd;
    uint8_t *codes;
    uint16_t *s, *z;
    int group;
    int rms;
    float eps, inv_h;
    int T, H;
    int waves, llog;   // set by the launcher: waves of a workgroup, log2 lanes of a row
};
hipError_t launch_layer_norm(const LayerNormArgs &a, int dtype, hipStream_t stream);

// Its backward pass, from x (16-bit) or its payload. mean NULL: RMS norm. w and
// dres may be NULL; dw and db (binary32 [H]) may be NULL. part: binary32
// [parts][2][H] for the workgroups' sums, layer_norm_parts(T, H) of them.
struct LayerNormBackArgs {
    const uint16_t *dy, *x;
    Payload px;
    int group;
    const float *mean, *rstd;
    const uint16_t *w, *dres;
    uint16_t *dx;
    float *dw, *db;
    float *part;
    float inv_h;
    int T, H;
    int groups, waves, llog, teams, grid;   // set by the launcher
    uint32_t gmagic;
};
int layer_norm_parts(int T, int H);
bool layer_norm_sums_in_rows(int H);   // else a second kernel reads dy and x again
hipError_t launch_layer_norm_backward(const LayerNormBackArgs &a, int dtype, hipStream_t stream);

// dz = dy * mul * act'(z), dmul = dy * act(z), db = column sums of dz, for R
// ranks of T rows of H; z and mul (codes NULL: none) are payloads. act 0 has no z
// and writes db only. part: binary32 [R][parts][H], activation_parts(R, T, H).
struct ActBackArgs {
    const uint16_t *dy;
    Payload pz, pm;
    int group;
    int act;
    uint16_t *dz, *dmul;
    float *db, *part;
    int R, T, H;
    int parts, clog, blocks, groups;   // set by the launcher
    uint32_t gmagic;
};
int activation_parts(int R, int T, int H);
hipError_t launch_activation_backward(const ActBackArgs &a, int dtype, hipStream_t stream);

// out[r][c] = sum over p of part[r][p][c], p ascending in a fixed tree: cols
// columns of rows of `stride`, for R ranks with `parts` rows each. Columns from
// `split` on go to out2.
hipError_t launch_column_sum(const float *part, int R, int parts, int stride, int cols, int split,
                             float *out, float *out2, hipStream_t stream);

// n zeros
hipError_t launch_fill_zero(float *out, uint64_t n, hipStream_t stream);

// The epilogue of a linear layer: y = act(a w^T + bias) * mul + residual, z the
// value before the activation. Everything but y may be NULL; act as fc_act.
struct LinearEpilogue {
    const uint16_t *bias, *mul, *residual;
    uint16_t *y, *z;
    int act;
};
// a [R][T][K], w [R][H][K], bias [R][H], the others [R][T][H]; workspaces as
// linear_plan (fc_product_dispatch.h) has them
hipError_t launch_linear_act(const uint16_t *a, const uint16_t *w, int dtype, int R, int T, int K, int H,
                             const LinearEpilogue &e, void *workspace, hipStream_t stream);
// dx[r] = dy[r] w[r] (+ residual): dy [R][T][H], w [R][H][K], dx and residual [R][T][K]
hipError_t launch_linear_input_grad(const uint16_t *dy, const uint16_t *w, int dtype, int R, int T, int K,
                                    int H, const uint16_t *residual, uint16_t *dx, void *workspace,
                                    hipStream_t stream);
// dw[r] (+)= dy[r]^T x[r] for x a payload [R][T][K]; workspace as weight_grad_plan
// (fc_product_dispatch.h) has it
hipError_t launch_linear_weight_grad(const uint16_t *dy, const Payload &px, int group, int dtype, int R,
                                     int T, int K, int H, int accumulate, float *dw, void *workspace,
                                     hipStream_t stream);

}  // namespace fc
