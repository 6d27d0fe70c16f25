/*
 * fc/train.h -- C ABI of training through 8-bit activation checkpoints: the
 * activations that a backward pass needs are kept as the INT8 payloads that
 * fc_quantize_groups writes (fc.h, bits = 8; "Flash Communication: ...", Figure
 * 4), half the bytes of 16-bit ones, and the gradients read the payloads as they
 * are.
 *
 *   - layer norm and RMS norm, forward (with the payload of the input on the way)
 *     and backward (from the input or its payload);
 *   - the linear layer with bias, activation, a second factor and the residual in
 *     the product's epilogue, for training batches and for single tokens;
 *   - its gradients: of the input, and of the weights from the payload of the
 *     input;
 *   - the activation's backward pass from the payload of the pre-activations, with
 *     the bias gradient.
 *
 * The conventions of fc.h and fc/layer.h hold for every call here: device pointers
 * owned by the caller and 16-byte aligned, nothing allocated, asynchronous on
 * `stream`, every argument checked before anything is enqueued, dense row-major
 * layouts. Calls on different streams are independent of each other. An output may
 * not overlap an input or another output (FC_ERR_OVERLAP) except where a call says
 * so. With T == 0 nothing is written, and pointers may be NULL, but for gradients
 * that are sums over tokens: those are zeros then (or stay, where they accumulate; the
 * weight gradient's dw is not NULL in any call).
 *
 * Sums, statistics and sums' partial results are binary32, in an order that the
 * call's sizes fix: the same call gives the same bits. NaN and infinities of 16-bit
 * operands follow the formulas; payloads hold finite values.
 *
 * A payload (codes, s, z) of [..][H] values in groups of `group`: codes [..][H],
 * s and z [..][H / group], the value q * s + z. The calls that read one take groups
 * that are multiples of 8 and divide the row (FC_ERR_SHAPE).
 */
#ifndef FC_TRAIN_H_
#define FC_TRAIN_H_

#include "fc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest row of the norms and of a payload's row here. */
#define FC_TRAIN_MAX_NORM_H 65536
#define FC_TRAIN_MAX_ROW 524288

typedef enum {
    FC_ACT_NONE = 0,
    FC_ACT_RELU = 1,       /* max(z, 0) */
    FC_ACT_SILU = 2,       /* z / (1 + exp(-z)) */
    FC_ACT_GELU = 3,       /* z * Phi(z), Phi the normal distribution's */
    FC_ACT_GELU_TANH = 4   /* z * (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
} fc_act;

/*
 * Layer norm of rows x [T][H], or RMS norm (rms != 0: mean 0):
 *   mean = sum(x) / H, rstd = 1 / sqrt(sum((x - mean)^2) / H + eps)
 *   y = (x - mean) * rstd * w + b      in binary32, rounded once to dt
 *   w, b [H] in dt (NULL: 1 and 0) -> y [T][H] in dt; mean, rstd [T] binary32, both
 *   optional (NULL; mean must be NULL for the RMS norm).
 * With codes != NULL the call also writes the INT8 payload of x, bit for bit what
 * fc_quantize_groups(x, dt, 1, T, H, 8, group, codes, s, z) writes (any group that
 * it takes; powers of two of at most 512 are written by the norm's own launch).
 * Requires 1 <= H <= FC_TRAIN_MAX_NORM_H; eps finite and at least FLT_MIN
 * (FC_ERR_VALUE). Squares are summed in binary32, as for the block norms.
 */
fc_status fc_layer_norm(const void *x, fc_dtype dt, int T, int H, const void *w, const void *b,
                        float eps, int rms, void *y, float *mean, float *rstd, uint8_t *codes,
                        uint16_t *s, uint16_t *z, int group, void *stream);

/*
 * Its backward pass. With n = (x - mean) * rstd and g = dy * w:
 *   dx = rstd * (g - sum_H(g) / H - n * sum_H(g * n) / H) + dres
 *   dw = sum_T(dy * n), db = sum_T(dy)
 *   (mean NULL: RMS norm, n = x * rstd and no sum_H(g) term.)
 *   dy [T][H] in dt; x [T][H] in dt, or (x NULL) its payload codes, s, z; mean, rstd
 *   [T] binary32 as fc_layer_norm gives them (statistics of x itself also where the
 *   payload is read); w [H] in dt (NULL: 1); dres [T][H] in dt, the gradient that
 *   the skip connection brings (NULL: none) -> dx [T][H] in dt (may be dres, or dy);
 *   dw, db [H] binary32, each optional.
 * workspace: fc_layer_norm_backward_workspace_bytes(T, H) bytes where dw or db is
 * asked for (FC_ERR_WORKSPACE); its contents afterwards are unspecified.
 */
fc_status fc_layer_norm_backward(const void *dy, const void *x, const uint8_t *codes,
                                 const uint16_t *s, const uint16_t *z, int group, fc_dtype dt,
                                 int T, int H, const float *mean, const float *rstd, const void *w,
                                 const void *dres, void *dx, float *dw, float *db, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* 0 also where the arguments are unsupported. */
size_t fc_layer_norm_backward_workspace_bytes(int T, int H);

/*
 * Each rank's linear layer with its epilogue, on the matrix cores:
 *   z = sum_k a[r][t][k] * w[r][h][k] + bias[r][h]
 *   y = act(z) * mul[r][t][h] + residual[r][t][h]      rounded once to dt
 *   a [R][T][K], w [R][H][K], bias [R][H], mul, residual [R][T][H], all in dt -> y
 *   [R][T][H] in dt; z_out [R][T][H] in dt: z rounded, what the activation's backward
 *   pass needs a payload of. bias, mul, residual and z_out are optional (NULL). y may
 *   be the same pointer as residual. FC_ACT_NONE with mul (y = z * mul + residual) has no
 *   backward call here: fc_activation_backward takes a second factor with an activation.
 * Any sizes with R, K, H >= 1, K, H <= 2^22 and R * ceil(T/16) * ceil(H/16) < 2^31;
 * rows that are whole 16-byte vectors (K % 8 == 0) are faster. workspace:
 * fc_linear_act_workspace_bytes(R, T, K, H) bytes (0 and NULL allowed where the sums
 * are not split); its contents afterwards are unspecified.
 */
fc_status fc_linear_act(const void *a, const void *w, fc_dtype dt, int R, int T, int K, int H,
                        const void *bias, fc_act act, const void *mul, const void *residual,
                        void *y, void *z_out, void *workspace, size_t workspace_bytes,
                        void *stream);

/* 0 also where the arguments are unsupported. */
size_t fc_linear_act_workspace_bytes(int R, int T, int K, int H);

/*
 * The gradient of the layer's input: dx[r][t][k] = sum_h dy[r][t][h] * w[r][h][k] +
 * residual[r][t][k], rounded once to dt.
 *   dy [R][T][H], w [R][H][K], residual [R][T][K] (NULL: none; the gradient that the
 *   skip connection brings) -> dx [R][T][K], all in dt; dx may be the same pointer as
 *   residual. Sizes as for fc_linear_act.
 */
fc_status fc_linear_input_grad(const void *dy, const void *w, fc_dtype dt, int R, int T, int K,
                               int H, const void *residual, void *dx, void *workspace,
                               size_t workspace_bytes, void *stream);

/* 0 also where the arguments are unsupported. */
size_t fc_linear_input_grad_workspace_bytes(int R, int T, int K, int H);

/*
 * The gradient of the weights, from the payload of the layer's input:
 *   dw[r][h][k] = sum_t dy[r][t][h] * x[r][t][k]  (+ dw[r][h][k] with accumulate != 0)
 *   dy [R][T][H] in dt, payload of [R][T][K] -> dw [R][H][K] binary32.
 * x is the payload's value rounded to dt (what fc_dequantize writes): the matrix
 * cores take 16-bit operands. Sizes as for fc_linear_act, K <= FC_TRAIN_MAX_ROW.
 * workspace: fc_linear_weight_grad_workspace_bytes(R, T, K, H) bytes: the values as
 * 16-bit ones for layers of many outputs, parts of the sums where few outputs sum over
 * many tokens, else 0 (NULL allowed); its contents afterwards are unspecified.
 */
fc_status fc_linear_weight_grad(const void *dy, const uint8_t *codes, const uint16_t *s,
                                const uint16_t *z, int group, fc_dtype dt, int R, int T, int K,
                                int H, int accumulate, float *dw, void *workspace,
                                size_t workspace_bytes, void *stream);

/* 0 also where the arguments are unsupported. */
size_t fc_linear_weight_grad_workspace_bytes(int R, int T, int K, int H);

/*
 * The activation's backward pass from the payload (codes, s, z) of its input:
 *   dz = dy * mul * act'(z), dmul = dy * act(z)     each rounded once to dt
 *   db[r][h] = sum_t dz[r][t][h]                    of dz before its rounding
 *   dy [R][T][H] in dt; mul: the payload (mul_codes, mul_s, mul_z) of the second
 *   factor, in the same groups, NULL for none (dmul must then be NULL) -> dz, dmul
 *   [R][T][H] in dt (dz may be dy), db [R][H] binary32 (optional).
 * act == FC_ACT_NONE: the bias gradient of a layer without an activation, db =
 * sum_t dy; payloads, dz and dmul must be NULL, db not (FC_ERR_VALUE: a second factor
 * without an activation has no call here), and H is any up to 2^22.
 * The slope of relu at 0 is 0. workspace:
 * fc_activation_backward_workspace_bytes(R, T, H) bytes where db is asked for (0 and
 * NULL allowed where the tokens are not split).
 */
fc_status fc_activation_backward(const void *dy, const uint8_t *codes, const uint16_t *s,
                                 const uint16_t *z, const uint8_t *mul_codes,
                                 const uint16_t *mul_s, const uint16_t *mul_z, int group,
                                 fc_dtype dt, int R, int T, int H, fc_act act, void *dz,
                                 void *dmul, float *db, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* 0 also where the arguments are unsupported. */
size_t fc_activation_backward_workspace_bytes(int R, int T, int H);

#ifdef __cplusplus
}
#endif

#endif /* FC_TRAIN_H_ */
