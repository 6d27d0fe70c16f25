/*
 * fc/layer.h -- C ABI of the transformer-block operators next to the low-bit
 * all-reduce of fc.h ("Flash Communication: ...", Figure 3: the attention and
 * the MLP outputs are all-reduced, added to the residual stream and normed
 * before the next linear layers).
 *
 *   - block norms: the norm after a block (on its output), the gated and
 *     scaled residual update, and the norm before the next block, in one pass;
 *     on a 16-bit block output, on the all-gathered payload of the all-reduce,
 *     or as the last step of the emulated all-reduce;
 *   - microscaled 4-bit floating point (MXFP4): quantize, dequantize, and the
 *     linear layer on it.
 *
 * The conventions of fc.h hold for every call here: device pointers owned by
 * the caller and 16-byte aligned, nothing allocated, asynchronous on `stream`,
 * every argument checked before anything is enqueued, dense row-major layouts,
 * T == 0 valid. Calls on different streams are independent of each other (the
 * library keeps nothing between calls). An output may not overlap an input or
 * another output (FC_ERR_OVERLAP) except where a call says so.
 */
#ifndef FC_LAYER_H_
#define FC_LAYER_H_

#include "fc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest H of the block norms (a row is held in one workgroup's registers). */
#define FC_NORM_MAX_H 65536

/*
 * Block norms on a 16-bit block output. For every token t, in binary32 with
 * one rounding to dt for h and one for y:
 *   n = w_post ? w_post * x / sqrt(mean(x^2) + eps) : x
 *   h = res_scale * residual + out_scale * gate[t / gate_tokens] * n
 *   y = w_pre * h / sqrt(mean(h^2) + eps)        (of h before its rounding)
 *   x, residual [T][H], w_post, w_pre [H], gate [ceil(T / gate_tokens)][H],
 *   all in dt -> h, y [T][H] in dt.
 * w_post, gate and w_pre are optional (NULL): no post-norm, a gate of 1, no
 * y (y must then be NULL too). gate_tokens is the number of consecutive
 * tokens that share a gate row: 1 for a gate per token, T or more for one row
 * for all; ignored without a gate. h may be the same pointer as residual
 * (in-place update of the residual stream).
 * Requires 1 <= H <= FC_NORM_MAX_H and, with a gate, gate_tokens >= 1
 * (FC_ERR_SHAPE); res_scale and out_scale finite, eps finite and at least
 * FLT_MIN (FC_ERR_VALUE). Squares are summed in binary32: |x| or |h| above
 * about 1.8e19 / sqrt(H) overflows the sum, and the normed row is then 0.
 * NaN and infinities follow the formulas, within their own row.
 */
fc_status fc_residual_norm(const void *x, const void *residual, fc_dtype dt, int T, int H,
                           const void *w_post, const void *gate, int gate_tokens,
                           const void *w_pre, float res_scale, float out_scale, float eps, void *h,
                           void *y, void *stream);

/*
 * The same with x = fp32(q * s + z), the dequantized payload of the
 * All-Gather (not rounded to dt in between).
 *   codes2 [T][H*bits/8], s2, z2 [T][H/group2] as for fc_dequantize.
 * bits in {4, 8} (FC_ERR_BITS), group2 even and dividing H (FC_ERR_SHAPE).
 */
fc_status fc_dequantize_residual_norm(const uint8_t *codes2, const uint16_t *s2,
                                      const uint16_t *z2, int T, int H, int bits, int group2,
                                      fc_dtype dt, const void *residual, const void *w_post,
                                      const void *gate, int gate_tokens, const void *w_pre,
                                      float res_scale, float out_scale, float eps, void *h,
                                      void *y, void *stream);

/*
 * fc_allreduce_emulated_mixed whose last step is fc_dequantize_residual_norm:
 * x [R][T][H] -> h, y [T][H]. Shapes, widths, workspace and its layout as for
 * fc_allreduce_emulated_mixed; the payloads in the workspace are the same bits.
 */
fc_status fc_allreduce_emulated_norm(const void *x, fc_dtype dt, int R, int T, int H, int bits1,
                                     int bits2, int group, const void *residual,
                                     const void *w_post, const void *gate, int gate_tokens,
                                     const void *w_pre, float res_scale, float out_scale,
                                     float eps, void *h, void *y, void *workspace,
                                     size_t workspace_bytes, void *stream);

/*
 * MXFP4, the 4-bit format of the OCP Microscaling (MX) specification: 32
 * consecutive k values of a row share a scale 2^E (one byte, E + 127; 255 is
 * NaN), each value is an E2M1 code (sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6).
 * Layout of [R][rows][K] values, Kp = K rounded up to a multiple of 128:
 *   codes  [R][rows][Kp/2]    uint8, the even element in the low nibble
 *   scales [R][rows][Kp/32]   uint8
 * The values past K are zeros: codes 0 and, where a whole block lies past K,
 * scale 0. A caller that brings codes of its own pads them the same way.
 * Requires R >= 1, rows (T or H) >= 0, 1 <= K <= 2^22 and R * rows * Kp <= 2^47.
 */

/*
 * Quantize x [R][T][K] in dt: per block
 *   E = clamp(floor(log2(max|x|)) - 2, -127, 127)   (an all-zero block: -127)
 *   code = the E2M1 value nearest to x / 2^E, ties to the even code,
 *          saturating at 6, the sign kept
 * A block that holds a NaN or an infinity gets scale 255 and codes 0 (it
 * dequantizes to NaN); other blocks are not touched by it.
 */
fc_status fc_quantize_mxfp4(const void *x, fc_dtype dt, int R, int T, int K, uint8_t *codes,
                            uint8_t *scales, void *stream);

/* out [R][T][K] in dt = code * 2^E, rounded to dt (exact in bf16 for E <= 125). */
fc_status fc_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int R, int T, int K,
                              fc_dtype dt, void *out, void *stream);

/*
 * Each rank's linear layer on MXFP4 operands, on the scaled matrix cores:
 *   y[r][t][h] = round_half_even_to_dt(sum_k a[r][t][k] * w[r][h][k])
 *   a codes and scales [R][T][K], w codes and scales [R][H][K] as above,
 *   y [R][T][H] in dt.
 * Products are summed in binary32, in an order that the call's shape fixes:
 * calls of different T or R may differ in a sum's last bits. Subnormal sums are
 * kept, what lies below 2^-149 is rounded away (both scales near 2^-127: the
 * outputs are zeros), and sums that overflow on the way are infinities or NaN.
 * A NaN scale makes the outputs of its token row (or output channel) NaN.
 * Requires 1 <= H <= 2^24 and R * ceil(T/16) * ceil(H/16) < 2^31 besides.
 */
fc_status fc_matmul_mxfp4(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                          const uint8_t *w_scales, int R, int T, int K, int H, fc_dtype dt,
                          void *y, void *stream);

/*
 * The same for 16-bit activations a [R][T][K] in dt, quantized in the call as
 * fc_quantize_mxfp4 does. workspace: fc_linear_mxfp4_workspace_bytes(R, T, K)
 * bytes for the activations' codes and scales (0, and NULL allowed, where the
 * product quantizes them itself); its contents afterwards are unspecified.
 */
fc_status fc_linear_mxfp4(const void *a, const uint8_t *w_codes, const uint8_t *w_scales,
                          fc_dtype dt, int R, int T, int K, int H, void *y, void *workspace,
                          size_t workspace_bytes, void *stream);

/* 0 also where the arguments are unsupported. */
size_t fc_linear_mxfp4_workspace_bytes(int R, int T, int K);

#ifdef __cplusplus
}
#endif

#endif /* FC_LAYER_H_ */
