// Argument checks of the transformer-block operators (include/fc/layer.h):
// plain C++, no HIP runtime calls, like fc_validate.h.
#pragma once

#include <float.h>
#include <string.h>

#include "fc/layer.h"
#include "fc_validate.h"

namespace fc {
namespace validate {

constexpr int kMxBlock = 32;              // values that share a scale
constexpr int kMxStep = 128;              // rows are padded to whole matrix-core steps
constexpr int kMxMaxK = 1 << 22;          // row offsets of a tile fit 32 bits
constexpr int kMxMaxH = 1 << 24;
constexpr uint64_t kMxMaxValues = uint64_t(1) << 47;   // of an operand, with its padding: a grid holds them
// a rank's operand rows and a grid's tiles are counted in 32 bits
constexpr long long kMxMaxTiles = 0x7FFFFFFFll;

// By the bits: the build lets the compiler assume that no float is a NaN.
inline bool finite(float v) {
    uint32_t b;
    memcpy(&b, &v, sizeof b);
    return (b & 0x7F800000u) != 0x7F800000u;
}

struct Span {
    const void *p;
    size_t bytes;
};

inline bool overlap(const Span &a, const Span &b) {
    if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return pa < pb + b.bytes && pb < pa + a.bytes;
}

// No output overlaps an input or another output.
inline fc_status check_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (auto p = outs.begin(); p != o; ++p)
            if (overlap(*o, *p)) return FC_ERR_OVERLAP;
        for (const Span &i : ins)
            if (overlap(*o, i)) return FC_ERR_OVERLAP;
    }
    return FC_OK;
}

inline bool optional_aligned(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (p != nullptr && !aligned(p)) return false;
    return true;
}

// What the block-norm calls have in common: T, H, the scalars, and the
// buffers besides the block output itself, which `src` lists.
inline fc_status check_norm(int T, int H, fc_dtype dt, std::initializer_list<Span> src,
                            const void *residual, const void *w_post, const void *gate,
                            int gate_tokens, const void *w_pre, float res_scale, float out_scale,
                            float eps, void *h, void *y) {
    if (T < 0 || H < 1 || H > FC_NORM_MAX_H) return FC_ERR_SHAPE;
    if (gate != nullptr && gate_tokens < 1) return FC_ERR_SHAPE;
    if (dt != FC_F16 && dt != FC_BF16) return FC_ERR_DTYPE;
    if (!finite(res_scale) || !finite(out_scale) || !finite(eps) || eps < FLT_MIN)
        return FC_ERR_VALUE;
    if (T == 0) return FC_OK;
    for (const Span &s : src)
        if (s.p == nullptr) return FC_ERR_NULL;
    if (residual == nullptr || h == nullptr) return FC_ERR_NULL;
    if ((w_pre == nullptr) != (y == nullptr)) return FC_ERR_NULL;
    for (const Span &s : src)
        if (!aligned(s.p)) return FC_ERR_ALIGN;
    if (!optional_aligned({residual, h, y, w_post, gate, w_pre})) return FC_ERR_ALIGN;
    const size_t row = (size_t)H * 2, n = (size_t)T * row;
    const size_t gates = gate ? ((size_t)T + (size_t)gate_tokens - 1) / (size_t)gate_tokens : 0;
    const Span hs = {h, n}, ys = {y, n};
    const Span rest[] = {{residual, h == residual ? 0 : n}, {w_post, row}, {w_pre, row},
                         {gate, gates * row}};
    for (const Span &s : src)
        if (overlap(hs, s) || overlap(ys, s)) return FC_ERR_OVERLAP;
    for (const Span &s : rest)
        if (overlap(hs, s) || overlap(ys, s)) return FC_ERR_OVERLAP;
    return overlap(hs, ys) ? FC_ERR_OVERLAP : FC_OK;
}

inline size_t mx_padded(int K) { return ((size_t)K + kMxStep - 1) / kMxStep * kMxStep; }
inline size_t mx_code_bytes(int R, int rows, int K) { return (size_t)R * (size_t)rows * (mx_padded(K) / 2); }
inline size_t mx_scale_bytes(int R, int rows, int K) {
    return (size_t)R * (size_t)rows * (mx_padded(K) / kMxBlock);
}

inline fc_status check_mx(int R, int rows, int K) {
    if (R < 1 || rows < 0 || K < 1 || K > kMxMaxK) return FC_ERR_SHAPE;
    if ((uint64_t)R * (uint64_t)rows > kMxMaxValues / mx_padded(K)) return FC_ERR_SHAPE;
    return FC_OK;
}

// Both operands, and the tiles of the product's grids: 16 x 16 outputs is the
// smallest tile of any.
inline fc_status check_mx_product(int R, int T, int K, int H) {
    fc_status st = check_mx(R, T, K);
    if (st != FC_OK) return st;
    if (H < 1 || H > kMxMaxH || check_mx(R, H, K) != FC_OK) return FC_ERR_SHAPE;
    const long long tt = ((long long)T + 15) / 16, th = ((long long)H + 15) / 16;
    if (tt * th > kMxMaxTiles / R) return FC_ERR_SHAPE;
    return FC_OK;
}

// Slices of fc_linear_mxfp4's workspace: codes, then scales at the next
// multiple of kSliceAlign.
inline size_t mx_workspace_scales(int R, int T, int K) { return round_up(mx_code_bytes(R, T, K)); }

}  // namespace validate
}  // namespace fc
