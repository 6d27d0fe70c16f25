// Argument checks of the training operators (include/fc/train.h): plain C++, no HIP
// runtime calls, like fc_validate.h.
#pragma once

#include "fc/train.h"
#include "fc_validate_layer.h"

namespace fc {
namespace validate {

constexpr int kProductMaxSize = 1 << 22;        // K and H: row offsets of a tile fit 32 bits
constexpr long long kProductMaxTiles = 0x7FFFFFFFll;
constexpr uint64_t kMaxElems = uint64_t(1) << 48;   // of an operand: byte counts fit 64 bits with room

inline bool payload_group_ok(int H, int group) {
    return group >= 8 && group % 8 == 0 && H <= FC_TRAIN_MAX_ROW && H % group == 0;
}

inline size_t elems(int R, int T, int H) { return (size_t)R * (size_t)T * (size_t)H; }

inline bool elems_ok(int R, int T, int H) {
    return (uint64_t)R * (uint64_t)T <= kMaxElems / (uint64_t)H;
}

// Required pointers are there, and all that are there are aligned.
inline fc_status check_spans(std::initializer_list<Span> required, std::initializer_list<Span> optional) {
    for (const Span &s : required)
        if (s.p == nullptr) return FC_ERR_NULL;
    for (const Span &s : required)
        if (!aligned(s.p)) return FC_ERR_ALIGN;
    for (const Span &s : optional)
        if (s.p != nullptr && !aligned(s.p)) return FC_ERR_ALIGN;
    return FC_OK;
}

inline bool dtype_ok(fc_dtype dt) { return dt == FC_F16 || dt == FC_BF16; }

// The sizes of a product and of its gradients: blocks of 16 x 16 outputs are counted in 31
// bits. No workgroup has fewer: the few-token kernel has 16 channels of all its tokens (up to
// 8), the others tiles of 64 x 64 and more.
inline fc_status check_product(int R, int T, int K, int H) {
    if (R < 1 || T < 0 || K < 1 || H < 1 || K > kProductMaxSize || H > kProductMaxSize) return FC_ERR_SHAPE;
    const long long tt = ((long long)T + 15) / 16, th = ((long long)H + 15) / 16, tk = ((long long)K + 15) / 16;
    if (tt * th > kProductMaxTiles / R || tt * tk > kProductMaxTiles / R || th * tk > kProductMaxTiles / R)
        return FC_ERR_SHAPE;
    return FC_OK;
}

}  // namespace validate
}  // namespace fc
