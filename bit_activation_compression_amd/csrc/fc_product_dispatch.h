// The rules that choose the tiles of the matrix products (fc_product.h): host code
// without HIP, so that tests can run it on its own.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace fc {

constexpr int kLargeTile = 256, kMiddleTile = 128, kSmallTile = 64;

// The tiles of a product of M x N outputs, `batches` of them: up to two parts, rows
// [from_m, to_m) x columns [from_n, to_n) in tiles of `tile` (0: no such part).
struct ProductPlan {
    struct Part {
        int tile, from_m, to_m, from_n, to_n;
    } part[2];
};

inline long long tile_count(long long n, int tile) { return (n + tile - 1) / tile; }

// Cost of `tiles` tiles in units of a tile of 256 that has a compute unit to itself. A
// compute unit holds one workgroup of 256, two of 128 or four of 64.
inline double tile_cost(long long tiles, int tile, int cus) {
    const int at_once = tile == kLargeTile ? 1 : tile == kMiddleTile ? 2 : 4;
    const double one = tile == kLargeTile ? 1.0 : tile == kMiddleTile ? 0.34 : 0.16;     // alone on its compute unit
    const double full = tile == kLargeTile ? 1.0 : tile == kMiddleTile ? 0.58 : 0.40;    // with the others beside it
    const long long per = (tiles + cus - 1) / cus;       // of the fullest compute unit
    const long long rounds = per / at_once, rest = per % at_once;
    return (double)rounds * full + (rest ? one + (full - one) * (double)(rest - 1) / (double)(at_once - 1 ? at_once - 1 : 1) : 0.0);
}

// large: tiles of 256 exist for the operands.
inline ProductPlan product_plan(long long batches, int M, int N, int cus, bool large) {
    ProductPlan plan = {};
    double best = -1.0;
    auto consider = [&](double cost, ProductPlan::Part a, ProductPlan::Part b) {
        if (best >= 0.0 && cost >= best) return;
        best = cost;
        plan.part[0] = a;
        plan.part[1] = b;
    };
    const ProductPlan::Part none = {};
    for (int tile : {kMiddleTile, kSmallTile})
        consider(tile_cost(batches * tile_count(M, tile) * tile_count(N, tile), tile, cus), {tile, 0, M, 0, N}, none);
    if (!large) return plan;
    const long long tm = tile_count(M, kLargeTile), tn = tile_count(N, kLargeTile);
    consider(tile_cost(batches * tm * tn, kLargeTile, cus), {kLargeTile, 0, M, 0, N}, none);
    // whole rounds of large tiles over the first columns (rows), the others in middle ones
    const long long rounds = batches * tm * tn / cus;
    if (rounds >= 1) {
        const long long c = rounds * cus / (batches * tm), r = rounds * cus / (batches * tn);
        if (c >= 1 && c < tn) {
            const int cut = (int)(c * kLargeTile);
            consider(tile_cost(batches * tm * c, kLargeTile, cus) +
                         tile_cost(batches * tile_count(M, kMiddleTile) * tile_count(N - cut, kMiddleTile), kMiddleTile, cus),
                     {kLargeTile, 0, M, 0, cut}, {kMiddleTile, 0, M, cut, N});
        }
        if (r >= 1 && r < tm) {
            const int cut = (int)(r * kLargeTile);
            consider(tile_cost(batches * r * tn, kLargeTile, cus) +
                         tile_cost(batches * tile_count(M - cut, kMiddleTile) * tile_count(N, kMiddleTile), kMiddleTile, cus),
                     {kLargeTile, 0, cut, 0, N}, {kMiddleTile, cut, M, 0, N});
        }
    }
    return plan;
}

// How a weight gradient of R x H x K sums over T tokens runs. It goes by the sizes
// alone, so that the workspace is the same on every device.
struct WeightGradPlan {
    size_t value_bytes;   // of the activations as 16-bit values, 0: codes are read by the product
    size_t part_bytes;    // of the splits' sums (after the values), 0: one split
    int split, split_k;   // tokens in `split` runs of split_k, none of them empty
};

inline WeightGradPlan weight_grad_plan(int R, int T, int K, int H) {
    constexpr long long kStage = 64, kFill = 512;   // tokens of a stage; tiles of 128 that fill the device
    WeightGradPlan p = {};
    const double work = (double)R * (double)T * (double)K * (double)H;
    if (H >= 1024 && H % 8 == 0 && work >= 1.5e10)
        p.value_bytes = ((size_t)R * (size_t)T * (size_t)K * 2 + 255) / 256 * 256;
    const long long stages = (T - 1) / kStage + 1;
    const long long tiles = R * tile_count(H, kMiddleTile) * tile_count(K, kMiddleTile);
    // at least 8 stages to a split: a part costs a write and a read of the outputs
    long long split = tiles < kFill / 2 ? kFill / tiles : 1;
    if (split > stages / 8) split = stages / 8;
    if (split < 1) split = 1;
    const long long run = (stages + split - 1) / split;
    p.split_k = (int)(run * kStage < T ? run * kStage : T);
    p.split = (int)((T - 1) / (run * kStage) + 1);
    if (p.split > 1) p.part_bytes = (size_t)p.split * (size_t)R * (size_t)H * (size_t)K * 4;
    return p;
}

}  // namespace fc
