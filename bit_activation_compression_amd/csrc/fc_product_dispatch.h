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

// Cost of `tiles` tiles in units of a round of tiles of 256, one on every compute unit
// (K = 4096 bf16: 115 us). A compute unit holds one workgroup of 256, two of 128 or of 64
// (four stages in LDS); alone on it, or with half of the device idle, they are faster.
// Measured without the L2 prefetch of linear layers, us at K = N = 4096 and 64 / 512 / 768 / 1024 / 1536 / 2048 / 4096 rows: tiles of
// 64 25 / 32 / 53 / 68 / 94 / 130 / 245, of 128 54 / 54 / 58 / 72 / 75 / 81 / 158, of 256
// 86 / 88 / 97 / 108 / 112 / 112 / 115. The ratios stand for every K; all in tiles of 64 / 128 /
// 256, 8192 rows: N = 4096, K = 64 58 / 39 / 36, K = 320 85 / 58 / 51, K = 1024 158 / 106 / 82,
// K = 8192 929 / 587 / 432; N = 7168 (the rule has two parts), K = 64 101 / 65 / 68 and 66, K =
// 320 144 / 95 / 96 and 92.
inline double tile_cost(long long tiles, int tile, int cus) {
    const double one = tile == kLargeTile ? 0.75 : tile == kMiddleTile ? 0.47 : 0.22;    // half a round or less
    const double full = tile == kLargeTile ? 1.0 : tile == kMiddleTile ? 0.69 : 0.275;   // a round
    const long long round = tile == kLargeTile ? cus : 2 * cus;
    const long long rounds = tiles / round, rest = tiles % round;
    if (rest == 0) return (double)rounds * full;
    const double part = 2.0 * (double)rest / (double)round - 1.0;   // beyond half a round
    return (double)rounds * full + one + (part > 0.0 ? part * (full - one) : 0.0);
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

// A sum over K in `split` runs of split_k (whole stages), none of them empty.
struct SplitPlan {
    int split, split_k;
};

inline SplitPlan split_runs(long long K, long long want) {
    constexpr long long kStage = 64;
    const long long stages = (K - 1) / kStage + 1;
    // at least 8 stages to a run: a run costs a write and a read of the outputs
    long long split = want < stages / 8 ? want : stages / 8;
    if (split < 1) split = 1;
    const long long run = (stages + split - 1) / split * kStage;
    SplitPlan p;
    p.split_k = (int)(run < K ? run : K);
    p.split = (int)((K - 1) / run + 1);
    return p;
}

// Linear layers and input gradients of few outputs: sums over K are split where the
// tiles of 64 would leave compute units idle. It goes by the sizes alone, so that the
// workspace (binary32 [split][batches][M][N]) is the same on every device. us in one run and
// as split here, N = 4096, K = 1024 / 1536 / 2048 / 4096: 64 rows 9.5 / 12.1 / 14.8 / 24.9 and
// 10.5 / 10.6 / 11.6 / 14.6, 128 rows 9.6 / 12.1 / 14.7 / 25.0 and 10.5 / 14.1 / 15.3 / 16.0, 256
// rows (all of kFill / 2 tiles) 9.7 / 12.3 / 15.0 / 25.3 and 13.4 / 15.4 / 16.8 / 22.9; from
// there on whole runs are as fast or faster (320 rows, K = 4096 31.5, in two runs 32.4). So
// sums of 64 stages gain 2 to 10 us, and those of 16 to 32 stages lose 1 to 4 from 128 tiles on.
inline SplitPlan linear_plan(long long batches, int M, int N, int K) {
    constexpr long long kFill = 512;   // tiles of 64 that fill 256 compute units, two on each
    const long long tiles = batches * tile_count(M, kSmallTile) * tile_count(N, kSmallTile);
    return split_runs(K, tiles <= kFill / 2 ? kFill / tiles : 1);
}

// How a weight gradient of R x H x K sums over T tokens runs, by the sizes alone too.
// Codes that many rows of tiles would each turn into values are turned into them once,
// before the product; us with the codes read by the product against values first, T x K x
// H: 8192 x 4096 x 512 92 against 80, 2048 x 4096 x 1024 61 against 43, 256 x 4096 x 4096
// 32 against 25, four ranks of 512 x 1024 x 1024 20 against 17; 1024^3 16 against 16, 16 x
// 4096 x 4096 18 against 19; few rows of tiles: 8192 x 4096 x 64 26 against 47, 65536 x 256
// x 256 37 against 42.
struct WeightGradPlan {
    size_t value_bytes;   // of the activations as 16-bit values, 0: codes are read by the product
    size_t part_bytes;    // of the splits' sums (after the values), 0: one split
    SplitPlan split;
};

inline WeightGradPlan weight_grad_plan(int R, int T, int K, int H) {
    constexpr long long kFill = 512;   // tiles of 128 that fill 256 compute units, two on each
    WeightGradPlan p = {};
    const double work = (double)R * (double)T * (double)K * (double)H;
    if (H >= 512 && H % 8 == 0 && work >= 1e9)
        p.value_bytes = ((size_t)R * (size_t)T * (size_t)K * 2 + 255) / 256 * 256;
    const long long tiles = R * tile_count(H, kMiddleTile) * tile_count(K, kMiddleTile);
    p.split = split_runs(T, tiles < kFill / 2 ? kFill / tiles : 1);
    if (p.split.split > 1) p.part_bytes = (size_t)p.split.split * (size_t)R * (size_t)H * (size_t)K * 4;
    return p;
}

// Tokens up to which a linear layer runs without LDS stages, its weights streamed
// through the registers (fc_linear_act.hip); us at 1 / 4 / 8 / 16 tokens, streamed against
// tiles: K = 8192, H = 7168 27 / 30 / 33 / 37 against 33 / 33 / 33 / 32; four ranks of
// K = 2048, H = 8192 28 / 30 / 33 / 40 against 32 / 32 / 32 / 33.
constexpr int kFewTokens = 8;

}  // namespace fc
