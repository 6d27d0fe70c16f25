// Which kernel a product of MXFP4 operands (include/fc/layer.h) takes: plain
// C++, no HIP runtime calls, so that the rules can be checked on a host.
// `cus` is the device's compute units.
#pragma once

#include <stdint.h>

namespace fc {

// Workgroups or tiles of b that n elements (up to 2^31 - 1) take.
inline int mxfp4_tiles(int n, int b) { return (int)(((unsigned)n + (unsigned)b - 1u) / (unsigned)b); }

// --- few tokens (fc_matmul_mxfp4_few.hip) ---

// Most activations of a rank that the kernel quantizes itself, which saves the
// quantizer's launch: 4 ranks, K = 2048, H = 8192, bf16, 4 / 6 / 8 tokens 9.5 /
// 10.5 / 11.0 us against 12.1 / 12.3 / 12.3 with it; twice as many are no faster.
constexpr int kMxfp4QuantizeMost = 16384;
constexpr int kMxfp4LongSteps = 32;       // of k = 128, see mxfp4_split_rounds

// Rounds of workgroups over the compute units with split waves, where those are
// worth it: one, or two of long rows. us split / unsplit / tiles (fc_matmul_mxfp4,
// 1 token, 1 rank, bf16; K, H): 4096, 4096 5.4 / 9.3 / 10.1; 4096, 8192 9.3 / 9.5 /
// 10.5; 8192, 8192 11.0 / 15.2 / 16.3; 1024, 8192 7.1 / 5.2 / 5.9; 4096, 14336 15.8 /
// 9.9 / 11.1. 0: not worth it (or no device).
inline int mxfp4_split_rounds(int R, int H, int steps, int cus) {
    const int64_t groups = (int64_t)R * mxfp4_tiles(H, 16);
    if (groups <= cus) return 1;
    return groups <= 2 * (int64_t)cus && steps >= kMxfp4LongSteps ? 2 : 0;
}

// Up to 64 tokens in one round of 16 channels of all ranks per compute unit, up to
// 24 in two of long rows; more would fill the device with tiles. us against tiles,
// bf16; R, T, K, H: 1, 16, 4096, 4096 6.4 / 10.1; 1, 64, 4096, 4096 10.0 / 10.4; 1, 64,
// 4096, 6144 17.0 / 11.2; 1, 17, 8192, 8192 14.5 / 16.3; 1, 32, 8192, 8192 18.0 / 16.5.
inline bool mxfp4_few_tokens(int R, int T, int steps, int H, int cus) {
    const int rounds = mxfp4_split_rounds(R, H, steps, cus);
    return rounds == 1 ? T <= 64 : rounds == 2 && T <= 24;
}

inline bool mxfp4_quantizes_in_place(int T, int Kp) {
    return T <= 16 && (int64_t)T * Kp <= kMxfp4QuantizeMost;
}

// --- tiles (fc_matmul_mxfp4.hip) ---

enum class Mxfp4Tile { k256, k128, k64, k64Deep };

// Rounds of tiles over the compute units decide: larger tiles move fewer bytes
// per product, smaller ones waste less of the last round. A round of 256 tiles
// takes twice one of 128; up to two tiles of 64 per unit take less than a round
// of 128, and up to five less than two. At most 64 tokens take tiles of 64.
// Measured, us with tiles of 64 / 128 / 256 (bf16; R, T, K, H):
//   2, 160, 4096, 5120: 14.2 / 16.9 / 27.3      1, 640, 4096, 4096: 19.4 / 16.9 / 27.9
//   1, 1408, 4096, 3200: 26.3 / 28.9 / 30.2     3, 256, 4096, 7168: 32.3 / 28.2 / 28.9
//   2, 1024, 4096, 4096: 42.7 / 30.2 / 30.8     1, 2176, 4096, 4096: 45.2 / 42.6 / 30.5
//   2, 520, 3584, 6144: 32.9 / 27.3 / 27.7      1, 4352, 4096, 4096: 86.4 / 67.1 / 59.0
//   4, 128, 2048, 8192: 16.1 / 13.8 / 19.8      4, 8192, 7168, 8192: 2111 / 1378 / 913
// At most one tile of 64 per unit leaves the LDS for twice the stages (8 against 4:
// 1, 256, 4096, 4096 11.6 against 12.1).
inline Mxfp4Tile mxfp4_tile(int R, int T, int H, int cus) {
    const uint64_t n = (uint64_t)cus;
    auto tiles = [&](int b) { return (uint64_t)R * (uint64_t)mxfp4_tiles(T, b) * (uint64_t)mxfp4_tiles(H, b); };
    auto rounds = [&](int b) { return (tiles(b) + n - 1) / n; };
    if (T > 64) {
        if (2 * rounds(256) < rounds(128)) return Mxfp4Tile::k256;
        if (tiles(64) > n * (rounds(128) == 2 ? 5 : 2)) return Mxfp4Tile::k128;
    }
    return tiles(64) <= n ? Mxfp4Tile::k64Deep : Mxfp4Tile::k64;
}

}  // namespace fc
