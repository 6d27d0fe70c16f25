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
// worth it: one, or two of long rows. us split / unsplit / tiles of 64 (fc_matmul_mxfp4,
// 1 token, 1 rank, bf16; K, H): 4096, 4096 5.4 / 9.3 / 9.1; 4096, 8192 9.3 / 9.5 /
// 9.5; 8192, 8192 11.0 / 15.2 / 15.4; 1024, 8192 7.1 / 5.2 / 5.0; 4096, 14336 15.8 /
// 9.9 / 10.0. 0: not worth it (or no device).
inline int mxfp4_split_rounds(int R, int H, int steps, int cus) {
    const int64_t groups = (int64_t)R * mxfp4_tiles(H, 16);
    if (groups <= cus) return 1;
    return groups <= 2 * (int64_t)cus && steps >= kMxfp4LongSteps ? 2 : 0;
}

// Up to 32 tokens in one round of 16 channels of all ranks per compute unit, up to 64
// of long rows; up to 4 in two rounds of long rows, up to 16 of rows twice as long.
// More would fill the device with tiles. us against tiles (of 64), bf16, in a graph on
// operands from HBM; R, T, K, H: 1, 16, 512, 4096 4.6 / 4.3; 1, 32, 1024, 4096 4.5 / 5.0;
// 1, 33, 1024, 4096 5.9 / 5.1; 1, 16, 4096, 4096 6.2 / 9.1; 1, 48, 4096, 4096 8.7 / 9.3;
// 1, 64, 4096, 4096 9.7 / 9.4; 1, 64, 14336, 1024 22.2 / 23.1; in two rounds 1, 1, 4096, 4200
// 8.4 / 9.1; 1, 1, 4096, 8192 9.6 / 9.6; 1, 8, 4096, 6144 9.7 / 9.4; 1, 16, 8192, 8192 14.6 /
// 15.5; 1, 24, 8192, 8192 17.3 / 15.8; 2, 16, 14336, 4096 21.7 / 24.0.
inline bool mxfp4_few_tokens(int R, int T, int steps, int H, int cus) {
    const int rounds = mxfp4_split_rounds(R, H, steps, cus);
    if (rounds == 1) return T <= (steps >= kMxfp4LongSteps ? 64 : 32);
    return rounds == 2 && T <= (steps >= 2 * kMxfp4LongSteps ? 16 : 4);
}

inline bool mxfp4_quantizes_in_place(int T, int Kp) {
    return T <= 16 && (int64_t)T * Kp <= kMxfp4QuantizeMost;
}

// --- tiles (fc_matmul_mxfp4.hip) ---

enum class Mxfp4Tile { k256, k128, k64 };

// Rounds of tiles over the compute units decide: larger tiles move fewer bytes
// per product, smaller ones waste less of the last round. A round of 256 tiles
// takes twice one of 128; up to two tiles of 64 per unit take less than a round
// of 128, and up to five less than two. At most 64 tokens take tiles of 64.
// us with tiles of 64 / 128 / 256 (bf16, in a graph on operands from HBM; a tenth
// or so less from the Infinity Cache; R, T, K, H):
//   2, 160, 4096, 5120: 16.5 / 17.2 / 33.3      1, 640, 4096, 4096: 18.5 / 16.1 / 27.2
//   1, 1408, 4096, 3200: 27.3 / 28.9 / 32.9     3, 256, 4096, 7168: 40.8 / 32.8 / 37.2
//   2, 1024, 4096, 4096: 49.6 / 33.0 / 37.3     1, 2176, 4096, 4096: 50.7 / 43.3 / 36.4
//   2, 520, 3584, 6144: 38.6 / 28.6 / 32.6      1, 4352, 4096, 4096: 88.3 / 69.0 / 62.5
//   4, 128, 2048, 8192: 19.4 / 15.7 / 22.4      4, 8192, 7168, 8192: 2269 / 1429 / 936
// (Twice the stages in LDS for calls of at most one tile of 64 per unit, which then
// do not fit two to a unit, took 0.8 to 2 us longer on each of 16 such shapes: 1, 256,
// 4096, 4096 11.3 against 10.2, 1, 300, 512, 512 5.0 against 4.1.)
inline Mxfp4Tile mxfp4_tile(int R, int T, int H, int cus) {
    const uint64_t n = (uint64_t)cus;
    auto tiles = [&](int b) { return (uint64_t)R * (uint64_t)mxfp4_tiles(T, b) * (uint64_t)mxfp4_tiles(H, b); };
    auto rounds = [&](int b) { return (tiles(b) + n - 1) / n; };
    if (T > 64) {
        if (2 * rounds(256) < rounds(128)) return Mxfp4Tile::k256;
        if (tiles(64) > n * (rounds(128) == 2 ? 5 : 2)) return Mxfp4Tile::k128;
    }
    return Mxfp4Tile::k64;
}

}  // namespace fc
