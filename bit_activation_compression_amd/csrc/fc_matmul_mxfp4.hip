// Linear layer on MXFP4 operands (include/fc/layer.h): y[r] = a[r] w[r]^T on
// the scaled matrix cores, v_mfma_scale_f32_32x32x64_f8f6f4 with both operands
// FP4. Lane l holds row l % 32 of its operand at k = 32 (l / 32) + 0..31: 16
// bytes of codes and one scale byte, which is one block of the format. An
// accumulator holds rows 8 (v / 4) + 4 (l / 32) + v % 4 of column l % 32.
//
// Work layout:
//   - a workgroup owns a BH (channels) x BT (tokens) tile of one rank's
//     output, its WH x WT waves (BH / WH) x (BT / WT) each, in 32 x 32 blocks;
//   - K is walked in stages of 256: 128 bytes of codes (a whole line) and 8 of
//     scales a row. NB stages are held in LDS, filled straight from global
//     memory (buffer_load ... lds) as soon as a buffer is free. The eight
//     16-byte chunks of a row are rotated by (row / 2) % 8, so that a fragment
//     read (32 rows x one chunk) is free of bank conflicts;
//   - the scales are fetched 16 bytes a row at a time, for 2 stages: a load of
//     8 bytes a row touches as many lines for half the use, and that way the
//     scales cost the cache more accesses than the codes (70B d_proj slices
//     1.08 -> 1.03 ms). A stage's scales are read from LDS 8 bytes a row at a time:
//     at a stride of 16, words would take four bank passes each (1.03 -> 1.02);
//   - a stage is 4 matrix-core steps of k = 64. Step ks takes blocks 2 ks (lanes
//     0..31) and 2 ks + 1 (lanes 32..63) of each row: the scale words of a row
//     (one for steps 0 and 1, one for 2 and 3) are shifted right by a byte in
//     the upper lanes, and the instruction's byte selection picks byte 0 or 2;
//   - small tiles read a stage's fragments from LDS while they multiply the
//     stage before (their few matrix instructions would not cover the latency
//     of reads a step ahead); large ones, short of registers, read a step ahead;
//   - y is written in whole lines: for tiles of 128 and 256 the rows are tokens and
//     the columns channels, NH i + nb in column i of the NH blocks nb of a wave's
//     channels (w is staged in that order), so that a lane has NH consecutive
//     channels of a token and 32 lanes 64 NH bytes of it. With channels as rows,
//     where a store has 32 bytes of each of 32 tokens, 70B o_proj slices take 338 us
//     for 297 and 4 x 1024 tokens, K = 3584, H = 4096 39 for 36. Outputs of 128 MiB
//     and more are stored past the caches (321 -> 297). Near that size it is so and so:
//     on operands that the Infinity Cache holds it loses (64 MiB, 2 ranks of 4096 x 4096
//     x 4096, 72.5 -> 75.8; 128 MiB, 8 ranks of 2048 x 1024 x 4096, 49.3 -> 53.7), on
//     others it gains (75.7 -> 75.7; 56.1 -> 53.0). Tiles of 64 have one block: the
//     rows are channels and two lanes have 32 bytes of a token;
//   - rows past H or T lie past the buffer resources and read as zeros. Where K
//     is an odd multiple of 128, the second half of the last stage is not
//     fetched (zeros again) and gets scales of 0;
//   - long calls prefetch into the L2: the workgroups of an XCD that stage the
//     same rows (4 token tiles x 8 channel tiles run at a time) each touch a
//     share of the next two stages' lines, in the place of every other scale
//     load, which has nothing to fetch. Two stages in LDS do not cover the way
//     past the L2: 70B d_proj slices 980 -> 924 us, 8192 x 8192 x 8192 270 ->
//     257. Calls of fewer than 4 tiles per compute unit lose on operands that the
//     Infinity Cache holds (2 ranks of 4096 x 4096 x 4096 76.0 -> 78.6; 1 rank of 8192 x
//     4096 x 4096 72.6 -> 74.6) and gain on others (82.7 -> 77.9; 80.6 -> 77.2);
//   - workgroups are persistent: stages of consecutive tiles form one stream,
//     so the next tile's first stages are in flight during a tile's epilogue.
//     The tiles are split into one contiguous run per XCD (workgroup b runs on
//     XCD b % 8), in groups of 4 token tiles x all channel tiles, so that the
//     workgroups of an XCD share operands in its L2.
//
// What bounds it: the 70B d_proj slices (R = 4, T = 8192, K = 7168, H = 8192)
// take 0.91 to 0.93 ms, 4.1 to 4.2 PFLOP/s. The large tile's matrix instructions alone run at
// 5.3 PFLOP/s with all compute units on random operands (9.8 without the
// toggling: the power management lowers the clock). With everything else the
// clock is 1.6 to 1.7 GHz and the matrix cores are busy 60% of the cycles: a
// stage is 2048 of theirs, and the waves of a workgroup meet once in each. Four
// waves of 128 x 128, which read a third less from LDS, and stages of half the
// length, fetched further ahead, were no faster.
// Small calls are bound by the latency of the fills: about 128 KiB per compute
// unit in flight.
#include <type_traits>

#include "fc_grid.h"
#include "fc_launch.h"
#include "fc_mxfp4.h"
#include "fc_mxfp4_dispatch.h"

namespace fc {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
// stores at the alignment of one output
typedef u32x2 u32x2_u16 __attribute__((aligned(2)));
typedef uint32_t u32_u16 __attribute__((aligned(2)));

constexpr int kStageBytes = 128;          // bytes of codes of a row in a stage
constexpr int kStageScales = 8;           // bytes of scales
constexpr int kStageSteps = 4;
constexpr int kScaleStages = 2;           // stages of one scale load
constexpr int kScaleBytes = kScaleStages * kStageScales;
constexpr int kSink = 1024;               // where the loads land that only keep the count
constexpr int kGroupT = 4;                // token tiles per scheduling group
constexpr uint64_t kPastCache = uint64_t(128) << 20;   // bytes of y
constexpr int kPrefetchTiles = 4;         // tiles per compute unit from which it is done
constexpr int kShareA = 8;                // channel tiles among which a token tile's prefetch is shared
constexpr int kXcds = 8;
constexpr int kLdsBytes = 160 * 1024;     // LDS of a compute unit
constexpr int kNonTemporal = 2;           // cache policy of a buffer store

// SEL: byte of both scale words (0 or 2)
template <int SEL>
__device__ __forceinline__ f32x16 mfma_mx(const u32x4 &w, const u32x4 &a, const f32x16 &c, uint32_t sw,
                                          uint32_t sa) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(w), mx_operand(a), c, kFp4, kFp4, SEL, (int)sw,
                                                           SEL, (int)sa);
}

// s_waitcnt until at most N vector-memory operations of this wave are
// outstanding and all of its LDS operations are done (gfx9 encoding: vmcnt in
// bits 3:0 and 15:14, expcnt left at its maximum, lgkmcnt 0).
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Workgroup barrier that leaves this wave's loads in flight.
__device__ __forceinline__ void barrier_keep_loads() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

struct MxArgs {
    const uint8_t *ac, *as, *wc, *ws;
    uint16_t *y;
    int T, H;
    int stages;                   // of a tile: ceil(Kp / 256)
    uint32_t code_row, scale_row; // bytes of an operand row: Kp / 2, Kp / 32
    int tiles_t, tiles_h;
    uint32_t total;               // tiles of all ranks
    int grid;
    bool prefetch;                // the next stages' lines into the L2
    bool past_cache;              // y is stored past the caches
};

template <int BH, int BT, int WH, int WT, int NB>
struct Shape {
    static constexpr int kRows = BH + BT;
    static constexpr int kLds = NB * kRows * (kStageBytes + kScaleBytes) + kSink;
    static constexpr int kPerCu = kLdsBytes / kLds > 2 ? 2 : kLdsBytes / kLds;
    static_assert(kPerCu >= 1, "");
};

template <int DT, int BH, int BT, int WH, int WT, int NB, bool AHEAD>
__global__ __launch_bounds__(WH *WT * 64) __attribute__((amdgpu_waves_per_eu(2, 2)))
void matmul_mxfp4_kernel(const MxArgs p) {
    constexpr int NW = WH * WT;                    // waves
    constexpr int SH = BH / WH, ST = BT / WT;      // span of a wave
    constexpr int NH = SH / 32, NT = ST / 32;      // its blocks
    constexpr int BR = BH + BT;                    // rows of a stage: w, then a
    constexpr int RW = BR / NW;                    // rows that a wave stages
    constexpr int kCodeLoads = RW / 8, kScaleLoads = RW >= 64 ? RW / 64 : 1;
    constexpr int kLoads = kCodeLoads + kScaleLoads;   // per wave and stage
    constexpr int kCodes = BR * kStageBytes, kScales = BR * kScaleBytes;
    using S = Shape<BH, BT, WH, WT, NB>;
    // with one wave per SIMD (LDS for one workgroup, 4 waves) the compiler keeps
    // the accumulators in the other half of the registers
    constexpr bool kAgprs = NW <= 4 && S::kPerCu == 1;
    constexpr bool kPrefetch = BH * BT >= 256 * 256;   // tiles that many-tile calls use
    constexpr bool kLines = NH > 1;                // outputs in whole lines
    static_assert(!kLines || (RW == 64 && (NH == 2 || NH == 4)), "the staging order and the stores below");
    static_assert((RW == 32 || RW % 64 == 0) && BH % RW == 0, "a wave stages rows of one operand, whole instructions");
    __shared__ __attribute__((aligned(16))) uint8_t lds[S::kLds];
    uint8_t *const lsc = lds + NB * kCodes;
    uint8_t *const sink = lsc + NB * kScales;

    const uint32_t tid = __builtin_amdgcn_workitem_id_x();
    const uint32_t lane = tid & 63u;
    const int wave = __builtin_amdgcn_readfirstlane((int)(tid >> 6));
    const int wh = wave % WH, wt = wave / WH;

    const bool on_w = wave * RW < BH;              // stages rows of w, or of a

    // this XCD's run of tiles, and this workgroup's place in it
    const uint32_t bid = __builtin_amdgcn_workgroup_id_x();
    const uint32_t xcd = bid % kXcds;
    const uint32_t base_wgs = (uint32_t)p.grid / kXcds, more_wgs = (uint32_t)p.grid % kXcds;
    const uint32_t before = xcd * base_wgs + (xcd < more_wgs ? xcd : more_wgs);
    const uint32_t wgs = base_wgs + (xcd < more_wgs ? 1u : 0u);
    const uint32_t first = (uint32_t)((uint64_t)p.total * before / (uint32_t)p.grid);
    const uint32_t last = (uint32_t)((uint64_t)p.total * (before + wgs) / (uint32_t)p.grid);

    struct Tile {
        uint32_t r, h0, t0;
        uint32_t share;           // this wave's among the workgroups that stage the same rows
    };
    auto tile_at = [&](uint32_t it, Tile &t) -> bool {
        const uint32_t logical = first + it * wgs + bid / kXcds;
        if (logical >= last) return false;
        const uint32_t per_rank = (uint32_t)p.tiles_t * (uint32_t)p.tiles_h;
        t.r = logical / per_rank;
        const uint32_t i = logical - t.r * per_rank;
        const uint32_t in_full = kGroupT * (uint32_t)p.tiles_h;
        const uint32_t grp = i / in_full, in_grp = i - grp * in_full;
        const uint32_t left = (uint32_t)p.tiles_t - grp * kGroupT;
        const uint32_t gsize = left < kGroupT ? left : kGroupT;
        t.t0 = (grp * kGroupT + in_grp % gsize) * BT;
        t.h0 = in_grp / gsize * BH;
        t.share = on_w ? in_grp % gsize : in_grp / gsize % kShareA;
        return true;
    };

    // --- staging: the load cursor ---
    struct Source {
        const uint8_t *codes, *scales;     // first row that this wave stages
        uint32_t code_bytes, scale_bytes;  // up to the operand's last row
    };
    auto source_of = [&](const Tile &t) {
        const uint32_t n = on_w ? (uint32_t)p.H : (uint32_t)p.T;           // rows of a rank
        const uint32_t span = kLines && on_w ? SH : RW;                    // of rows that it may stage
        const uint32_t r0 = on_w ? t.h0 + (kLines ? wave * RW / SH * SH : wave * RW) : t.t0 + (wave * RW - BH);
        const uint64_t g = (uint64_t)t.r * n + (r0 < n ? r0 : 0u);
        const uint32_t rows = r0 < n ? (n - r0 < span ? n - r0 : span) : 0u;
        Source s;
        s.codes = (on_w ? p.wc : p.ac) + g * p.code_row;
        s.scales = (on_w ? p.ws : p.as) + g * p.scale_row;
        s.code_bytes = rows * p.code_row;
        s.scale_bytes = rows * p.scale_row;
        return s;
    };
    uint32_t lt = 0;          // tile and stage that the next loads fetch
    int ls = 0;
    uint32_t lbuf = 0, lslot = 0;
    Tile cur;
    if (!tile_at(0, cur)) return;
    Source src = source_of(cur);
    uint32_t share = cur.share;
    const bool odd_k = p.code_row % kStageBytes != 0;

    // Loads [from, to) of the cursor's stage: a code load covers 8 rows x 8
    // chunks, a scale load 64 rows (or the wave's 32). A stage that shares the
    // scales of the one before loads into the sink instead (the number of loads
    // in flight stays fixed): nothing, or a prefetch, 16 bytes of each line of
    // the wave's share of its rows, two stages of them. The whole offset is a lane's (the
    // resource's bounds check covers it), recomputed for every call (`fresh`)
    // so that none of it is live across the epilogue.
    auto load_part = [&](int from, int to) {
        const __amdgpu_buffer_rsrc_t cres = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(src.codes), (short)0, (int)src.code_bytes, kRawBufferFlags);
        const bool real = ls % kScaleStages == 0, tail = odd_k && ls + 1 == p.stages;
        const bool ahead = kPrefetch && p.prefetch && !real;
        const __amdgpu_buffer_rsrc_t sres = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(ahead ? src.codes : src.scales), (short)0,
            (int)(ahead ? src.code_bytes : src.scale_bytes), kRawBufferFlags);
        uint8_t *lc = lds + lbuf * kCodes + (uint32_t)wave * (RW * kStageBytes);
        uint8_t *lw = real ? lsc + lslot * kScales + (uint32_t)wave * (RW * kScaleBytes) : sink;
        const uint32_t l = fresh(lane);
        const uint32_t ch = (l & 7u) ^ (l >> 4);      // the chunk of even loads; odd ones take ch ^ 4
        // rows are staged in order, but those of w with kLines: LDS row 32 nb + i of
        // a span of SH is row NH i + nb of it
        const bool spread = kLines && on_w;
        const uint32_t step = spread ? NH : 1u, nb0 = spread ? (uint32_t)wave * RW % SH / 32u : 0u;
        const uint32_t co = ((l >> 3) * step + nb0) * p.code_row + (uint32_t)ls * kStageBytes;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (j < from || j >= to) continue;
            if (j < kCodeLoads) {
                const uint32_t c = ch ^ (4u * (j & 1));
                const uint32_t row = spread ? 8u * NH * (j % 4) + j / 4 : 8u * j;
                const uint32_t vo = tail && c >= 4u ? kPast : co + row * p.code_row + (c << 4);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    cres, (__attribute__((address_space(3))) void *)(lc + j * 1024), 16, vo, 0, 0, 0);
            } else {
                const int i = j - kCodeLoads;
                const uint32_t row = spread ? (l & 31u) * NH + nb0 + (l >> 5) : l + 64u * i;
                uint32_t vo = real ? row * p.scale_row + (uint32_t)ls * kStageScales : kPast;
                if (ahead && i == 0) {
                    const uint32_t of = on_w ? kGroupT : kShareA, rows = (uint32_t)RW / of;
                    const uint32_t st = (uint32_t)ls + 1u + l / rows;
                    if (l < kScaleStages * rows && st < (uint32_t)p.stages)
                        vo = (nb0 * 32u + l % rows * of + share) * p.code_row + st * kStageBytes;
                }
                if (RW >= 64 || l < RW)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        sres, (__attribute__((address_space(3))) void *)(lw + (real ? i * 1024 : 0)), 16, vo, 0, 0, 0);
            }
        }
    };
    // to the next stage of the stream; past the last tile the resources are
    // empty (the loads still count, and fill buffers that nobody reads)
    auto load_advance = [&]() {
        lbuf = lbuf + 1 == NB ? 0 : lbuf + 1;
        if (++ls == p.stages || ls % kScaleStages == 0) lslot = lslot + 1 == NB ? 0 : lslot + 1;
        if (ls == p.stages) {
            ls = 0;
            Tile t;
            if (tile_at(++lt, t)) {
                src = source_of(t);
                share = t.share;
            } else {
                src.code_bytes = src.scale_bytes = 0;
            }
        }
    };

    // --- fragments ---
    // per-lane offsets within a stage, taken afresh for every tile so that none
    // of them is live across the epilogue
    struct Offs {
        uint32_t ch[kStageSteps];   // the row's chunk of step ks
        uint32_t sc, sh;            // its scales, and the shift to this half's byte
    };
    auto offs = [&]() {
        const uint32_t l = fresh(lane);
        Offs o;
#pragma unroll
        for (uint32_t ks = 0; ks < kStageSteps; ++ks)
            o.ch[ks] = (l & 31u) * kStageBytes + (((2u * ks + (l >> 5)) ^ ((l >> 1) & 7u)) << 4);
        o.sc = (l & 31u) * kScaleBytes;
        o.sh = (l >> 5) * 8u;
        return o;
    };
    // fragments of a step and scale words of two, of every block
    struct Frags {
        u32x4 w[NH], a[NT];
    };
    struct Words {
        uint32_t w[NH], a[NT];
    };
    auto frag = [&](Frags &f, const Offs &o, uint32_t buf, int ks, int b) {
        const uint8_t *st = lds + buf * kCodes;
        if (b < NH) f.w[b] = *reinterpret_cast<const u32x4 *>(st + (wh * SH + b * 32) * kStageBytes + o.ch[ks]);
        if (b < NT) f.a[b] = *reinterpret_cast<const u32x4 *>(st + (BH + wt * ST + b * 32) * kStageBytes + o.ch[ks]);
    };
    // both words (of steps 0 and 1, of 2 and 3) of stage q (of a scale load's two)
    // in a slot, as read
    auto words = [&](Words &r0, Words &r1, const Offs &o, uint32_t slot, uint32_t q, int b) {
        const uint8_t *st = lsc + slot * kScales + q * kStageScales;
        if (b < NH) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(st + (wh * SH + b * 32) * kScaleBytes + o.sc);
            r0.w[b] = v.x;
            r1.w[b] = v.y;
        }
        if (b < NT) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(st + (BH + wt * ST + b * 32) * kScaleBytes + o.sc);
            r0.a[b] = v.x;
            r1.a[b] = v.y;
        }
    };
    auto shifted = [&](const Words &r, const Offs &o, bool zero) {
        Words c;
#pragma unroll
        for (int b = 0; b < NH; ++b) c.w[b] = zero ? 0u : r.w[b] >> o.sh;
#pragma unroll
        for (int b = 0; b < NT; ++b) c.a[b] = zero ? 0u : r.a[b] >> o.sh;
        return c;
    };
    constexpr int NF = NH > NT ? NH : NT;
    uint32_t cbuf = 0, cslot = 0;

#pragma unroll
    for (int i = 0; i < NB; ++i) {
        load_part(0, kLoads);
        load_advance();
    }
    wait_loads<(NB - 1) * kLoads>();
    barrier_keep_loads();

    for (uint32_t it = 0;; ++it) {
        f32x16 acc[NH][NT];
#pragma unroll
        for (int a = 0; a < NH; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b) acc[a][b] = f32x16{};
        // The accumulators pass through here: without it the compiler gathers
        // a stage's matrix instructions at its end, with all fragments live.
        auto pin = [&](int nb) {
#pragma unroll
            for (int tb = 0; tb < NT; ++tb) {
                if constexpr (kAgprs) asm volatile("" : "+a"(acc[nb][tb]));
                else asm volatile("" : "+v"(acc[nb][tb]));
            }
        };
        // row nb of a step's blocks
        auto multiply = [&](auto odd_, int nb, const Frags &f, const Words &c) {
            constexpr int kSel = decltype(odd_)::value * 2;
#pragma unroll
            for (int tb = 0; tb < NT; ++tb) {
                if constexpr (kLines) acc[nb][tb] = mfma_mx<kSel>(f.a[tb], f.w[nb], acc[nb][tb], c.a[tb], c.w[nb]);
                else acc[nb][tb] = mfma_mx<kSel>(f.w[nb], f.a[tb], acc[nb][tb], c.w[nb], c.a[tb]);
            }
        };
        constexpr std::integral_constant<int, 0> kEven;
        constexpr std::integral_constant<int, 1> kOdd;
        // from stage s to the next one of the stream
        auto next_buf = [&]() { return cbuf + 1 == NB ? 0u : cbuf + 1; };
        auto next_slot = [&](int s) {
            const bool fresh_slot = s + 1 == p.stages || (s + 1) % kScaleStages == 0;
            return !fresh_slot ? cslot : cslot + 1 == NB ? 0u : cslot + 1;
        };
        auto stage_of_slot = [&](int s) { return s == p.stages ? 0u : (uint32_t)s % kScaleStages; };
        // the wait for the next stage's loads (this wave's; the barrier makes
        // them everybody's); every wave has then also done its reads of this
        // stage, whose buffer can be filled again
        auto next_ready = [&]() {
            wait_loads<(NB - 2) * kLoads>();
            barrier_keep_loads();
        };
        const Offs o = offs();
        if constexpr (AHEAD) {
            struct Stage {
                Frags f[kStageSteps];
                Words r[2];
            } st[2];
            auto read = [&](Stage &x, uint32_t buf, uint32_t slot, uint32_t q) {
#pragma unroll
                for (int ks = 0; ks < kStageSteps; ++ks)
#pragma unroll
                    for (int b = 0; b < NF; ++b) {
                        frag(x.f[ks], o, buf, ks, b);
                        if (ks == 0) words(x.r[0], x.r[1], o, slot, q, b);
                    }
            };
            auto body = [&](Stage &x, Stage &y, int s) {
                next_ready();
                const uint32_t nbuf = next_buf(), nslot = next_slot(s);
                read(y, nbuf, nslot, stage_of_slot(s + 1));
                load_part(0, kLoads);
                load_advance();
                const Words c0 = shifted(x.r[0], o, false), c1 = shifted(x.r[1], o, odd_k && s + 1 == p.stages);
#pragma unroll
                for (int nb = 0; nb < NH; ++nb) {
                    multiply(kEven, nb, x.f[0], c0);
                    multiply(kOdd, nb, x.f[1], c0);
                    multiply(kEven, nb, x.f[2], c1);
                    multiply(kOdd, nb, x.f[3], c1);
                    pin(nb);
                }
                cbuf = nbuf;
                cslot = nslot;
            };
            read(st[0], cbuf, cslot, 0);
            int s = 0;
            for (; s + 1 < p.stages; s += 2) {
                body(st[0], st[1], s);
                body(st[1], st[0], s + 1);
            }
            if (s < p.stages) body(st[0], st[1], s);
        } else {
            // the tile's first fragments (the last step before a tile's epilogue
            // reads them too, but none is live across the epilogue)
            Frags f[2];
            Words r0, r1;
#pragma unroll
            for (int b = 0; b < NF; ++b) {
                frag(f[0], o, cbuf, 0, b);
                words(r0, r1, o, cslot, 0, b);
            }
            // step ks with `side`, the reads and loads that overlap it
            auto step = [&](auto odd_, const Words &c, auto &&side) {
#pragma unroll
                for (int nb = 0; nb < NH; ++nb) {
                    multiply(odd_, nb, f[decltype(odd_)::value], c);
                    side(nb);
                    if (nb == NH - 1)
                        for (int b = NH; b < NF; ++b) side(b);
                    pin(nb);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            auto load_share = [&](int part, int parts) {
                if (part < parts) load_part(part * kLoads / parts, (part + 1) * kLoads / parts);
            };
            for (int s = 0; s < p.stages; ++s) {
                const uint32_t nbuf = next_buf(), nslot = next_slot(s), nq = stage_of_slot(s + 1);
                const Words c0 = shifted(r0, o, false);
                step(kEven, c0, [&](int b) { frag(f[1], o, cbuf, 1, b); });
                step(kOdd, c0, [&](int b) { frag(f[0], o, cbuf, 2, b); });
                const Words c1 = shifted(r1, o, odd_k && s + 1 == p.stages);
                step(kEven, c1, [&](int b) { frag(f[1], o, cbuf, 3, b); });
                next_ready();
                step(kOdd, c1, [&](int b) {
                    frag(f[0], o, nbuf, 0, b);
                    words(r0, r1, o, nslot, nq, b);
                    load_share(b, NH);
                });
                load_advance();
                cbuf = nbuf;
                cslot = nslot;
            }
        }

        if constexpr (kLines) {
            // A lane has NH consecutive channels of a token, 32 lanes whole lines
            // of it; accumulator v is token 8 (v / 4) + 4 (lane / 32) + v % 4.
            uint16_t *const yr = p.y + (uint64_t)cur.r * (uint32_t)p.T * (uint32_t)p.H;
            const uint32_t el = fresh(lane), t0 = cur.t0 + (uint32_t)(wt * ST), h0 = cur.h0 + (uint32_t)(wh * SH);
            const uint32_t lt0 = (el >> 5) * 4u, lh0 = (el & 31u) * NH;
            auto token = [](int tb, int v) { return (uint32_t)(tb * 32 + v / 4 * 8 + v % 4); };
            auto pair = [&](int tb, int v, int k) { return mx_round2<DT>(acc[2 * k][tb][v], acc[2 * k + 1][tb][v]); };
            if (p.H % 2 == 0 && h0 + SH <= (uint32_t)p.H) {
                const uint32_t rows = t0 < (uint32_t)p.T ? ((uint32_t)p.T - t0 < ST ? (uint32_t)p.T - t0 : ST) : 0u;
                const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
                    yr + (uint64_t)(rows ? t0 : 0u) * (uint32_t)p.H + h0, (short)0,
                    rows ? (int)((rows * (uint32_t)p.H - h0) * 2u) : 0, kRawBufferFlags);
                const uint32_t row_bytes = (uint32_t)p.H * 2u;
                const uint32_t off = lt0 * row_bytes + lh0 * 2u;
                auto store = [&](auto aux_) {
                    constexpr int kAux = decltype(aux_)::value;
#pragma unroll
                    for (int tb = 0; tb < NT; ++tb)
#pragma unroll
                        for (int v = 0; v < 16; ++v) {
                            const int o = (int)(off + token(tb, v) * row_bytes);
                            if constexpr (NH == 4)
                                __builtin_amdgcn_raw_buffer_store_b64(u32x2{pair(tb, v, 0), pair(tb, v, 1)}, res, o, 0, kAux);
                            else
                                __builtin_amdgcn_raw_buffer_store_b32(pair(tb, v, 0), res, o, 0, kAux);
                        }
                };
                if (p.past_cache) store(std::integral_constant<int, kNonTemporal>{});
                else store(std::integral_constant<int, 0>{});
            } else {
#pragma unroll
                for (int tb = 0; tb < NT; ++tb)
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const uint32_t t = t0 + lt0 + token(tb, v), h = h0 + lh0;
                        uint32_t w[NH / 2];
#pragma unroll
                        for (int k = 0; k < NH / 2; ++k) w[k] = pair(tb, v, k);
                        if (t >= (uint32_t)p.T) continue;
                        uint16_t *yt = yr + (uint64_t)t * (uint32_t)p.H;
                        if (h + NH <= (uint32_t)p.H) {
                            if constexpr (NH == 4) *reinterpret_cast<u32x2_u16 *>(yt + h) = u32x2{w[0], w[1]};
                            else *reinterpret_cast<u32_u16 *>(yt + h) = w[0];
                        } else {
#pragma unroll
                            for (uint32_t k = 0; k < NH; ++k)
                                if (h + k < (uint32_t)p.H) yt[h + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
                        }
                    }
            }
        } else {
            // groups 2 q and 2 q + 1 of 4 channels, swapped between the
            // halves of the wave, give each lane 8 consecutive channels of a token
            const uint32_t el = fresh(lane), row = el & 31u, half = el >> 5;
            uint16_t *const yr = p.y + (uint64_t)cur.r * (uint32_t)p.T * (uint32_t)p.H;
#pragma unroll
            for (int tb = 0; tb < NT; ++tb) {
                const uint32_t t = cur.t0 + (uint32_t)(wt * ST + tb * 32) + row;
                uint16_t *yt = yr + (uint64_t)t * (uint32_t)p.H;
#pragma unroll
                for (int nb = 0; nb < NH; ++nb) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const f32x16 &v = acc[nb][tb];
                        uint32_t a0 = mx_round2<DT>(v[8 * q + 0], v[8 * q + 1]), a1 = mx_round2<DT>(v[8 * q + 2], v[8 * q + 3]);
                        uint32_t b0 = mx_round2<DT>(v[8 * q + 4], v[8 * q + 5]), b1 = mx_round2<DT>(v[8 * q + 6], v[8 * q + 7]);
                        const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
                        const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
                        const uint32_t w[4] = {(uint32_t)s0[0], (uint32_t)s1[0], (uint32_t)s0[1], (uint32_t)s1[1]};
                        const uint32_t h = cur.h0 + (uint32_t)(wh * SH + nb * 32 + q * 16) + half * 8u;
                        if (t < (uint32_t)p.T) {
                            if (h + 8u <= (uint32_t)p.H) {
                                *reinterpret_cast<u32x4_u16 *>(yt + h) = u32x4{w[0], w[1], w[2], w[3]};
                            } else {
#pragma unroll
                                for (uint32_t k = 0; k < 8; ++k)
                                    if (h + k < (uint32_t)p.H) yt[h + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
                            }
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        if (!tile_at(it + 1, cur)) break;
    }
    wait_loads<0>();   // nothing may land in LDS after the workgroup has ended
}

template <int DT, int BH, int BT, int WH, int WT, int NB, bool AHEAD>
hipError_t launch_tiles(MxArgs p, int R, int cus, hipStream_t stream) {
    constexpr int per_cu = Shape<BH, BT, WH, WT, NB>::kPerCu;
    p.tiles_t = mxfp4_tiles(p.T, BT);
    p.tiles_h = mxfp4_tiles(p.H, BH);
    const uint64_t total = (uint64_t)R * (uint64_t)p.tiles_t * (uint64_t)p.tiles_h;
    if (total > 0x7FFFFFFFull) return hipErrorInvalidConfiguration;
    p.total = (uint32_t)total;
    p.past_cache = (uint64_t)R * (uint64_t)p.T * (uint64_t)p.H * 2 >= kPastCache;
    p.prefetch = total >= (uint64_t)cus * kPrefetchTiles;
    p.grid = (int)(total < (uint64_t)cus * per_cu ? total : (uint64_t)cus * per_cu);
    hipLaunchKernelGGL((matmul_mxfp4_kernel<DT, BH, BT, WH, WT, NB, AHEAD>), dim3((unsigned)p.grid),
                       dim3(WH * WT * 64), 0, stream, p);
    return hipGetLastError();
}

template <int DT>
hipError_t by_shape(const MxArgs &p, int R, int cus, hipStream_t stream) {
    switch (mxfp4_tile(R, p.T, p.H, cus)) {
    case Mxfp4Tile::k256: return launch_tiles<DT, 256, 256, 2, 4, 2, false>(p, R, cus, stream);
    case Mxfp4Tile::k128: return launch_tiles<DT, 128, 128, 2, 2, 4, false>(p, R, cus, stream);
    case Mxfp4Tile::k64: return launch_tiles<DT, 64, 64, 2, 2, 4, true>(p, R, cus, stream);
    }
    return hipErrorInvalidConfiguration;
}

}  // namespace

hipError_t launch_matmul_mxfp4(const uint8_t *a_codes, const uint8_t *a_scales,
                               const uint8_t *w_codes, const uint8_t *w_scales, int R, int T, int Kp,
                               int H, int dtype, uint16_t *y, hipStream_t stream) {
    const int cus = compute_units();
    if (cus <= 0) return hipErrorInvalidDevice;
    if (mxfp4_few_tokens(R, T, Kp / kMxStepElems, H, cus))
        return launch_matmul_mxfp4_few(a_codes, a_scales, w_codes, w_scales, R, T, Kp, H, dtype, y, stream);
    MxArgs p = {};
    p.ac = a_codes;
    p.as = a_scales;
    p.wc = w_codes;
    p.ws = w_scales;
    p.y = y;
    p.T = T;
    p.H = H;
    p.stages = (Kp / kMxStepElems + 1) / 2;
    p.code_row = (uint32_t)Kp / 2;
    p.scale_row = (uint32_t)Kp / kMxBlockElems;
    return dtype == 0 ? by_shape<0>(p, R, cus, stream) : by_shape<1>(p, R, cus, stream);
}

}  // namespace fc
