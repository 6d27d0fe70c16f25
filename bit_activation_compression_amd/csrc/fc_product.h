// Matrix products on the matrix cores with 16-bit operands and binary32 sums:
//
//   out[r][m][n] = sum_k A[r](m, k) * B[r](n, k)
//
// for the linear layer (A = activations, B = weights), its input gradient (A = dy,
// B = weights read down their columns) and its weight gradient (A = dy and B = the
// saved activations, both read down their columns; B as an INT8 payload).
//
// An operand lies in memory with its k side by side (kRows: [m][k]) or with its m (n)
// side by side (kCols: [k][m]; kCodes: [k][m] INT8 codes with scales and zeros).
// Tiles of TM x TN outputs, stages of 64 k in LDS:
//   - kRows: 64 k of a row are 128 bytes; its eight 16-byte chunks are rotated by
//     (row / 2) % 8, so that the fragment reads (ds_read_b128: 16 rows x one chunk
//     per 16 lanes) meet each bank once;
//   - kCols, kCodes: a stage is 64 rows of TM values; fragments are read with the
//     transposing ds_read_b64_tr_b16 (16 lanes read 4 rows x 16 values and get 4 k
//     of one column each). A half wave reads 32 bytes of 8 rows: their 32-byte
//     units are swapped by k % 4 and bit 3 of k, so that these meet each bank once.
// 16-bit operands whose rows are whole 16-byte chunks go to LDS straight from
// memory (buffer_load ... lds), the rotation done by which chunk a lane fetches;
// others, and codes, go through registers: loads before a stage's products, stores
// to LDS after them.
//
// Measured (bf16, call by call in turn with a library's product of the same operands, medians
// of 60, most within 4%): linear layer of 8192^3 867 us against 689, of 8192 x 8192 x 7168 782
// against 631 (1.23 and 1.52 PFLOP/s), with bias, GELU and z kept 815 against 688 for a product
// with bias and a GELU of its own; input gradient 782 against 691; weight gradient from codes
// to binary32 849, 36 of it for the values, against 970 from 16-bit values to 16-bit ones. The
// matrix cores are busy 61 to 62% of the cycles of a launch of tiles of 256. 32 x 32 x 16
// instructions ran 8192^3 in 864 us against 834; four waves of 128 x 128 spill (0.72
// PFLOP/s). The loads to LDS are inline asm: behind the builtin the compiler waits for all
// of them before a transposing read (8192^3 input gradient 1061 us against 885 at the time).
//
// v_mfma_f32_16x16x32: lane l holds row (column) l % 16 and k 8 (l / 16) + 0..7 of an
// operand, and of the result column l % 16 and rows 4 (l / 16) + 0..3.
#pragma once

#include "fc_act.h"
#include "fc_grid.h"
#include "fc_launch_train.h"
#include "fc_product_dispatch.h"
#include "fc_rows.h"

namespace fc {
namespace {

constexpr int kRows = 0, kCols = 1, kCodes = 2;
constexpr int kStageK = 64;
constexpr int kBlock = 16, kStepK = 32;         // of a matrix instruction
constexpr int kChunk = 8;                      // values of a 16-byte chunk
constexpr uint32_t kOutside = 0xFFFFFFF0u;     // an offset past every buffer
constexpr uint32_t kRawBuffer = 0x00020000;         // resource word 3: raw 32-bit buffer

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

#define FC_LDS __attribute__((address_space(3)))

template <int DT>
__device__ __forceinline__ f32x4 mfma(const u32x4 &a, const u32x4 &b, const f32x4 &c) {
    if constexpr (DT == 1)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Wait until at most N vector-memory operations of this wave are outstanding and
// its LDS operations are done.
template <int N>
__device__ __forceinline__ void wait_memory() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// A workgroup barrier that leaves loads in flight.
__device__ __forceinline__ void meet() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// 16 bytes per lane from offset base + off of a buffer (zeros past its end) to LDS at `to` + 16 * lane. The
// instruction has no result register; whoever reads the LDS waits with wait_memory.
// (The builtin for it would have the compiler wait for all such loads before every
// transposing LDS read.) A write of M0 needs a wait state before its use, a resource
// written by a vector instruction five.
// The range check takes `base` into account: what lies past the buffer's end with it,
// however far, reads as zeros.
__device__ __forceinline__ void load_to_lds(const u32x4 &res, uint8_t FC_LDS *to, uint32_t off, uint32_t base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"((uint32_t)(uintptr_t)to), "v"(off), "s"(res), "s"(base)
                 : "memory", "m0");
}

// A dword per lane to LDS the same way.
__device__ __forceinline__ void touch_to_lds(const u32x4 &res, uint8_t FC_LDS *to, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"((uint32_t)(uintptr_t)to), "v"(off), "s"(res)
                 : "memory", "m0");
}

struct ProductArgs {
    const uint16_t *a, *b;
    Payload pb;             // B of kCodes
    int group;
    int R, M, N, K;         // per rank
    int from_m, from_n;     // the tiles cover rows [from_m, to_m) and columns [from_n, to_n)
    int to_m, to_n;
    int tiles_m, tiles_n;   // (these and total: set by the launcher)
    uint64_t total;         // tiles of all ranks and splits
    int split, split_k;     // k in `split` runs of split_k (a multiple of the stage)
    LinearEpilogue e;       // 16-bit results
    float *out;             // binary32 results [split][R][M][N]
    int accumulate;
};

template <int TM, int TN, int WM, int WN, int NS>
struct Shape {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
    static constexpr int kSM = TM / WM, kSN = TN / WN;         // of a wave
    static constexpr int kBM = kSM / kBlock, kBN = kSN / kBlock;
    static constexpr int kBytesA = TM * kStageK * 2, kBytesB = TN * kStageK * 2, kStage = kBytesA + kBytesB;
    static constexpr int kRing = NS * kStage;                  // stages in LDS
    // waves that share a SIMD: of the workgroups that fit the LDS, but at most 4
    static constexpr int kGroups = 160 * 1024 / kRing, kPerSimd = kGroups * kWaves / 4 < 4 ? kGroups * kWaves / 4 : 4;
    // the epilogue's rows of a wave: 32 rows of binary32, padded so that the two
    // halves of a wave (4 rows apart) write different banks
    static constexpr int kPitch = kSN + 4;
    static constexpr int kEpilogue = kWaves * 32 * kPitch * 4;
    static constexpr int kRingOrEpilogue = kRing > kEpilogue ? kRing : kEpilogue;
};

// Byte swap of 32-byte units for row k of a kCols stage of W values.
template <int W>
__device__ __forceinline__ uint32_t unit_swap(uint32_t k) {
    const uint32_t u = (k & 3u) | (k >> 1 & 4u);
    if constexpr (W >= 128) return u << 5;
    else return (u >> 1) << 5;
}

// Where 16-byte chunk `pos` of stage row `row` lies in LDS.
template <int OP, int W>
__device__ __forceinline__ uint32_t chunk_at(uint32_t row, uint32_t pos) {
    if constexpr (OP == kRows) return row * (kStageK * 2) + ((pos ^ ((row >> 1) & 7u)) << 4);
    else return row * (W * 2) + ((pos << 4) ^ unit_swap<W>(row));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, (int)kRawBuffer);
}

__device__ __forceinline__ uint32_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
}

// One operand's part of a workgroup: W rows (columns) in LDS at `lds`.
template <int DT, int OP, int W, int WAVES, bool DIRECT>
struct Stager {
    static constexpr int kThreads = WAVES * kWave;
    static constexpr int kChunks = W * kStageK / kChunk;              // of a stage
    static constexpr int kPer = kChunks / kThreads;                   // of a thread
    static constexpr int kRowChunks = OP == kRows ? kStageK / kChunk : W / kChunk;
    static_assert(kChunks % kThreads == 0, "whole chunks per thread");
    static constexpr int kLoads = DIRECT ? kPer : 0;                  // DMA loads in flight per stage

    // of codes a thread takes two neighbouring chunks at a time
    static constexpr int kTurns = OP == kCodes ? kPer / 2 : kPer;
    static_assert(OP != kCodes || kPer % 2 == 0, "pairs of chunks");

    u32x4 raw[DIRECT ? 1 : kTurns];
    uint32_t sz[OP == kCodes ? kTurns : 1][2];   // scale (low half) and zero of each chunk

    // Stage row and chunk of this thread's load j.
    static __device__ __forceinline__ void place(uint32_t tid, int j, uint32_t &row, uint32_t &pos) {
        const uint32_t c = tid + (uint32_t)j * kThreads;
        row = c / kRowChunks;
        pos = c % kRowChunks;
    }

    // Byte offset of the thread's first chunk from the stage's first; turn j's lies
    // kTurnRows memory rows further, at the same chunk and rotation.
    static constexpr uint32_t kTurnRows = kThreads / kRowChunks;
    static_assert(!DIRECT || kTurnRows % 16 == 0, "the rotations repeat from turn to turn");
    static __device__ __forceinline__ uint32_t source(uint32_t tid) {
        const uint32_t row = tid / kRowChunks, pos = tid % kRowChunks;
        return OP == kRows ? pos ^ ((row >> 1) & 7u) : pos ^ (unit_swap<W>(row) >> 4);
    }

    // Turns [from, to) straight into LDS. p16: kRows the tile's first row at the stage's
    // first k, kCols the stage's first k row at the tile's first column; k_left: k from
    // the stage's first to the end (positive).
    static __device__ __forceinline__ void direct(const uint16_t *p16, uint32_t ld, int live, int k_left, uint8_t FC_LDS *lds,
                                                  uint32_t tid, int from, int to) {
        const uint32_t records = (uint32_t)(OP == kRows ? live : k_left < kStageK ? k_left : kStageK) * ld * 2u;
        const uint64_t at = reinterpret_cast<uint64_t>(p16);
        const u32x4 res = {(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, records, kRawBuffer};
        const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const uint32_t src = source(tid);
        uint32_t off = tid / kRowChunks * (ld * 2u) + src * 16u;
        off = (int)(src * kChunk) < (OP == kRows ? k_left : live) ? off : kOutside;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (j < from || j >= to) continue;
            load_to_lds(res, lds + ((uint32_t)j * kThreads + wave * kWave) * 16u, off, (uint32_t)j * kTurnRows * (ld * 2u));
        }
    }

    // Turns [from, to): 16-bit values at any alignment and length, into registers.
    __device__ __forceinline__ void fetch(const uint16_t *p16, uint32_t ld, int live, int k_left, uint32_t tid, int from, int to) {
        const int wide = OP == kRows ? k_left : live;       // values left along a memory row
        const int high = OP == kRows ? live : k_left;       // memory rows left
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            if (j < from || j >= to) continue;
            uint32_t row, pos;
            place(tid, j, row, pos);
            const int e = (int)pos * kChunk;
            u32x4 v = {0, 0, 0, 0};
            if ((int)row < high) {
                const uint16_t *p = p16 + (uint64_t)row * ld + (uint32_t)e;
                if (e + kChunk <= wide) {
                    v = *reinterpret_cast<const u32x4_a2 *>(p);
                } else if (e < wide) {
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < kChunk; ++i)
                        if (e + i < wide) w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
                    v = u32x4{w[0], w[1], w[2], w[3]};
                }
            }
            raw[j] = v;
        }
    }

    // Turns [from, to) of codes with their scales and zeros, always the same number of
    // loads (3 a turn, 5 where chunks are not paired): what lies past the tile's columns or the rows reads as 0. A chunk
    // that starts at the row's end belongs to columns that are not stored.
    __device__ __forceinline__ void fetch_codes(const uint8_t *codes, const uint16_t *s, const uint16_t *z, uint32_t ld,
                                                uint32_t groups, uint32_t n0, uint32_t magic, bool paired, int live, int k_left,
                                                uint32_t tid, int from, int to) {
        const uint32_t rows = (uint32_t)(k_left < kStageK ? k_left : kStageK);
        const __amdgpu_buffer_rsrc_t cr = buffer_of(codes, rows * ld), sr = buffer_of(s, rows * groups * 2), zr = buffer_of(z, rows * groups * 2);
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            if (j < from || j >= to) continue;
            const uint32_t c = (tid + (uint32_t)j * kThreads) * 2;
            const uint32_t row = c / kRowChunks, e = c % kRowChunks * kChunk;
            const bool in = (int)e < live;
            const uint32_t v = (n0 + e) / kChunk;
            const uint32_t at = in ? row * ld + n0 + e : kOutside, g = in ? (row * groups + group_of(v, magic)) * 2 : kOutside;
            raw[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(cr, (int)at, 0, 0));
            sz[j][0] = load16(sr, g) | load16(zr, g) << 16;
            sz[j][1] = sz[j][0];
            if (!paired) {   // the two chunks may lie in two groups
                const uint32_t h = in ? (row * groups + group_of(v + 1, magic)) * 2 : kOutside;
                sz[j][1] = load16(sr, h) | load16(zr, h) << 16;
            }
        }
    }

    __device__ __forceinline__ void commit(uint8_t FC_LDS *lds, uint32_t tid, int from, int to) {
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            if (j < from || j >= to) continue;
            if constexpr (OP == kCodes) {
                const uint32_t c = (tid + (uint32_t)j * kThreads) * 2;
                const uint32_t row = c / kRowChunks, pos = c % kRowChunks;
                const uint32_t w[2][2] = {{raw[j].x, raw[j].y}, {raw[j].z, raw[j].w}};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[kLaneElems];
                    dequant8<8>(w[h], (uint16_t)sz[j][h], (uint16_t)(sz[j][h] >> 16), x);
                    *(FC_LDS u32x4 *)(lds + chunk_at<OP, W>(row, pos + h)) = narrow8<DT>(x);
                }
            } else {
                uint32_t row, pos;
                place(tid, j, row, pos);
                *(FC_LDS u32x4 *)(lds + chunk_at<OP, W>(row, pos)) = raw[j];
            }
        }
    }
};

// Fragments of 16 rows (columns) and 32 k. at(): the lane's first byte in block 0 of
// the wave, whose first row (column) is `first`; a block further and a step of k are
// a constant added or XORed (the blocks' and steps' bits are free in it).
template <int OP, int W>
struct Fragment {
    static __device__ __forceinline__ uint32_t at(uint32_t first, uint32_t lane) {
        const uint32_t q = lane & 15u, g = lane >> 4;
        if constexpr (OP == kRows) return chunk_at<kRows, W>(first + q, g);
        const uint32_t k = g * 8 + (q >> 2);
        return k * (W * 2) + (((first + (q & 3u) * 4) * 2) ^ unit_swap<W>(k));   // k + 4 is swapped alike
    }
    static __device__ __forceinline__ u32x4 read(const uint8_t FC_LDS *lds, uint32_t at0, uint32_t block, uint32_t ks) {
        if constexpr (OP == kRows) {
            return *(const FC_LDS u32x4 *)(lds + (at0 ^ (ks << 6)) + block * (kBlock * kStageK * 2));
        } else {
            const uint32_t a = opaque(at0);   // the blocks' addresses are not kept from stage to stage
            const uint8_t FC_LDS *p = lds + (a ^ (block << 5)) + ks * (kStepK * W * 2);
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FC_LDS i16x4 *)p);
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FC_LDS i16x4 *)(p + 4 * (W * 2)));
            const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
            return u32x4{l.x, l.y, h.x, h.y};
        }
    }
};

template <int DT>
__device__ __forceinline__ void widen4(const uint16_t *p, int n, float (&v)[4]) {
    if (n >= 4) {
        const u32x2 w = *reinterpret_cast<const u32x2_a2 *>(p);
        v[0] = widen1<DT>((uint16_t)w.x);
        v[1] = widen1<DT>((uint16_t)(w.x >> 16));
        v[2] = widen1<DT>((uint16_t)w.y);
        v[3] = widen1<DT>((uint16_t)(w.y >> 16));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? widen1<DT>(p[i]) : 0.0f;
    }
}

// Two binary32 values rounded to the dtype, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    const f32x2 pair = {as_f32(a), as_f32(b)};
    if constexpr (DT == 1) return __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, bf16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, f16x2));
}

template <int DT>
__device__ __forceinline__ void store4(uint16_t *p, int n, const float (&v)[4]) {
    const uint32_t lo = narrow2<DT>(v[0], v[1]), hi = narrow2<DT>(v[2], v[3]);
    if (n >= 4) {
        *reinterpret_cast<u32x2_a2 *>(p) = u32x2{lo, hi};
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n) p[i] = (uint16_t)((i < 2 ? lo : hi) >> (16 * (i & 1)));
    }
}

template <int ACT>
__device__ __forceinline__ void activate4(float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_value<ACT>(v[i]);
}

__device__ __forceinline__ void activate4(float (&v)[4], int act) {
    switch (act) {
    case kActRelu: activate4<kActRelu>(v); break;
    case kActSilu: activate4<kActSilu>(v); break;
    case kActGelu: activate4<kActGelu>(v); break;
    case kActGeluTanh: activate4<kActGeluTanh>(v); break;
    default: break;
    }
}

// Four outputs of row m from column n (`left` of them exist): the epilogue of a
// linear layer.
template <int DT>
__device__ __forceinline__ void finish4(const LinearEpilogue &e, uint64_t at, int left, const float (&bias)[4], float (&v)[4]) {
    float m[4], r[4];
    if (e.mul != nullptr) widen4<DT>(e.mul + at, left, m);
    if (e.residual != nullptr) widen4<DT>(e.residual + at, left, r);
    if (e.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += bias[i];
    }
    if (e.z != nullptr) store4<DT>(e.z + at, left, v);
    activate4(v, e.act);
    if (e.mul != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= m[i];
    }
    if (e.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += r[i];
    }
    store4<DT>(e.y + at, left, v);
}

// Workgroup b runs on XCD b % 8: each XCD takes its own run of the tiles, so that its
// workgroups share operands in its L2.
constexpr uint32_t kXcds = 8;
__device__ __forceinline__ uint64_t by_xcd(uint64_t id, uint64_t total) {
    const uint64_t q = total / kXcds, rest = total % kXcds;
    const uint64_t x = id % kXcds;
    return x * q + (x < rest ? x : rest) + id / kXcds;
}

// Tiles in groups of 4 rows, a group column by column.
__device__ __forceinline__ void grouped(uint32_t tile, uint32_t tiles_m, uint32_t tiles_n, uint32_t &tm, uint32_t &tn) {
    const uint32_t per = 4 * tiles_n, g = tile / per, in = tile - g * per;
    const uint32_t rows = tiles_m - 4 * g < 4 ? tiles_m - 4 * g : 4;
    tn = in / rows;
    tm = 4 * g + in - tn * rows;
}

// F32: binary32 results (the weight gradient), else 16-bit ones with the epilogue.
// DIRECT: 16-bit operands go to LDS straight from memory.
template <int DT, int OPA, int OPB, int TM, int TN, int WM, int WN, int NS, bool DIRECT, bool F32>
__global__ __launch_bounds__((Shape<TM, TN, WM, WN, NS>::kThreads)) __attribute__((amdgpu_waves_per_eu(Shape<TM, TN, WM, WN, NS>::kPerSimd)))
void product_kernel(const ProductArgs a, uint32_t magic, bool paired) {
    using S = Shape<TM, TN, WM, WN, NS>;
    constexpr int kSink = OPA == kRows && OPB == kRows && TM == kLargeTile ? 256 : 0;   // of the L2 prefetch
    __shared__ __attribute__((aligned(16))) uint8_t shared[S::kRingOrEpilogue + kSink];
    uint8_t FC_LDS *lds = (uint8_t FC_LDS *)shared;
    const uint32_t tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63u;
    const int wave = (int)__builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const uint64_t flat = grid_index();
    if (flat >= a.total) return;
    const uint64_t id = by_xcd(flat, a.total);
    const uint64_t per = (uint64_t)a.tiles_m * (uint32_t)a.tiles_n;
    const uint64_t batch = id / per;                       // rank, then split
    const uint32_t tile = (uint32_t)(id - batch * per);
    const uint32_t r = (uint32_t)(batch % (uint32_t)a.R), part = (uint32_t)(batch / (uint32_t)a.R);
    uint32_t tm, tn;
    grouped(tile, (uint32_t)a.tiles_m, (uint32_t)a.tiles_n, tm, tn);
    const int m0 = a.from_m + (int)tm * TM, n0 = a.from_n + (int)tn * TN;
    const int64_t k0 = (int64_t)part * a.split_k;
    const int k_count = (int)(a.K - k0 < a.split_k ? a.K - k0 : a.split_k);
    const int stages = (k_count - 1) / kStageK + 1;
    const int live_m = a.M - m0 < TM ? a.M - m0 : TM, live_n = a.N - n0 < TN ? a.N - n0 : TN;

    const uint64_t mk = (uint64_t)a.M * (uint32_t)a.K, nk = (uint64_t)a.N * (uint32_t)a.K;
    const uint32_t lda = (uint32_t)(OPA == kRows ? a.K : a.M), ldb = (uint32_t)(OPB == kRows ? a.K : a.N);
    const uint16_t *pa = a.a + r * mk + (OPA == kRows ? (uint64_t)(uint32_t)m0 * lda + k0 : k0 * lda + (uint32_t)m0);
    const uint16_t *pb = nullptr;
    const uint8_t *codes = nullptr;
    const uint16_t *cs = nullptr, *cz = nullptr;
    uint32_t groups = 0;
    if constexpr (OPB == kCodes) {
        groups = (uint32_t)(a.N / a.group);
        const uint64_t row = r * (uint64_t)(uint32_t)a.K + (uint64_t)k0;
        codes = a.pb.codes + row * ldb;
        cs = a.pb.s + row * groups;
        cz = a.pb.z + row * groups;
    } else {
        pb = a.b + r * nk + (OPB == kRows ? (uint64_t)(uint32_t)n0 * ldb + k0 : k0 * ldb + (uint32_t)n0);
    }

    // Measured on the linear layer (both operands by rows), with and without in turn, T x K x H,
    // us: 8192 x 4096 x 14336 784 and 800, 4096^3 117 and 119, 8192 x 1024 x 8192 160 and 167;
    // 8192^3 848 and 840, 8192 x 8192 x 7168 779 and 776. A stage ahead of the newest staged;
    // two and four stages ahead 1 and 2% slower than one. With an operand by columns it is 3 to
    // 6% slower (whole kilobytes are staged from neighbouring lines there).
    constexpr bool kPrefetch = OPA == kRows && OPB == kRows && DIRECT && TM == kLargeTile;
    constexpr bool kThroughRegs = !DIRECT || OPB == kCodes;   // some of a stage goes through registers
    Stager<DT, OPA, TM, S::kWaves, DIRECT> sa;
    Stager<DT, OPB, TN, S::kWaves, DIRECT && OPB != kCodes> sb;
    // Part `part` of `parts` of stage p's loads straight into the ring's place `at`.
    auto issue = [&](int p, uint32_t at, int part, int parts) {
        if constexpr (DIRECT) {
            const int64_t ko = (int64_t)p * kStageK;
            const int left = k_count - p * kStageK;
            uint8_t FC_LDS *la = lds + at, *lb = la + S::kBytesA;
            constexpr int na = decltype(sa)::kPer, nb = decltype(sb)::kPer;
            sa.direct(pa + (OPA == kRows ? ko : ko * lda), lda, live_m, left, la, tid, na * part / parts, na * (part + 1) / parts);
            if constexpr (OPB != kCodes)
                sb.direct(pb + (OPB == kRows ? ko : ko * ldb), ldb, live_n, left, lb, tid, nb * part / parts, nb * (part + 1) / parts);
        }
    };
    // The same for what goes through registers: into these, and from there to LDS.
    auto fetch = [&](int p, int part, int parts) {
        const int64_t ko = (int64_t)p * kStageK;
        const int left = k_count - p * kStageK;
        constexpr int na = decltype(sa)::kTurns, nb = decltype(sb)::kTurns;
        if constexpr (!DIRECT)
            sa.fetch(pa + (OPA == kRows ? ko : ko * lda), lda, live_m, left, tid, na * part / parts, na * (part + 1) / parts);
        if constexpr (OPB == kCodes)
            sb.fetch_codes(codes + ko * ldb, cs + ko * groups, cz + ko * groups, ldb, groups, (uint32_t)n0, magic, paired, live_n,
                           left, tid, nb * part / parts, nb * (part + 1) / parts);
        else if constexpr (!DIRECT)
            sb.fetch(pb + (OPB == kRows ? ko : ko * ldb), ldb, live_n, left, tid, nb * part / parts, nb * (part + 1) / parts);
    };
    auto commit = [&](uint32_t at, int part, int parts) {
        uint8_t FC_LDS *la = lds + at, *lb = la + S::kBytesA;
        constexpr int na = decltype(sa)::kTurns, nb = decltype(sb)::kTurns;
        if constexpr (!DIRECT) sa.commit(la, tid, na * part / parts, na * (part + 1) / parts);
        if constexpr (kThroughRegs) sb.commit(lb, tid, nb * part / parts, nb * (part + 1) / parts);
    };

    // L2 prefetch: the workgroups beside this one on its XCD run the tiles of 4 rows and 8
    // columns; those of a row stage the same part of A, those of a column the same part of
    // B. Each fetches its share of the lines (a row's 64 k) that all of them will stage, a
    // dword of each, into a part of LDS that nothing reads. One load a wave and stage, in
    // any case: what is past the last stage or row lies outside the buffer.
    auto prefetch = [&](int p) {
        constexpr int kHalf = S::kWaves / 2;   // of the waves: for A, for B
        constexpr uint32_t kLinesA = TM / 8 / kHalf, kLinesB = TN / 4 / kHalf;   // of a wave
        const bool on_a = wave < kHalf;
        const uint32_t lines = on_a ? kLinesA : kLinesB, ld = on_a ? lda : ldb;
        const uint32_t first = on_a ? (tn % 8 * kHalf + (uint32_t)wave) * kLinesA
                                    : (tm % 4 * kHalf + (uint32_t)(wave - kHalf)) * kLinesB;
        const uint64_t at = reinterpret_cast<uint64_t>(on_a ? pa : pb) + (uint64_t)p * (kStageK * 2);
        const uint32_t bytes = p < stages ? (uint32_t)(on_a ? live_m : live_n) * ld * 2u : 0u;
        const u32x4 res = {(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at),
                           (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32) & 0xFFFFu),
                           (uint32_t)__builtin_amdgcn_readfirstlane(bytes), kRawBuffer};
        touch_to_lds(res, lds + S::kRingOrEpilogue, lane < lines ? (first + lane) * ld * 2u : kOutside);
    };

    f32x4 acc[S::kBM][S::kBN];
#pragma unroll
    for (int i = 0; i < S::kBM; ++i)
#pragma unroll
        for (int j = 0; j < S::kBN; ++j) acc[i][j] = f32x4{};

    // A stage is 2 steps of 32 k. The fragments of a step are read during the products
    // of the step before, those of a block of columns after that block's products. In
    // the last step these are the next stage's: after its first products each wave waits
    // for its own loads of that stage and the workgroup meets; from there on the place
    // of this stage is free, every wave having read the last of it, and takes the loads
    // of the stage NS further. What goes through registers is written to LDS in the step
    // before the meeting, and its registers take the stage after next at once.
    const uint32_t fa0 = Fragment<OPA, TM>::at((uint32_t)(wm * S::kSM), lane);
    const uint32_t fb0 = Fragment<OPB, TN>::at((uint32_t)(wn * S::kSN), lane);
    u32x4 fa[2][S::kBM], fb[S::kBN];
    auto read_a = [&](uint32_t at, int ks, int i) {
        if (i >= 0 && i < S::kBM) fa[ks & 1][i] = Fragment<OPA, TM>::read(lds + at, fa0, (uint32_t)i, (uint32_t)ks);
    };
    auto read_b = [&](uint32_t at, int ks, int j) {
        fb[j] = Fragment<OPB, TN>::read(lds + at + S::kBytesA, fb0, (uint32_t)j, (uint32_t)ks);
    };
    static_assert(S::kBM <= S::kBN, "a part of a step has a block of columns");
    auto step = [&](int ks, auto &&side) {
#pragma unroll
        for (int j = 0; j < S::kBN; ++j) {
#pragma unroll
            for (int i = 0; i < S::kBM; ++i) acc[i][j] = mfma<DT>(fa[ks & 1][i], fb[j], acc[i][j]);
            side(j);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr int kSteps = kStageK / kStepK;
    // products of the last step before the meeting: they cover the last reads' latency
    constexpr int kBefore = 1;
    static_assert(S::kBN - kBefore + 1 >= S::kBM, "the next stage's rows are read after the meeting");
    constexpr int kLoads = decltype(sa)::kLoads + decltype(sb)::kLoads;   // straight into LDS, a wave's of a stage
    static_assert(NS == 2 || !kThroughRegs, "what goes through registers is one stage ahead");
    if constexpr (kThroughRegs) {
        fetch(0, 0, 1);
        commit(0, 0, 1);
        if (stages > 1) fetch(1, 0, 1);
    }
#pragma unroll
    for (int p = 0; p < NS; ++p)
        if (p < stages) issue(p, (uint32_t)p * S::kStage, 0, 1);
    // every stage's loads have one prefetch behind them, which the waits below count
    if constexpr (kPrefetch) prefetch(NS);
    if (!kThroughRegs && stages >= NS) wait_memory<(NS - 1) * kLoads + (kPrefetch ? 1 : 0)>();
    else wait_memory<0>();
    meet();
#pragma unroll
    for (int j = 0; j < S::kBN; ++j) {
        read_a(0, 0, j);
        read_b(0, 0, j);
    }
    uint32_t here = 0;   // the ring's place of stage p
    for (int p = 0; p < stages; ++p) {
        const uint32_t next = here + S::kStage == S::kRing ? 0 : here + S::kStage;
        const bool more = p + 1 < stages, after = p + 2 < stages, ahead = p + NS < stages;
#pragma unroll
        for (int ks = 0; ks < kSteps - 1; ++ks) {
            if constexpr (kThroughRegs) {
                if (more) commit(next, ks, kSteps - 1);
                if (after) fetch(p + 2, ks, kSteps - 1);
            }
            step(ks, [&](int j) {
                read_a(here, ks + 1, j);
                read_b(here, ks + 1, j);
            });
        }
        step(kSteps - 1, [&](int j) {
            if (j < kBefore - 1) return;
            const uint32_t from = more ? next : here;
            if (j == kBefore - 1) {
                // Stage p + 1 has landed: the loads of the later ones, and what was fetched
                // into registers meanwhile, are younger.
                if constexpr (!DIRECT) {
                    wait_memory<63>();
                } else if constexpr (kThroughRegs) {
                    if (!after) wait_memory<0>();
                    else if (paired) wait_memory<3 * decltype(sb)::kTurns>();
                    else wait_memory<5 * decltype(sb)::kTurns>();
                } else {
                    if (p + NS - 1 < stages) wait_memory<(NS - 2) * kLoads + (kPrefetch ? 1 : 0)>();
                    else wait_memory<0>();
                }
                meet();
#pragma unroll
                for (int i = 0; i < kBefore; ++i) read_b(from, 0, i);
            } else {
                read_b(from, 0, j);
            }
            read_a(from, 0, j - kBefore + 1);
            if (ahead) issue(p + NS, here, j - kBefore + 1, S::kBN - kBefore + 1);
            if constexpr (kPrefetch) {
                if (j == S::kBN - 1) prefetch(p + NS + 1);
            }
        });
        here = next;
    }

    // 32 rows of the wave at a time through its own part of LDS, from where a lane takes 4
    // neighbouring columns of a row: whole lines go out
    constexpr int kLanesRow = S::kSN / 4, kRowsTurn = kWave / kLanesRow;
    if constexpr (kPrefetch) wait_memory<0>();   // the last prefetch's store to LDS
    meet();   // every wave has read its last fragments
    FC_LDS float *mine = (FC_LDS float *)(lds) + wave * 32 * S::kPitch;
    const int c = (int)(lane % kLanesRow) * 4, n = n0 + wn * S::kSN + c, left = a.N - n;
    float bias[4] = {};
    if (!F32 && a.e.bias != nullptr && left > 0) widen4<DT>(a.e.bias + (uint64_t)r * (uint32_t)a.N + (uint32_t)n, left, bias);
#pragma unroll
    for (int i = 0; i < S::kBM; i += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < S::kBN; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    mine[(h * kBlock + 4 * (lane >> 4) + v) * S::kPitch + j * kBlock + (lane & 15u)] = acc[i + h][j][v];
        for (int t = 0; t < 32; t += kRowsTurn) {
            const int row = t + (int)(lane / kLanesRow), m = m0 + wm * S::kSM + i * kBlock + row;
            const f32x4 w = *(const FC_LDS f32x4 *)(mine + row * S::kPitch + c);
            float v[4] = {w.x, w.y, w.z, w.w};
            if (m >= a.M || left <= 0) continue;
            if constexpr (F32) {
                float *o = a.out + ((uint64_t)batch * (uint32_t)a.M + (uint32_t)m) * (uint32_t)a.N + (uint32_t)n;
                if (left >= 4) {
                    f32x4_a4 *q = reinterpret_cast<f32x4_a4 *>(o);
                    f32x4_a4 sum = {v[0], v[1], v[2], v[3]};
                    if (a.accumulate) sum += *q;
                    *q = sum;
                } else {
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        if (k < left) o[k] = a.accumulate ? o[k] + v[k] : v[k];
                }
            } else {
                finish4<DT>(a.e, ((uint64_t)r * (uint32_t)a.M + (uint32_t)m) * (uint32_t)a.N + (uint32_t)n, left, bias, v);
            }
        }
    }
}

template <int DT, int OPA, int OPB, int TM, int TN, int WM, int WN, int NS, bool DIRECT, bool F32>
hipError_t launch_product(ProductArgs a, hipStream_t stream) {
    using S = Shape<TM, TN, WM, WN, NS>;
    a.tiles_m = (a.to_m - a.from_m - 1) / TM + 1;
    a.tiles_n = (a.to_n - a.from_n - 1) / TN + 1;
    a.total = (uint64_t)a.tiles_m * (uint64_t)a.tiles_n * (uint64_t)a.R * (uint64_t)a.split;
    uint32_t magic = 0;
    if (OPB == kCodes && a.group != kChunk) {
        const uint64_t d = (uint64_t)(a.group / kChunk);
        magic = (uint32_t)(((uint64_t(1) << 32) + d - 1) / d);
    }
    hipLaunchKernelGGL((product_kernel<DT, OPA, OPB, TM, TN, WM, WN, NS, DIRECT, F32>), grid_of_blocks(a.total),
                       dim3(S::kThreads), 0, stream, a, magic, a.group % (2 * kChunk) == 0);
    return hipGetLastError();
}

// A product's tiles: those of 256 over the region that fills the device with them in
// whole rounds, smaller ones over the rest (fc_product_dispatch.h).
template <int DT, int OPA, int OPB, bool DIRECT, bool F32>
hipError_t launch_tiles(ProductArgs a, hipStream_t stream) {
    const int cus = compute_units();
    if (cus <= 0) return hipErrorInvalidDevice;
    constexpr bool kLarge = DIRECT && OPB != kCodes;
    const ProductPlan plan = product_plan(a.R * a.split, a.M, a.N, cus, kLarge);
    for (const ProductPlan::Part &p : plan.part) {
        if (p.tile == 0) continue;
        a.from_m = p.from_m;
        a.from_n = p.from_n;
        a.to_m = p.to_m;
        a.to_n = p.to_n;
        hipError_t err;
        if (p.tile == kSmallTile) {
            err = launch_product<DT, OPA, OPB, 64, 64, 2, 2, kLarge ? 4 : 2, DIRECT, F32>(a, stream);
        } else if (p.tile == kMiddleTile) {
            err = launch_product<DT, OPA, OPB, 128, 128, 2, 2, 2, DIRECT, F32>(a, stream);
        } else {
            if constexpr (kLarge) err = launch_product<DT, OPA, OPB, 256, 256, 4, 2, 2, DIRECT, F32>(a, stream);
            else err = hipErrorInvalidValue;
        }
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// The epilogue of a product whose sums are split: binary32 parts [split][n] of
// [R][M][N], added in their order, 4 columns of a row to a thread.
template <int DT>
__global__ __launch_bounds__(kBlockThreads) void join_epilogue_kernel(const float *part, int split, uint64_t rows, int M, int N,
                                                                      LinearEpilogue e) {
    const uint32_t quads = ((uint32_t)N + 3) / 4;
    const uint64_t i = grid_index() * kBlockThreads + __builtin_amdgcn_workitem_id_x();
    const uint64_t row = i / quads;
    if (row >= rows) return;
    const int n = (int)(i - row * quads) * 4, left = N - n;
    const uint64_t at = row * (uint32_t)N + (uint32_t)n, all = rows * (uint32_t)N;
    float v[4] = {};
    for (int p = 0; p < split; ++p) {
        const float *q = part + (uint64_t)p * all + at;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] += k < left ? q[k] : 0.0f;
    }
    float bias[4] = {};
    if (e.bias != nullptr) widen4<DT>(e.bias + row / (uint32_t)M * (uint32_t)N + (uint32_t)n, left, bias);
    finish4<DT>(e, at, left, bias, v);
}

// A product with the linear layer's epilogue, its sums split as `plan` has it (few
// outputs: tiles of 64).
template <int DT, int OPA, int OPB, bool DIRECT>
hipError_t launch_split(ProductArgs a, const SplitPlan &plan, float *part, hipStream_t stream) {
    a.split = plan.split;
    a.split_k = plan.split_k;
    if (plan.split == 1) return launch_tiles<DT, OPA, OPB, DIRECT, false>(a, stream);
    a.out = part;
    a.to_m = a.M;
    a.to_n = a.N;
    const hipError_t err = launch_product<DT, OPA, OPB, 64, 64, 2, 2, DIRECT ? 4 : 2, DIRECT, true>(a, stream);
    if (err != hipSuccess) return err;
    const uint64_t rows = (uint64_t)a.R * (uint64_t)a.M, threads = rows * (((uint32_t)a.N + 3) / 4);
    hipLaunchKernelGGL((join_epilogue_kernel<DT>), grid_of_blocks((threads + kBlockThreads - 1) / kBlockThreads),
                       dim3(kBlockThreads), 0, stream, part, plan.split, rows, a.M, a.N, a.e);
    return hipGetLastError();
}

}  // namespace
}  // namespace fc
