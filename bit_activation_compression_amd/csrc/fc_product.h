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
//     (row / 2) % 8, so that the fragment reads (ds_read_b128: 32 rows x one chunk
//     per half wave) meet each bank once;
//   - kCols, kCodes: a stage is 64 rows of TM values; fragments are read with the
//     transposing ds_read_b64_tr_b16 (16 lanes read 4 rows x 16 values and get 4 k
//     of one column each). A half wave reads 64 bytes of 4 rows: their 64-byte
//     units are swapped by k % 4, so that these meet each bank once as well.
// 16-bit operands whose rows are whole 16-byte chunks go to LDS straight from
// memory (buffer_load ... lds), the rotation done by which chunk a lane fetches;
// others, and codes, go through registers: loads before a stage's products, stores
// to LDS after them.
//
// v_mfma_f32_32x32x16: lane l holds row (column) l % 32 and k 8 (l / 32) + 0..7 of an
// operand, and of the result column l % 32 and rows 8 (v / 4) + 4 (l / 32) + v % 4.
#pragma once

#include "fc_act.h"
#include "fc_grid.h"
#include "fc_launch_train.h"
#include "fc_rows.h"

namespace fc {
namespace {

constexpr int kRows = 0, kCols = 1, kCodes = 2;
constexpr int kStageK = 64;
constexpr int kChunk = 8;                      // values of a 16-byte chunk
constexpr uint32_t kOutside = 0xFFFFFFF0u;     // an offset past every buffer
constexpr int kRawBuffer = 0x00020000;         // resource word 3: raw 32-bit buffer

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

#define FC_LDS __attribute__((address_space(3)))

template <int DT>
__device__ __forceinline__ f32x16 mfma(const u32x4 &a, const u32x4 &b, const f32x16 &c) {
    if constexpr (DT == 1)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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

struct ProductArgs {
    const uint16_t *a, *b;
    Payload pb;             // B of kCodes
    int group;
    int R, M, N, K;         // per rank
    int tiles_m, tiles_n;
    uint64_t total;         // tiles of all ranks and splits
    int split, split_k;     // k in `split` runs of split_k (a multiple of the stage)
    LinearEpilogue e;       // 16-bit results
    float *out;             // binary32 results [split][R][M][N]
    int accumulate;
};

// The memory of one operand's tile: `rows` real rows (of m or n) from the base.
template <int OP>
struct Operand {
    const uint16_t *base;   // kRows: row m0, k 0; kCols: row k 0, column m0
    uint32_t ld;            // values per memory row
    int live;               // rows (kRows) or columns (kCols) that exist, from m0
};

template <int TM, int TN, int WM, int WN>
struct Shape {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
    static constexpr int kSM = TM / WM, kSN = TN / WN;         // of a wave
    static constexpr int kBM = kSM / 32, kBN = kSN / 32;
    static constexpr int kBytesA = TM * kStageK * 2, kBytesB = TN * kStageK * 2, kStage = kBytesA + kBytesB;
    // the epilogue's rows of a wave: 32 rows of binary32, padded so that the two
    // halves of a wave (4 rows apart) write different banks
    static constexpr int kPitch = kSN + 8;
    static constexpr int kEpilogue = kWaves * 32 * kPitch * 4;
};

// Byte of the 64-byte-unit swap for row k of a kCols stage of W values.
template <int W>
__device__ __forceinline__ uint32_t unit_swap(uint32_t k) {
    if constexpr (W >= 128) return (k & 3u) << 6;
    else return ((k >> 1) & 1u) << 6;
}

// Where 16-byte chunk `pos` of stage row `row` lies in LDS.
template <int OP, int W>
__device__ __forceinline__ uint32_t chunk_at(uint32_t row, uint32_t pos) {
    if constexpr (OP == kRows) return row * (kStageK * 2) + ((pos ^ ((row >> 1) & 7u)) << 4);
    else return row * (W * 2) + ((pos << 4) ^ unit_swap<W>(row));
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

    u32x4 raw[DIRECT || OP == kCodes ? 1 : kPer];
    u32x2 code[OP == kCodes ? kPer : 1];
    uint32_t sz[OP == kCodes ? kPer : 1];

    // Stage row and chunk of this thread's load j.
    static __device__ __forceinline__ void place(uint32_t tid, int j, uint32_t &row, uint32_t &pos) {
        const uint32_t c = tid + (uint32_t)j * kThreads;
        row = c / kRowChunks;
        pos = c % kRowChunks;
    }

    // p16: kRows the tile's first row, kCols the stage's first k row at the tile's
    // first column; k_left: k from the stage's first to the end (positive).
    __device__ __forceinline__ void direct(const uint16_t *p16, uint32_t ld, int live, int k_left, uint8_t FC_LDS *lds,
                                           uint32_t tid) {
        const uint32_t records = OP == kRows ? (uint32_t)live * ld * 2u : (uint32_t)(k_left < kStageK ? k_left : kStageK) * ld * 2u;
        const __amdgpu_buffer_rsrc_t res =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(p16), (short)0, (int)records, kRawBuffer);
        const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            uint32_t row, pos, src;
            place(tid, j, row, pos);
            uint32_t off;
            if constexpr (OP == kRows) {
                src = pos ^ ((row >> 1) & 7u);
                off = row * ld * 2u + src * 16u;
                off = (int)(src * kChunk) < k_left ? off : kOutside;
            } else {
                src = pos ^ (unit_swap<W>(row) >> 4);
                off = row * ld * 2u + src * 16u;
                off = (int)(src * kChunk) < live ? off : kOutside;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (FC_LDS void *)(lds + ((uint32_t)j * kThreads + wave * kWave) * 16u), 16,
                                                     off, 0, 0, 0);
        }
    }

    // 16-bit values at any alignment and length, into registers.
    __device__ __forceinline__ void fetch(const uint16_t *p16, uint32_t ld, int live, int k_left, uint32_t tid) {
        const int wide = OP == kRows ? k_left : live;       // values left along a memory row
        const int high = OP == kRows ? live : k_left;       // memory rows left
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
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

    // Codes with their scale and zero: codes, s and z at the stage's first k row.
    __device__ __forceinline__ void fetch_codes(const uint8_t *codes, const uint16_t *s, const uint16_t *z, uint32_t ld,
                                                uint32_t groups, uint32_t n0, uint32_t magic, int live, int k_left,
                                                uint32_t tid) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            uint32_t row, pos;
            place(tid, j, row, pos);
            const uint32_t e = pos * kChunk;
            u32x2 v = {0, 0};
            uint32_t m = 0;   // scale and zero 0: the value 0
            if ((int)row < k_left && (int)e < live) {
                v = *reinterpret_cast<const u32x2 *>(codes + (uint64_t)row * ld + n0 + e);
                const uint64_t g = (uint64_t)row * groups + group_of((n0 + e) / kChunk, magic);
                m = (uint32_t)s[g] | (uint32_t)z[g] << 16;
            }
            code[j] = v;
            sz[j] = m;
        }
    }

    __device__ __forceinline__ void commit(uint8_t FC_LDS *lds, uint32_t tid) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            uint32_t row, pos;
            place(tid, j, row, pos);
            u32x4 v;
            if constexpr (OP == kCodes) {
                const uint32_t w[2] = {code[j].x, code[j].y};
                float x[kLaneElems];
                dequant8<8>(w, (uint16_t)sz[j], (uint16_t)(sz[j] >> 16), x);
                v = narrow8<DT>(x);
            } else {
                v = raw[j];
            }
            *(FC_LDS u32x4 *)(lds + chunk_at<OP, W>(row, pos)) = v;
        }
    }
};

// Fragment of 32 rows (columns) from `first` and 16 k from 16 ks.
template <int OP, int W>
__device__ __forceinline__ u32x4 fragment(const uint8_t FC_LDS *lds, uint32_t first, uint32_t ks, uint32_t lane) {
    if constexpr (OP == kRows) {
        const uint32_t row = first + (lane & 31u);
        return *(const FC_LDS u32x4 *)(lds + chunk_at<kRows, W>(row, 2 * ks + (lane >> 5)));
    } else {
        const uint32_t q = lane & 15u, k = ks * 16 + (lane >> 5) * 8 + (q >> 2);
        const uint32_t col = (first + ((lane >> 4) & 1u) * 16 + (q & 3u) * 4) * 2;
        const uint32_t at = k * (W * 2) + (col ^ unit_swap<W>(q >> 2));   // k % 4 is q / 4
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FC_LDS i16x4 *)(lds + at));
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FC_LDS i16x4 *)(lds + at + 4 * (W * 2)));
        const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
        return u32x4{l.x, l.y, h.x, h.y};
    }
}

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

template <int DT>
__device__ __forceinline__ void store4(uint16_t *p, int n, const float (&v)[4]) {
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = narrow1<DT>(v[i]);
    if (n >= 4) {
        *reinterpret_cast<u32x2_a2 *>(p) = u32x2{(uint32_t)h[0] | (uint32_t)h[1] << 16, (uint32_t)h[2] | (uint32_t)h[3] << 16};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = h[i];
    }
}

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
    case kActRelu: return act_value<kActRelu>(z);
    case kActSilu: return act_value<kActSilu>(z);
    case kActGelu: return act_value<kActGelu>(z);
    case kActGeluTanh: return act_value<kActGeluTanh>(z);
    default: return z;
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
    if (e.act != kActNone) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate(v[i], e.act);
    }
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

// F32: binary32 results (the weight gradient), else 16-bit ones with the epilogue.
// DIRECT: 16-bit operands go to LDS straight from memory.
template <int DT, int OPA, int OPB, int TM, int TN, int WM, int WN, bool DIRECT, bool F32>
__global__ __launch_bounds__((Shape<TM, TN, WM, WN>::kThreads)) __attribute__((amdgpu_waves_per_eu(2, 2)))
void product_kernel(const ProductArgs a, uint32_t magic) {
    using S = Shape<TM, TN, WM, WN>;
    constexpr int kLds = 2 * S::kStage > S::kEpilogue || F32 ? 2 * S::kStage : S::kEpilogue;
    __shared__ __attribute__((aligned(16))) uint8_t shared[kLds];
    uint8_t FC_LDS *lds = (uint8_t FC_LDS *)shared;
    const uint32_t tid = __builtin_amdgcn_workitem_id_x(), lane = tid & 63u;
    const int wave = (int)__builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const uint64_t id = grid_index();
    if (id >= a.total) return;
    const uint64_t per = (uint64_t)a.tiles_m * (uint32_t)a.tiles_n;
    const uint64_t batch = id / per;                       // rank, then split
    const uint32_t tile = (uint32_t)(id - batch * per);
    const uint32_t r = (uint32_t)(batch % (uint32_t)a.R), part = (uint32_t)(batch / (uint32_t)a.R);
    const int m0 = (int)(tile / (uint32_t)a.tiles_n) * TM, n0 = (int)(tile % (uint32_t)a.tiles_n) * TN;
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

    Stager<DT, OPA, TM, S::kWaves, DIRECT> sa;
    Stager<DT, OPB, TN, S::kWaves, DIRECT && OPB != kCodes> sb;
    // stage p: from memory into LDS buffer p % 2, or into registers
    auto issue = [&](int p) {
        const int64_t ko = (int64_t)p * kStageK;
        const int left = k_count - p * kStageK;
        const uint16_t *qa = pa + (OPA == kRows ? ko : ko * lda);
        uint8_t FC_LDS *la = lds + (p & 1) * S::kStage, *lb = la + S::kBytesA;
        if constexpr (DIRECT) sa.direct(qa, lda, live_m, left, la, tid);
        else sa.fetch(qa, lda, live_m, left, tid);
        if constexpr (OPB == kCodes) {
            sb.fetch_codes(codes + ko * ldb, cs + ko * groups, cz + ko * groups, ldb, groups, (uint32_t)n0, magic, live_n, left, tid);
        } else {
            const uint16_t *qb = pb + (OPB == kRows ? ko : ko * ldb);
            if constexpr (DIRECT) sb.direct(qb, ldb, live_n, left, lb, tid);
            else sb.fetch(qb, ldb, live_n, left, tid);
        }
    };
    auto commit = [&](int p) {
        uint8_t FC_LDS *la = lds + (p & 1) * S::kStage, *lb = la + S::kBytesA;
        if constexpr (!DIRECT) sa.commit(la, tid);
        if constexpr (!DIRECT || OPB == kCodes) sb.commit(lb, tid);
    };

    f32x16 acc[S::kBM][S::kBN];
#pragma unroll
    for (int i = 0; i < S::kBM; ++i)
#pragma unroll
        for (int j = 0; j < S::kBN; ++j) acc[i][j] = f32x16{};

    issue(0);
    commit(0);
    for (int p = 0; p < stages; ++p) {
        // stage p is in LDS and every wave is done with stage p - 1, whose buffer
        // stage p + 1 then fills
        wait_memory<0>();
        meet();
        const bool more = p + 1 < stages;
        if (more) issue(p + 1);
        const uint8_t FC_LDS *la = lds + (p & 1) * S::kStage, *lb = la + S::kBytesA;
#pragma unroll
        for (uint32_t ks = 0; ks < kStageK / 16; ++ks) {
            u32x4 fa[S::kBM], fb[S::kBN];
#pragma unroll
            for (int i = 0; i < S::kBM; ++i) fa[i] = fragment<OPA, TM>(la, (uint32_t)(wm * S::kSM + i * 32), ks, lane);
#pragma unroll
            for (int j = 0; j < S::kBN; ++j) fb[j] = fragment<OPB, TN>(lb, (uint32_t)(wn * S::kSN + j * 32), ks, lane);
#pragma unroll
            for (int i = 0; i < S::kBM; ++i)
#pragma unroll
                for (int j = 0; j < S::kBN; ++j) acc[i][j] = mfma<DT>(fa[i], fb[j], acc[i][j]);
        }
        if (more) commit(p + 1);
    }

    if constexpr (F32) {
        // a row's 32 columns of a block are one line
        float *out = a.out + (uint64_t)batch * ((uint64_t)a.M * (uint32_t)a.N);
#pragma unroll
        for (int i = 0; i < S::kBM; ++i)
#pragma unroll
            for (int j = 0; j < S::kBN; ++j) {
                const int n = n0 + wn * S::kSN + j * 32 + (int)(lane & 31u);
                const int mb = m0 + wm * S::kSM + i * 32 + (int)(lane >> 5) * 4;
                if (n < a.N) {
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int m = mb + 8 * (v / 4) + v % 4;
                        if (m < a.M) {
                            float *o = out + (uint64_t)(uint32_t)m * (uint32_t)a.N + (uint32_t)n;
                            *o = a.accumulate ? *o + acc[i][j][v] : acc[i][j][v];
                        }
                    }
                }
            }
    } else {
        // 32 rows of the wave at a time through its own part of LDS, from where a lane
        // takes 4 neighbouring columns of a row
        constexpr int kLanesRow = S::kSN / 4, kRowsTurn = kWave / kLanesRow;
        meet();   // every wave has read its last fragments
        FC_LDS float *mine = (FC_LDS float *)(lds) + wave * 32 * S::kPitch;
        const int c = (int)(lane % kLanesRow) * 4, n = n0 + wn * S::kSN + c, left = a.N - n;
        float bias[4] = {};
        if (a.e.bias != nullptr && left > 0) widen4<DT>(a.e.bias + (uint64_t)r * (uint32_t)a.N + (uint32_t)n, left, bias);
#pragma unroll
        for (int i = 0; i < S::kBM; ++i) {
#pragma unroll
            for (int j = 0; j < S::kBN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    mine[(8 * (v / 4) + 4 * (lane >> 5) + v % 4) * S::kPitch + j * 32 + (lane & 31u)] = acc[i][j][v];
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            for (int t = 0; t < 32; t += kRowsTurn) {
                const int row = t + (int)(lane / kLanesRow), m = m0 + wm * S::kSM + i * 32 + row;
                const f32x4 w = *(const FC_LDS f32x4 *)(mine + row * S::kPitch + c);
                float v[4] = {w.x, w.y, w.z, w.w};
                if (m < a.M && left > 0)
                    finish4<DT>(a.e, ((uint64_t)r * (uint32_t)a.M + (uint32_t)m) * (uint32_t)a.N + (uint32_t)n, left, bias, v);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    }
}

template <int DT, int OPA, int OPB, int TM, int TN, int WM, int WN, bool DIRECT, bool F32>
hipError_t launch_product(ProductArgs a, hipStream_t stream) {
    using S = Shape<TM, TN, WM, WN>;
    a.tiles_m = (a.M - 1) / TM + 1;
    a.tiles_n = (a.N - 1) / TN + 1;
    a.total = (uint64_t)a.tiles_m * (uint64_t)a.tiles_n * (uint64_t)a.R * (uint64_t)a.split;
    uint32_t magic = 0;
    if (OPB == kCodes && a.group != kChunk) {
        const uint64_t d = (uint64_t)(a.group / kChunk);
        magic = (uint32_t)(((uint64_t(1) << 32) + d - 1) / d);
    }
    hipLaunchKernelGGL((product_kernel<DT, OPA, OPB, TM, TN, WM, WN, DIRECT, F32>), grid_of_blocks(a.total),
                       dim3(S::kThreads), 0, stream, a, magic);
    return hipGetLastError();
}

}  // namespace
}  // namespace fc
