// pkv_tree.cu -- attention of a tree of drafted tokens per sequence over the
// paged cache (fp16 or FP8), on the fifth-generation tensor cores.
//
// Sequence i holds L tokens, the last Q of them drafted; query row r sees the
// context 0 .. L-Q-1 and the drafted tokens whose mask bit is set:
//     out = sum_vis 2^(s_j - m) V_j / sum_vis 2^(s_j - m),
//     s_j = scale log2(e) q . K_j,  m any reference near the largest s_j.
//
// The rows of a (sequence, KV head) -- drafted token j, head g of the group:
// row j*G + g -- are cut into tiles of 128 (the MMA's M), the cache into steps
// of 128 keys.  The work is the list of (tile, sequence, KV head) items, each
// its steps plus a start-up cost; one persistent CTA per SM takes an equal
// contiguous stretch of the whole list, so a single long sequence fills the
// GPU as well as a batch does, and the CTAs that work on different tiles of
// the same keys do so at about the same time, out of L2.  An item cut by a stretch's border leaves fp32
// partial states (m, l, O) in the workspace, and a second small kernel, whose
// CTAs start as the first one's leave, merges them.  Bound: HBM while a tile's
// 128-key step (64 KB of fp16 keys and values) costs less than its bytes, i.e.
// to about 128 rows per KV head; the step's chain of MMAs and softmax above.
//
// Per CTA, warp-specialised, every hand-off an mbarrier with a bounded wait:
//  * warp 0 walks the stretch, publishes its pieces and stages their keys, one
//    tensor copy per block, in a ring; warp 1 stages the values likewise;
//  * warp 2 stages a piece's query tile and issues S = Q K^T into one of two
//    score buffers, so the scores of the next step are computed while the
//    softmax works on this one; warp 3 issues O += P V;
//  * warps 4-11, two threads per row: the softmax, with the tree's mask.
//    Weights are rounded to fp16 for the MMA, the normaliser sums them as they
//    were, in 32 bits.  The reference m is set 2^11 below the largest score and
//    moves only when that grows by more than 2^4 (O is rescaled in tensor memory
//    first), so the row's largest weight lies in [2^11, 2^15] and uses fp16's
//    range: rounding costs a weight 2^-11 of itself where it is above 2^-25 of
//    the row's largest one, and 2^-36 of the largest below that, which many
//    keys of little weight behind one of large weight would add up;
//  * FP8: the rings hold codes, and warps 12-15 turn them into fp16 tiles
//    (exact) for the MMAs.  A key's scale, times scale log2(e), multiplies its
//    score and its value's scale the weight, both in fp32; m is then the largest visible log2 of
//    their product, so the scaled weights use fp16's range whatever the scales
//    are.  (A step's largest score plus its largest scale's logarithm is an
//    upper bound; the maximum itself is taken when that passes the reference.)
// Value rows behind the sequence's end hold anything and are zeroed before the
// MMA (by the softmax warps, FP8: as they are converted); drafted rows may be
// masked for some query rows, and 0 x NaN is NaN, so their non-finite elements
// are zeroed too and added, where visible, when the piece's O is read out.
// Rows of a tile past the last drafted one cost no softmax work: a warp whose
// 16 rows are all past it only passes the barriers on.
//
// The kernel's code is kept small (rolled loops where they run once per item):
// at 88 KB it missed the instruction cache in 27% of its requests, and a step
// of a short item cost 2.7x what it does in a long one.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "../../include/pagedkv.h"
#include "pkv_decode_host.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace tree {
namespace {

constexpr int kBS = 16;
constexpr int kRows = 128;                    // query rows per tile: the MMA's M
constexpr int kStepBlocks = 8;                // blocks per step
constexpr int kStepKeys = kStepBlocks * kBS;  // 128 keys: the score MMA's N
// softmax: warp 4 + 4 wh + q takes rows (tensor-memory lanes) 32 q + 16 wh ..
// + 15, two threads per row: lanes 16 h + i take keys 64 h .. of a step and
// the head dimensions (D/2) h .. of O
constexpr int kSoftmaxWarp = 4;
constexpr int kSoftmaxWarps = 8;
constexpr int kHalfKeys = kStepKeys / 2;
constexpr int kConvertWarp = kSoftmaxWarp + kSoftmaxWarps;
constexpr int kConvertWarps = 4;
// tensor memory: O in columns [0, head_dim), two score buffers of 128 columns
// (and what Geo says)
constexpr int kTmemCols = 512;
constexpr int kTmemO = 0;
constexpr int kTmemS = 128;
// The largest weight where the reference is set, and the largest that it stays
// for (fp16 ends below 2^16).  The higher it is set, the less is lost at the low
// end and the sooner it moves: set at 0 (staying up to 8), 7, 11 and 13, 32
// sequences of 63 nodes with groups of 8 take 131.2, 130.9, 130.8 and 149.2 us,
// FP8 with 16 x 8000..32768 tokens 184.0, 182.2, 182.0 and 183.9.
constexpr float kSetLog2 = 11.f;
constexpr float kTopLog2 = 15.f;
constexpr int kFlagWords = PKV_MAX_TREE_NODES / 32;
constexpr int kFlagRing = 4;   // pieces whose flags are kept (see the softmax)
constexpr int kValidRing = 8;  // steps whose blocks' validity is kept (see the softmax)
constexpr int kScaleRing = 3;  // steps whose scales are kept (see the converters)
// Units of an item: its steps and kItemUnits for its start-up.  2, 3, 4, 5: 32
// sequences of 63 nodes with groups of 8 take 135.2, 131.5, 131.3, 132.9 us, over
// FP8 caches 191.4, 193.6, 197.0, 201.4; 64 ragged sequences of 16 nodes 100.1,
// 99.4, 99.7, 99.7, over FP8 caches 96.3, 97.3, 98.7, 99.9.
constexpr int kItemUnits = 3;
// merge: threads and rows of a block
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 16;
// Partial states in flight per thread: the more of them, the fewer round trips
// for an item cut into many pieces, but the fewer blocks per SM.
constexpr int kMergeFew = 4, kMergeMany = 8;

struct TreeParams {
    CUtensorMap tm_k;
    CUtensorMap tm_v;
    CUtensorMap tm_q;    // query rows: 128 bytes of each row of a 128-row tile
    CUtensorMap tm_q16;  // the same of 16 rows
    __half *out;
    const __half *q;
    const void *k_cache;
    const void *v_cache;
    const float *k_scale;  // FP8: [NB, 16, Hk]
    const float *v_scale;
    const int32_t *block_tables;
    const int32_t *seq_lens;
    const int32_t *query_start;
    const uint64_t *mask;
    int32_t mask_words;
    float scale_log2;     // |scale| log2(e), > 0: scores times this are in log2 units
    int32_t negate;       // the scale is negative: the MMA negates the scores
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t num_seqs;
    int32_t max_blocks;
    int32_t num_query_tokens;
    int32_t max_query_len;
    int32_t max_tiles;  // of a (sequence, KV head)
    int32_t max_seq_len;
    int64_t num_blocks;
    ErrorRecord *err;
    struct Border *borders;  // [CTAs]
    float2 *part_ml;         // [2 CTAs][128] (m, l)
    float4 *part_o;          // [2 CTAs][D / 4][128] four dims each
};

// What a stretch's first border says about the item it falls into.
struct Border {
    int32_t pieces;  // of the item; 0: the border cuts none, or is not the
                     // item's first border
    int32_t rows;    // query rows of the tile
    int32_t q0;      // first query token of the tile
    int32_t kvh;
};

// A piece as warp 0 hands it to the other warps: steps [step0, step0 + nsteps)
// of an item.
struct PieceHead {
    int seq, kvh, tile, step0;
    int nsteps, nblk, L, Q;
    int q0, slot, done, pad;  // slot: partial state, or -1 for a whole item
};
struct Piece : PieceHead {
    int ids[32];  // of the piece's first blocks (-1: none, or out of range)
};

template <int D, bool FP8>
struct Geo {
    static constexpr int kThreads = (kConvertWarp + (FP8 ? kConvertWarps : 0)) * 32;
    // Where shared memory's bandwidth counts (FP8: the codes are read and the
    // tiles written there too, 2030 cycles of a 128-key step's 2790), or tensor memory
    // has the columns, the query tile is copied to tensor memory once and the
    // score MMAs read the keys alone from shared memory.  FP8 with 128 dims
    // gives one of the two weight buffers (64 columns of fp16 pairs each) for
    // it.  (FP8, 16 x 8000..32768 tokens: 186.6 -> 183.8 us, 64 ragged ones 99.0
    // -> 97.3; 64 dims 37.9 -> 37.7, FP8 47.5 -> 47.1.  fp16 with 128 dims and
    // one weight buffer: 131 -> 148.)
    static constexpr bool kQTmem = FP8 || D == 64;
    [[maybe_unused]] static constexpr int kTmemQ = D == 64 ? 64 : 384;
    static constexpr int kPBuffers = kQTmem && D == 128 ? 1 : 2;
    static constexpr int kTmemP = kPBuffers == 1 ? 448 : 384;
    static constexpr int kPApart = 64 * (kPBuffers - 1);
    static constexpr int kChunks = D / 64;                // 128-byte chunks of a head row
    static constexpr int kQ = kChunks * kRows * 128;      // [chunk][row][128 B]
    // fp16 tiles, as the MMAs read them: keys [8 rows][chunk][row][128 B],
    // values [block][chunk][token][128 B]
    static constexpr int kK = kChunks * kStepKeys * 128;
    static constexpr int kVBlock = kChunks * kBS * 128;
    static constexpr int kV = kStepBlocks * kVBlock;
    // the rings the copies fill: fp16 tiles, or codes [block][token][D]
    static constexpr int kKStages = 3;
    static constexpr int kVStages = FP8 ? 2 : 3;
    static constexpr int kBlockBytes = kBS * D * (FP8 ? 1 : 2);
    static constexpr int kStage = kStepBlocks * kBlockBytes;
    static constexpr int kOffK = kQ;
    static constexpr int kOffV = kOffK + kKStages * kStage;
    // FP8: one fp16 key tile and two value tiles, and the scales
    static constexpr int kOffK16 = kOffV + kVStages * kStage;
    static constexpr int kOffV16 = kOffK16 + (FP8 ? kK : 0);
    static constexpr int kOffScale = kOffV16 + (FP8 ? 2 * kV : 0);  // [ring][k, v, log2 v][128]
    static constexpr int kOffBar = kOffScale + (FP8 ? kScaleRing * 3 * kStepKeys * 4 : 0);
    static constexpr int kBars = 4 + 2 + 2 * kKStages + 2 * kVStages + 8 + 1 + 3;
    static constexpr int kOffPiece = kOffBar + kBars * 8;
    static constexpr int kOffFlags = kOffPiece + 2 * static_cast<int>(sizeof(Piece));
    static constexpr int kOffValid = kOffFlags + kFlagRing * kFlagWords * 4;
    static constexpr int kOffTop = kOffValid + kValidRing * 4;  // [ring][4] largest value scale
    static constexpr int kOffMisc = kOffTop + kScaleRing * kConvertWarps * 4;
    static constexpr int kOffScan = (kOffMisc + 4 + 7) / 8 * 8;  // the prologue's words
    static constexpr int kBytes = kOffScan + (kThreads / 32 + 4) * 8;
    static_assert(kBytes + dec::kTileAlign <= dec::kSmemPerSM, "more than an SM's shared memory");
};

// mbarrier addresses (shared space) by role
template <int KS, int VS>
struct Bars {
    uint32_t b;
    __device__ uint32_t piece_full(int s) const { return b + 8 * s; }
    __device__ uint32_t piece_empty(int s) const { return b + 8 * (2 + s); }
    __device__ uint32_t q_full() const { return b + 8 * 4; }
    __device__ uint32_t q_empty() const { return b + 8 * 5; }
    __device__ uint32_t k_full(int s) const { return b + 8 * (6 + s); }
    __device__ uint32_t k_empty(int s) const { return b + 8 * (6 + KS + s); }
    static constexpr int kV0 = 6 + 2 * KS;
    __device__ uint32_t v_full(int s) const { return b + 8 * (kV0 + s); }
    __device__ uint32_t v_empty(int s) const { return b + 8 * (kV0 + VS + s); }
    static constexpr int kS0 = kV0 + 2 * VS;
    __device__ uint32_t s_full(int s) const { return b + 8 * (kS0 + s); }
    __device__ uint32_t s_free(int s) const { return b + 8 * (kS0 + 2 + s); }
    __device__ uint32_t p_full(int s) const { return b + 8 * (kS0 + 4 + s); }
    __device__ uint32_t pv_done(int s) const { return b + 8 * (kS0 + 6 + s); }
    __device__ uint32_t o_free() const { return b + 8 * (kS0 + 8); }
    __device__ uint32_t k16_full() const { return b + 8 * (kS0 + 9); }
    __device__ uint32_t v16_full(int s) const { return b + 8 * (kS0 + 10 + s); }
};

// Wait for phase `parity` of an mbarrier, giving up after about two seconds:
// one small loop (the timer is read every 64th time round).
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .u32 n, k;\n\t.reg .u64 t, t0;\n\t"
        "mov.u32 %0, 1;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "mov.u64 t0, %%globaltimer;\n\t"
        "mov.u32 n, 0;\n\t"
        "AGAIN:\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "add.u32 n, n, 1;\n\t"
        "and.b32 k, n, 63;\n\t"
        "setp.ne.u32 p, k, 0;\n\t"
        "@p bra AGAIN;\n\t"
        "mov.u64 t, %%globaltimer;\n\t"
        "sub.u64 t, t, t0;\n\t"
        "setp.lt.u64 p, t, 2000000000;\n\t"
        "@p bra AGAIN;\n\t"
        "mov.u32 %0, 0;\n\t"
        "DONE:\n\t}"
        : "=&r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Every lane waits; false if any lane gave up.  The long wait is a call: in
// line at every place it cost a batch of short items 14% (instruction fetches).
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bounded(bar, parity));
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_long(bar, parity);
}

__device__ __forceinline__ void tensor_g2s_2d(uint32_t dst, const void *tmap, int c0, int c1,
                                              uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tensor_g2s_4d(uint32_t dst, const void *tmap, int c0, int c1,
                                              int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// After tc::wait_ld: registers of a tensor-memory load hold their values from
// here on (nothing computed from them moves above this).
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31]));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of a value scale's size as the reference counts it: no less than -40 (448
// times a smaller one is nothing in fp16, and a weight, at most 2^15 2^40, can be
// summed in fp32) and up to 128 (a weight of 2^11 2^-128 is still normal).
__device__ __forceinline__ float scale_log2(float vs) {
    return __log2f(fmaxf(fabsf(vs), 0x1p-40f));
}

// Packed fp32 pairs (one instruction for two lanes' worth of fma, mul or add)
// and the three-input maximum.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f32x2_split(uint64_t r) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t pack_scaled(uint32_t a, uint32_t b, float f) {
    return pack_half2(__uint_as_float(a) * f, __uint_as_float(b) * f);
}

// Transposes 4 x 4 16-byte elements held by groups of four lanes: afterwards
// element c of lane t of a group is element t of the group's lane c.
__device__ __forceinline__ void lane_transpose4(uint4 (&x)[4], int lane) {
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & m) continue;
            uint4 &lo = x[i], &hi = x[i | m];
            uint4 s = up ? lo : hi;
            s.x = __shfl_xor_sync(0xffffffffu, s.x, m);
            s.y = __shfl_xor_sync(0xffffffffu, s.y, m);
            s.z = __shfl_xor_sync(0xffffffffu, s.z, m);
            s.w = __shfl_xor_sync(0xffffffffu, s.w, m);
            if (up) lo = s;
            else hi = s;
        }
    }
}

__device__ __forceinline__ void prefetch_l1(const void *p) {
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// The step a place `x` units into an item falls on.
__device__ __forceinline__ int step_at(int64_t x, int steps) {
    const int64_t s = x - kItemUnits;
    return s <= 0 ? 0 : s >= steps ? steps : static_cast<int>(s);
}

// First unit of CTA c's stretch, of `busy` = min(CTAs, units) that have one
// (so no stretch is empty).
__device__ __forceinline__ int64_t stretch(int64_t units, int c, int busy) {
    const int64_t n = units * c;  // (a 32-bit division where it does)
    return n >> 31 ? n / busy : static_cast<int64_t>(static_cast<uint32_t>(n) / busy);
}

struct SeqGeo {
    int L, Q, q0, tiles, steps;
};

// Up to 64 rows are laid out as four groups of 16, one in each quarter of the
// tile, so that every quarter of the SM has one softmax warp at work instead of
// half of them two (FP8, 64 rows, 16 x 8000..32768 tokens: 208 -> 198 us then).
__device__ __forceinline__ bool spread_rows(int rows) { return rows <= kRows / 2; }

__device__ __forceinline__ SeqGeo make_geo(int L, int Q, int q0, int G) {
    return SeqGeo{L, Q, q0, (Q * G + kRows - 1) / kRows, (L + kStepKeys - 1) / kStepKeys};
}

// Geometry of sequence s; false if it has no rows or is invalid (recorded when
// `report`).
__device__ __forceinline__ bool seq_geo(const TreeParams &p, int s, int G, bool report,
                                        SeqGeo &sg) {
    const int L = __ldg(p.seq_lens + s);
    const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1);
    const bool in = q0 >= 0 && q1 >= q0 && q1 <= p.num_query_tokens;  // (so q1 - q0 fits)
    const int Q = in ? q1 - q0 : 0;
    if (!in || L < Q || L > p.max_seq_len || L > static_cast<int64_t>(p.max_blocks) * kBS ||
        Q > p.max_query_len) {
        if (report) record_error(p.err, PKV_DEVERR_SEQ_LEN, s);
        return false;
    }
    sg = make_geo(L, Q, q0, G);
    return Q > 0;
}

// Units of one tile of a sequence, all its KV heads.
__device__ __forceinline__ int64_t tile_units(const SeqGeo &sg, int Hk) {
    return static_cast<int64_t>(Hk) * (sg.steps + kItemUnits);
}

// Sum over the CTA of v, and the exclusive prefix of this thread's (every
// thread calls; `sh` holds one word per warp); one_warp: over each warp, which
// all hold the same.
template <int kWarps>
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t *sh, bool one_warp, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (one_warp) {
        total = __shfl_sync(0xffffffffu, x, 31);
        return x - v;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int64_t y = sh[w];
        if (w < warp) before += y;
        total += y;
    }
    __syncthreads();
    return before + x - v;
}

// The visible keys of a row among kb .. kb + 63 as bits: the context (before
// ctx), then the drafted tokens of `mask` (null: none of them, nor of the
// context), up to the sequence's end.
__device__ __forceinline__ uint64_t visible(const uint64_t *mask, int words, int kb, int ctx,
                                            int L) {
    if (mask == nullptr) return 0;
    const int d = kb - ctx;
    uint64_t m;
    if (d <= -64) {
        m = ~0ull;
    } else if (d < 0) {
        m = ((1ull << -d) - 1) | (__ldg(mask) << -d);
    } else {
        const int w = d >> 6, sh = d & 63;
        m = w < words ? __ldg(mask + w) >> sh : 0ull;
        if (sh && w + 1 < words) m |= __ldg(mask + w + 1) << (64 - sh);
    }
    const int n = L - kb;
    return n >= 64 ? m : n <= 0 ? 0ull : m & ((1ull << n) - 1);
}

// Loads that are issued where they stand (a plain one may sink to its use).
__device__ __forceinline__ int load_early(const int32_t *p) {
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float load_early(const float *p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// Entry b of a sequence's block table as it stands: looked up ahead of its use,
// so that only checked_id, at the use, waits for it.
__device__ __forceinline__ int table_entry(const TreeParams &p, int seq, int b) {
    return load_early(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks + b);
}
__device__ __noinline__ void record_block(const TreeParams &p, int seq, int b) {
    record_error(p.err, PKV_DEVERR_BLOCK_ID, static_cast<int64_t>(seq) * p.max_blocks + b);
}
// The block id of entry b, or -1 when it is out of range (recorded when
// `report`).
__device__ __forceinline__ int checked_id(const TreeParams &p, int id, int seq, int b, bool report) {
    if (id >= 0 && static_cast<int64_t>(id) < p.num_blocks) return id;
    if (report) record_block(p, seq, b);
    return -1;
}
__device__ __forceinline__ int block_id(const TreeParams &p, int seq, int b, bool report) {
    return checked_id(p, table_entry(p, seq, b), seq, b, report);
}

// Walks a CTA's stretch.
struct Walk {
    int64_t u, u1;  // the next unit, the stretch's end
    SeqGeo sg;
    int tile, seq, kvh;  // the item (of n units) that u falls into
    int n, x;            // and u's place in it
};

// The next piece of the stretch (done: none is left), and lane l's id of its
// block l.  Out of line: called at two places, once per piece.
__device__ __noinline__ PieceHead next_piece(const TreeParams &p, Walk &w, int cta, int &id) {
    const int lane = threadIdx.x & 31;
    const int Hk = p.num_kv_heads, G = p.num_heads / Hk;
    PieceHead pc;
    pc.done = 1;
    id = -1;
    while (w.u < w.u1) {
        if (w.x == w.n) {  // the next item
            w.x = 0;
            if (++w.kvh == Hk) {  // of the next sequence with such a tile
                w.kvh = 0;
                uint32_t found = 0;
                for (int s0 = w.seq + 1; found == 0; s0 += 32) {
                    if (s0 >= p.num_seqs) {
                        s0 = 0;
                        ++w.tile;
                        if (w.tile >= p.max_tiles) return pc;  // (not reached: u1 is inside the list)
                    }
                    SeqGeo sg;
                    const bool has = s0 + lane < p.num_seqs &&
                                     seq_geo(p, s0 + lane, G, false, sg) && sg.tiles > w.tile;
                    found = __ballot_sync(0xffffffffu, has);
                    if (found != 0) {
                        const int src = __ffs(found) - 1;
                        w.seq = s0 + src;
                        w.sg = make_geo(__shfl_sync(0xffffffffu, sg.L, src),
                                        __shfl_sync(0xffffffffu, sg.Q, src),
                                        __shfl_sync(0xffffffffu, sg.q0, src), G);
                    }
                }
                w.n = w.sg.steps + kItemUnits;
            }
        }
        const int take = static_cast<int>(min(w.u1 - w.u, static_cast<int64_t>(w.n - w.x)));
        const int s0 = step_at(w.x, w.sg.steps), s1 = step_at(w.x + take, w.sg.steps);
        w.u += take;
        w.x += take;
        if (s1 == s0) continue;
        pc.seq = w.seq;
        pc.kvh = w.kvh;
        pc.tile = w.tile;
        pc.step0 = s0;
        pc.nsteps = s1 - s0;
        pc.nblk = min((w.sg.L + kBS - 1) / kBS - s0 * kStepBlocks, pc.nsteps * kStepBlocks);
        pc.L = w.sg.L;
        pc.Q = w.sg.Q;
        pc.q0 = w.sg.q0;
        pc.slot = s0 == 0 && s1 == w.sg.steps ? -1 : 2 * cta + (s0 == 0);
        pc.done = 0;
        if (lane < pc.nblk) id = block_id(p, w.seq, s0 * kStepBlocks + lane, true);
        break;
    }
    return pc;
}

// The fp16 pair w with infinities and NaN zeroed.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
    if ((w & 0x7C00u) == 0x7C00u) w &= 0xFFFF0000u;
    if ((w & 0x7C000000u) == 0x7C000000u) w &= 0x0000FFFFu;
    return w;
}
// Non-zero if one of eight fp16 is infinite or NaN: all ones in an exponent
// carry into its sign's place.
__device__ __forceinline__ uint32_t any_non_finite(const uint4 &x) {
    return (((x.x & 0x7C007C00u) + 0x04000400u) | ((x.y & 0x7C007C00u) + 0x04000400u) |
            ((x.z & 0x7C007C00u) + 0x04000400u) | ((x.w & 0x7C007C00u) + 0x04000400u)) &
           0x80008000u;
}
// A staged unit of eight values of row `key`: zero at and past the sequence's
// end; of a drafted row its finite elements, and the row flagged.
__device__ __forceinline__ uint4 clean_unit(uint4 x, int key, int ctx, int L, uint32_t *flags) {
    if (key >= L) return make_uint4(0u, 0u, 0u, 0u);
    if (key >= ctx && any_non_finite(x) != 0) {
        x = make_uint4(finite_halves(x.x), finite_halves(x.y), finite_halves(x.z),
                       finite_halves(x.w));
        atomicOr(&flags[(key - ctx) >> 5], 1u << ((key - ctx) & 31));
    }
    return x;
}

// Byte offset of 16-byte unit i (row-major) of a staged fp16 value tile whose
// order inside a row does not matter (the swizzle only permutes it).
template <int CH>
__device__ __forceinline__ int v_unit(int i) {
    const int t = i / (8 * CH), u = i % (8 * CH);
    return (t >> 4) * (CH * kBS * 128) + (u >> 3) * (kBS * 128) + (t & 15) * 128 + (u & 7) * 16;
}

// Cleans the value tile `vb` of a step that reaches past the context: its
// first `keys` keys, the first of them key0.  The softmax threads share it,
// kScan units in flight each.
template <int CH>
__device__ __noinline__ void clean_values(uint8_t *vb, int key0, int keys, int ctx, int L,
                                          uint32_t *flags) {
    constexpr int kUnits = 8 * CH;  // units of a row
    constexpr int kThreads = kSoftmaxWarps * 32;
    constexpr int kScan = 2;
    const int end = keys * kUnits;
    const int thread = threadIdx.x - kSoftmaxWarp * 32;
#pragma unroll 1
    for (int i0 = max(ctx - key0, 0) * kUnits + thread; i0 < end; i0 += kThreads * kScan) {
        uint4 x[kScan];
#pragma unroll
        for (int k = 0; k < kScan; ++k)
            x[k] = *reinterpret_cast<const uint4 *>(vb + v_unit<CH>(min(i0 + kThreads * k, end - 1)));
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            const int i = i0 + kThreads * k;
            const int key = key0 + i / kUnits;
            if (i < end && (key >= L || any_non_finite(x[k]) != 0))
                *reinterpret_cast<uint4 *>(vb + v_unit<CH>(i)) =
                    clean_unit(x[k], key, ctx, L, flags);
        }
    }
    fence_proxy_async_smem();
}

// Adds to a row's stored results the elements that were left out, where the
// row sees them: a weight times an infinity or a NaN is that, whatever the
// (positive) weight.  n results from dim d0 on: fp16 ones, or the fp32 ones of
// a partial state (groups of four dims, kRows groups apart).
template <int D, bool FP8>
__device__ __noinline__ void add_non_finite(const TreeParams &p, int seq, int kvh, int ctx, int Q,
                                            const uint32_t *flags, const uint64_t *mask, int d0,
                                            int n, __half *out, float *part) {
    for (int node = 0; node < Q; ++node) {
        if (!((flags[node >> 5] >> (node & 31)) & 1u) ||
            !((__ldg(mask + (node >> 6)) >> (node & 63)) & 1))
            continue;
        const int key = ctx + node;
        const int id = block_id(p, seq, key / kBS, false);
        if (id < 0) continue;
        const int64_t at =
            ((static_cast<int64_t>(id) * kBS + key % kBS) * p.num_kv_heads + kvh) * D + d0;
#pragma unroll 1
        for (int d = 0; d < n; ++d) {
            float x;
            if constexpr (FP8) {
                __nv_fp8_e4m3 c;
                c.__x = static_cast<const uint8_t *>(p.v_cache)[at + d];
                x = static_cast<float>(c) * __ldg(p.v_scale + at / D);
            } else {
                x = __half2float(static_cast<const __half *>(p.v_cache)[at + d]);
            }
            if (isfinite(x)) continue;
            if (out != nullptr) out[d] = __float2half_rn(__half2float(out[d]) + x);
            else part[(d >> 2) * (4 * kRows) + (d & 3)] += x;
        }
    }
}

// Sixteen E4M3 codes as fp16 (exact; the NaN code becomes a NaN).
__device__ __forceinline__ void codes_to_half(const uint4 &c, uint4 &lo, uint4 &hi) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(out[2 * i]), "=r"(out[2 * i + 1])
            : "r"(in[i]));
    }
    lo = make_uint4(out[0], out[1], out[2], out[3]);
    hi = make_uint4(out[4], out[5], out[6], out[7]);
}

// A step's codes (staged [block][token][D bytes], swizzled as D asks) as the
// fp16 key (V = false) or value tile, by the 128 converter threads.  Eight
// lanes take half a row each of two neighbouring rows, opposite halves, so
// that their reads and their writes fall on eight different 16-byte columns;
// a thread's units are whole blocks apart, their places constants apart.
// `clean`: the values of a step that reaches past the context.  (Two units at a
// time in a rolled loop: unrolled, 64 ragged FP8 sequences took 109 us instead
// of 97, for the instruction cache.)
template <int D, bool V>
__device__ __forceinline__ void convert_tile(const uint8_t *codes, uint8_t *tile, int keys,
                                             bool clean, int key0, int ctx, int L,
                                             uint32_t *flags) {
    constexpr int CH = D / 64;
    constexpr int kRowsApart = 32 / CH;                      // rows between a thread's units
    constexpr int kUnits = kStepKeys / kRowsApart;           // per thread
    constexpr int kTileApart = kRowsApart / kBS * CH * kBS * 128;
    const int tid = threadIdx.x - kConvertWarp * 32;
    const int p = tid & 7, g = tid >> 3;
    const int t = 2 * (g / CH) + (p >> 2);
    const int u = CH == 2 ? (p & 3) | (((p >> 2) ^ (g & 1)) << 2) : p & 3;
    const int su = D == 128 ? u ^ (t & 7) : u ^ ((t >> 1) & 3);
    const uint8_t *src = codes + t * D + su * 16;
    const int c = u >> 2, x = 2 * (u & 3);
    uint8_t *row = tile + (V ? (t >> 4) * (CH * kBS * 128) + c * (kBS * 128) + (t & 15) * 128
                             : (t >> 3) * (CH * 1024) + c * 1024 + (t & 7) * 128);
    uint8_t *d0 = row + ((x ^ (t & 7)) * 16), *d1 = row + (((x + 1) ^ (t & 7)) * 16);
    if (keys == kStepKeys && !clean) {
#pragma unroll 1
        for (int i0 = 0; i0 < kUnits; i0 += 2) {
            uint4 in[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                in[i] = *reinterpret_cast<const uint4 *>(src + (i0 + i) * kRowsApart * D);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 lo, hi;
                codes_to_half(in[i], lo, hi);
                *reinterpret_cast<uint4 *>(d0 + (i0 + i) * kTileApart) = lo;
                *reinterpret_cast<uint4 *>(d1 + (i0 + i) * kTileApart) = hi;
            }
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < kUnits && t + i * kRowsApart < keys; ++i) {
            uint4 lo, hi;
            codes_to_half(*reinterpret_cast<const uint4 *>(src + i * kRowsApart * D), lo, hi);
            if (clean) {
                lo = clean_unit(lo, key0 + t + i * kRowsApart, ctx, L, flags);
                hi = clean_unit(hi, key0 + t + i * kRowsApart, ctx, L, flags);
            }
            *reinterpret_cast<uint4 *>(d0 + i * kTileApart) = lo;
            *reinterpret_cast<uint4 *>(d1 + i * kTileApart) = hi;
        }
    }
    fence_proxy_async_smem();
}

// The walk of a stretch from what the prologue left in `start`: tile | sequence,
// the first unit of that sequence's tile, L | Q, q0.
__device__ __forceinline__ Walk walk_from(const volatile int64_t *start, int64_t u0, int64_t u1,
                                          int G) {
    Walk w;
    w.seq = static_cast<int>(start[0]);
    w.tile = static_cast<int>(start[0] >> 32);
    w.u = u0;
    w.u1 = u1;
    w.sg = make_geo(static_cast<int>(start[2] >> 32), static_cast<int>(start[2]),
                    static_cast<int>(start[3]), G);
    w.n = w.sg.steps + kItemUnits;
    const int64_t in = u0 - start[1];  // units from the tile's first
    if (in >> 31) {
        w.kvh = static_cast<int>(in / w.n);
        w.x = static_cast<int>(in - static_cast<int64_t>(w.kvh) * w.n);
    } else {
        w.kvh = static_cast<int>(in) / w.n;
        w.x = static_cast<int>(in) - w.kvh * w.n;
    }
    return w;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Geo<D, FP8>::kThreads, 1)
    tree_tile_kernel(const __grid_constant__ TreeParams p) {
    using Gm = Geo<D, FP8>;
    constexpr int CH = Gm::kChunks;
    constexpr int KS = Gm::kKStages, VS = Gm::kVStages;
    constexpr int DH = D / 2;  // the head dimensions (of O) each softmax thread owns
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((dec::kTileAlign - (smem_u32(smem_raw) & (dec::kTileAlign - 1))) &
                                (dec::kTileAlign - 1));
    const uint32_t sb = smem_u32(smem);
    const Bars<KS, VS> br{sb + Gm::kOffBar};
    Piece *pieces = reinterpret_cast<Piece *>(smem + Gm::kOffPiece);
    uint32_t *flags = reinterpret_cast<uint32_t *>(smem + Gm::kOffFlags);
    volatile uint32_t *valid = reinterpret_cast<volatile uint32_t *>(smem + Gm::kOffValid);
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + Gm::kOffMisc);
    int64_t *scan = reinterpret_cast<int64_t *>(smem + Gm::kOffScan);
    volatile int64_t *start = scan + Gm::kThreads / 32;  // tile | sequence, its first unit, L | Q, q0
    float *scales = reinterpret_cast<float *>(smem + Gm::kOffScale);
    float *tops = reinterpret_cast<float *>(smem + Gm::kOffTop);

    const int Hk = p.num_kv_heads, H = p.num_heads;
    const int G = H / Hk, logG = __ffs(G) - 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;
    if (threadIdx.x == 0) {
        // readers of a piece record: the value producer, the two MMA warps,
        // every softmax warp and every converter
        constexpr int kPieceReaders = 3 + kSoftmaxWarps + (FP8 ? kConvertWarps : 0);
        for (int s = 0; s < 2; ++s) {
            mbar_init(br.piece_full(s), 1);
            mbar_init(br.piece_empty(s), kPieceReaders);
            mbar_init(br.s_full(s), 2);
            mbar_init(br.s_free(s), kSoftmaxWarps);
            mbar_init(br.p_full(s), kSoftmaxWarps);
            mbar_init(br.pv_done(s), 2);
            mbar_init(br.v16_full(s), kConvertWarps);
        }
        mbar_init(br.q_full(), 1);
        mbar_init(br.q_empty(), 1);
        for (int s = 0; s < KS; ++s) {
            mbar_init(br.k_full(s), 1);
            mbar_init(br.k_empty(s), FP8 ? kConvertWarps : 1);
        }
        for (int s = 0; s < VS; ++s) {
            mbar_init(br.v_full(s), 1);
            mbar_init(br.v_empty(s), FP8 ? kConvertWarps : 1);
        }
        mbar_init(br.o_free(), kSoftmaxWarps);
        mbar_init(br.k16_full(), kConvertWarps);
        fence_mbarrier_init();
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_v);
        prefetch_tensormap(&p.tm_q);
    }
    if (threadIdx.x < kFlagRing * kFlagWords) flags[threadIdx.x] = 0;
    if (warp == 2) {
        tc::tmem_alloc(sb + Gm::kOffMisc, kTmemCols);
        tc::tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();  // the merge: it waits for this grid

    // ---- the list's length, and where this CTA's stretch starts: the thread
    // that holds the sequence its first unit falls into says so
    const bool one_go = p.num_seqs <= Gm::kThreads;  // a thread per sequence
    // a lane per sequence: each warp goes through them, without a barrier (8
    // sequences of three tiles 50.9 -> 50.2 us, one of 1041 tokens 10.2 -> 10.1)
    const bool one_warp = p.num_seqs <= 32;
    const int s_mine = one_warp ? lane : threadIdx.x;
    int64_t units = 0, before = 0;
    SeqGeo sg{};
#pragma unroll 1
    for (int s0 = 0; s0 < p.num_seqs; s0 += Gm::kThreads) {
        const int s = s0 + s_mine;
        if (!(s < p.num_seqs && seq_geo(p, s, G, cta == 0 && !(one_warp && warp != 0), sg)))
            sg.tiles = 0;
        int64_t total;
        before =
            cta_scan<Gm::kThreads / 32>(sg.tiles * tile_units(sg, Hk), scan, one_warp, total);
        units += total;
    }
    const int busy = static_cast<int>(min(static_cast<int64_t>(ctas), units));  // CTAs with a stretch
    const int64_t u0 = busy ? stretch(units, cta, busy) : 0;
    const int64_t u1 = busy ? stretch(units, cta + 1, busy) : 0;
    {
        int64_t run = 0;  // units of the tiles and sequences gone through
        const bool known = one_go && p.max_tiles == 1;  // the scan above found the places
#pragma unroll 1
        for (int tile = 0; tile < p.max_tiles && run <= u0 && cta < busy; ++tile) {
#pragma unroll 1
            for (int s0 = 0; s0 < p.num_seqs; s0 += Gm::kThreads) {
                const int s = s0 + s_mine;
                if (!one_go && !(s < p.num_seqs && seq_geo(p, s, G, false, sg))) sg.tiles = 0;
                const int64_t w = sg.tiles > tile ? tile_units(sg, Hk) : 0;
                int64_t total = units;
                if (!known) before = run + cta_scan<Gm::kThreads / 32>(w, scan, one_warp, total);
                if (w > 0 && before <= u0 && u0 < before + w && !(one_warp && warp != 0)) {
                    start[0] = static_cast<int64_t>(tile) << 32 | s;
                    start[1] = before;
                    start[2] = static_cast<int64_t>(sg.L) << 32 | static_cast<unsigned>(sg.Q);
                    start[3] = sg.q0;
                }
                run += total;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = misc[0];
    const bool busy_cta = cta < busy;
    if (!busy_cta && threadIdx.x == 0) p.borders[cta].pieces = 0;

    bool ok = busy_cta;  // false: a wait gave up
    if (warp < kSoftmaxWarp) {
        if (!busy_cta) {
        } else if (warp == 0) {
            // ========================= pieces and keys =========================
            Walk w = walk_from(start, u0, u1, G);
            int cur_ids;
            PieceHead cur = next_piece(p, w, cta, cur_ids);
            int gs = 0;  // steps staged
#pragma unroll 1
            for (int it = 0; ok; ++it) {
                const int rec = it & 1;
                if (it >= 2 && !wait_all(br.piece_empty(rec), ((it >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                pieces[rec].ids[lane] = cur_ids;
                if (lane == 0) static_cast<PieceHead &>(pieces[rec]) = cur;
                __syncwarp();
                if (lane == 0) mbar_arrive(br.piece_full(rec));
                if (cur.done) break;
                // the ids of 32 blocks at a time, one per lane, the next ones --
                // of this piece or the next -- looked up a window ahead
                const int b0 = cur.step0 * kStepBlocks;
                PieceHead nxt;
                int nxt_ids = -1, ids = cur_ids, ahead = -1;
#pragma unroll 1
                for (int n = 0; n < cur.nsteps; ++n, ++gs) {
                    const int ks = gs % KS;
                    const int at = n * kStepBlocks;
                    if ((at & 31) == 0) {
                        if (at != 0 && at + lane < cur.nblk)
                            ids = checked_id(p, ahead, cur.seq, b0 + at + lane, true);
                        const int b = at + 32 + lane;
                        if (b < cur.nblk) ahead = table_entry(p, cur.seq, b0 + b);
                    }
                    if (gs >= KS && !wait_all(br.k_empty(ks), ((gs / KS) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const int nb = min(kStepBlocks, cur.nblk - at);
                    // lane l: block l of the step (a bad block reads rows before
                    // the cache: zeros)
                    const int id = __shfl_sync(0xffffffffu, ids, (at & 31) + (lane & 7));
                    const uint32_t good = __ballot_sync(0xffffffffu, id >= 0 || lane >= nb);
                    if (lane == 0) {
                        valid[gs % kValidRing] = good;
                        mbar_arrive_expect_tx(br.k_full(ks), nb * Gm::kBlockBytes);
                    }
                    __syncwarp();
                    if (lane < nb) {
                        const uint32_t dst =
                            sb + Gm::kOffK + ks * Gm::kStage + lane * Gm::kBlockBytes;
                        if constexpr (FP8)
                            tensor_g2s_2d(dst, &p.tm_k, cur.kvh * D, id >= 0 ? id * kBS : -kBS,
                                          br.k_full(ks));
                        else
                            tensor_g2s_4d(dst, &p.tm_k, 0, 0, cur.kvh * CH, id >= 0 ? 2 * id : -2,
                                          br.k_full(ks));
                    }
                    // (when the ring is full: the look-ups wait for memory)
                    if (n == min(KS, cur.nsteps) - 1) nxt = next_piece(p, w, cta, nxt_ids);
                }
                cur = nxt;
                cur_ids = nxt_ids;
            }
            if (!ok) {
                // let the last copies land before the CTA can exit
#pragma unroll 1
                for (int s = 0; s < KS && s < gs; ++s) {
                    const int last = gs - 1 - ((gs - 1 - s) % KS);
                    wait_bounded(br.k_full(s), (last / KS) & 1);
                }
            }
        } else if (warp == 1) {
            // ============================== values ==============================
            int gs = 0;
#pragma unroll 1
            for (int it = 0; ok; ++it) {
                const int rec = it & 1;
                if (!wait_all(br.piece_full(rec), (it >> 1) & 1)) {
                    ok = false;
                    break;
                }
                const PieceHead pc = pieces[rec];
                int ids = pieces[rec].ids[lane], ahead = -1;
                __syncwarp();
                if (lane == 0) mbar_arrive(br.piece_empty(rec));
                if (pc.done) break;
                const int b0 = pc.step0 * kStepBlocks;
#pragma unroll 1
                for (int n = 0; n < pc.nsteps; ++n, ++gs) {
                    const int vs = gs % VS;
                    const int at = n * kStepBlocks;
                    if ((at & 31) == 0) {
                        if (at != 0 && at + lane < pc.nblk)
                            ids = checked_id(p, ahead, pc.seq, b0 + at + lane, false);
                        const int b = at + 32 + lane;
                        if (b < pc.nblk) ahead = table_entry(p, pc.seq, b0 + b);
                    }
                    if (gs >= VS && !wait_all(br.v_empty(vs), ((gs / VS) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const int nb = min(kStepBlocks, pc.nblk - at);
                    if (lane == 0) mbar_arrive_expect_tx(br.v_full(vs), nb * Gm::kBlockBytes);
                    __syncwarp();
                    const int id = __shfl_sync(0xffffffffu, ids, (at & 31) + (lane & 7));
                    if (lane < nb) {
                        const uint32_t dst =
                            sb + Gm::kOffV + vs * Gm::kStage + lane * Gm::kBlockBytes;
                        if constexpr (FP8)
                            tensor_g2s_2d(dst, &p.tm_v, pc.kvh * D, id >= 0 ? id * kBS : -kBS,
                                          br.v_full(vs));
                        else
                            tensor_g2s_3d(dst, &p.tm_v, 0, id >= 0 ? id * kBS : -kBS, pc.kvh * CH,
                                          br.v_full(vs));
                    }
                }
            }
            if (!ok) {
#pragma unroll 1
                for (int s = 0; s < VS && s < gs; ++s) {
                    const int last = gs - 1 - ((gs - 1 - s) % VS);
                    wait_bounded(br.v_full(s), (last / VS) & 1);
                }
            }
        } else if (warp == 2) {
            // ==================== query tiles and score MMAs ====================
            int gs = 0, q_staged = 0;
#pragma unroll 1
            for (int it = 0; ok; ++it) {
                const int rec = it & 1;
                if (!wait_all(br.piece_full(rec), (it >> 1) & 1)) {
                    ok = false;
                    break;
                }
                const PieceHead pc = pieces[rec];
                __syncwarp();
                if (lane == 0) mbar_arrive(br.piece_empty(rec));
                if (pc.done) break;
                // the query tile, once the previous piece's last scores are done, or
                // it is in tensor memory
                if (it >= 1) ok = wait_all(br.q_empty(), (it - 1) & 1);
                if (!ok) break;
                if (lane == 0)
                    mbar_arrive_expect_tx(br.q_full(), spread_rows(pc.Q * G) ? Gm::kQ / 2 : Gm::kQ);
                __syncwarp();
                if (spread_rows(pc.Q * G)) {  // sixteen rows to each 32 of the tile
                    const int c = lane >> 2, k = lane & 3;
                    if (lane < 4 * CH)
                        tensor_g2s_3d(sb + c * (kRows * 128) + k * (32 * 128), &p.tm_q16, 128 * c,
                                      pc.kvh * G, pc.q0 + k * (16 >> logG), br.q_full());
                } else if (lane < CH) {
                    tensor_g2s_3d(sb + lane * (kRows * 128), &p.tm_q, 128 * lane, pc.kvh * G,
                                  pc.q0 + pc.tile * (kRows >> logG), br.q_full());
                }
                q_staged = it + 1;
                ok = wait_all(br.q_full(), it & 1);
                if constexpr (Gm::kQTmem) {
                    // (the previous piece's last scores are done with the last one)
                    if (ok && gs >= 1) ok = wait_all(br.s_full((gs - 1) & 1), ((gs - 1) >> 1) & 1);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (lane == 0) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc::cp_128x256b(tmem + Gm::kTmemQ + 8 * kk,
                                            tc::smem_desc(sb + (kk >> 2) * (kRows * 128) +
                                                              (kk & 3) * 32,
                                                          16, 1024, tc::kSwizzle128B));
                        tc::commit(br.q_empty());
                    }
                    __syncwarp();
                }
#pragma unroll 1
                for (int n = 0; n < pc.nsteps && ok; ++n, ++gs) {
                    const int ks = gs % KS, b = gs & 1;
                    ok = FP8 ? wait_all(br.k16_full(), gs & 1)
                             : wait_all(br.k_full(ks), (gs / KS) & 1);
                    // the softmax has read the scores of two steps back
                    if (ok && gs >= 2) ok = wait_all(br.s_free(b), ((gs >> 1) - 1) & 1);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (lane == 0) {
                        const int nb = min(kStepBlocks, pc.nblk - n * kStepBlocks);
                        // (bit 13: A is negated)
                        const uint32_t idesc = tc::idesc_f16_f32(kRows, nb * kBS, false, false) |
                                               (static_cast<uint32_t>(p.negate) << 13);
                        const uint32_t k_s =
                            sb + (FP8 ? Gm::kOffK16 : Gm::kOffK + ks * Gm::kStage);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t k_desc =
                                tc::smem_desc(k_s + (kk >> 2) * 1024 + (kk & 3) * 32, 16, CH * 1024,
                                              tc::kSwizzle128B);
                            if constexpr (Gm::kQTmem)
                                tc::mma_ts(tmem + kTmemS + 128 * b, tmem + Gm::kTmemQ + 8 * kk,
                                           k_desc, idesc, kk > 0);
                            else
                                tc::mma_ss(tmem + kTmemS + 128 * b,
                                           tc::smem_desc(sb + (kk >> 2) * (kRows * 128) +
                                                             (kk & 3) * 32,
                                                         16, 1024, tc::kSwizzle128B),
                                           k_desc, idesc, kk > 0);
                        }
                        tc::commit(br.s_full(b));
                        mbar_arrive(br.s_full(b));  // passes the step's validity and scales on
                        if (!FP8) tc::commit(br.k_empty(ks));
                        if (!Gm::kQTmem && n == pc.nsteps - 1) tc::commit(br.q_empty());
                    }
                    __syncwarp();
                }
            }
            if (!ok) {
                if (q_staged) wait_bounded(br.q_full(), (q_staged - 1) & 1);
            }
        } else {
            // ============================= P V MMAs =============================
            constexpr uint32_t kIdescPV = tc::idesc_f16_f32(kRows, D, false, true);
            // the border at u0, for the merge (every CTA writes one, whether or
            // not its stretch holds a step)
            if (lane == 0) {
                const Walk w = walk_from(start, u0, u1, G);
                Border border;
                const int64_t a = u0 - w.x;  // the item's first unit
                const bool cuts = cta > 0 && step_at(w.x, w.sg.steps) > 0 &&
                                  step_at(stretch(units, cta - 1, busy) - a, w.sg.steps) == 0;
                // pieces: the CTA before this one, and those up to the item's last unit
                border.pieces =
                    cuts ? static_cast<int>(((a + w.n) * busy - 1) / units) - (cta - 1) + 1 : 0;
                border.rows = min(kRows, w.sg.Q * G - w.tile * kRows);
                border.q0 = w.sg.q0 + w.tile * (kRows >> logG);
                border.kvh = w.kvh;
                p.borders[cta] = border;
            }
            __syncwarp();
            int gs = 0;
#pragma unroll 1
            for (int it = 0; ok; ++it) {
                const int rec = it & 1;
                if (!wait_all(br.piece_full(rec), (it >> 1) & 1)) {
                    ok = false;
                    break;
                }
                const PieceHead pc = pieces[rec];
                __syncwarp();
                if (lane == 0) mbar_arrive(br.piece_empty(rec));
                if (pc.done) break;
#pragma unroll 1
                for (int n = 0; n < pc.nsteps && ok; ++n, ++gs) {
                    const int vs = gs % VS, b = gs & 1;
                    const int nb = min(kStepBlocks, pc.nblk - n * kStepBlocks);
                    // the previous piece's O has been read
                    if (n == 0 && it > 0) ok = wait_all(br.o_free(), (it - 1) & 1);
                    if (ok)
                        ok = FP8 ? wait_all(br.v16_full(b), (gs >> 1) & 1)
                                 : wait_all(br.v_full(vs), (gs / VS) & 1);
                    if (ok) ok = wait_all(br.p_full(b), (gs >> 1) & 1);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (lane == 0) {
                        const uint32_t v_s =
                            sb + (FP8 ? Gm::kOffV16 + b * Gm::kV : Gm::kOffV + vs * Gm::kStage);
#pragma unroll 1
                        for (int k = 0; k < nb; ++k)
                            tc::mma_ts(tmem + kTmemO, tmem + Gm::kTmemP + Gm::kPApart * b + 8 * k,
                                       tc::smem_desc(v_s + k * Gm::kVBlock, kBS * 128, 1024,
                                                     tc::kSwizzle128B),
                                       kIdescPV, (n > 0 || k > 0) ? 1u : 0u);
                        tc::commit(br.pv_done(b));
                        mbar_arrive(br.pv_done(b));  // passes the piece's flags on
                        if (!FP8) tc::commit(br.v_empty(vs));
                    }
                    __syncwarp();
                }
            }
        }
    } else if (FP8 && warp >= kConvertWarp) {
        // ========================= codes to fp16 tiles =========================
        // Thread i also looks up key i's scales: its block id two steps ahead,
        // the scales one step ahead.
        const int tid = threadIdx.x - kConvertWarp * 32;
        int gs = 0;
#pragma unroll 1
        for (int it = 0; ok; ++it) {
            const int rec = it & 1;
            if (!wait_all(br.piece_full(rec), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const PieceHead pc = pieces[rec];
            const int b_key = tid / kBS;  // block of this thread's key in a step
            const int id0 = pieces[rec].ids[b_key], id1 = pieces[rec].ids[kStepBlocks + b_key];
            __syncwarp();
            if (lane == 0) mbar_arrive(br.piece_empty(rec));
            if (pc.done) break;
            const int ctx = pc.L - pc.Q;
            uint32_t *my_flags = flags + (it % kFlagRing) * kFlagWords;
            const int64_t off = static_cast<int64_t>(tid % kBS) * Hk + pc.kvh;
            // the scales of key tid of step n, whose block is id; 0: no such key
            auto scale_of = [&](const float *scale, int id, int n) {
                return id >= 0 && (pc.step0 + n) * kStepKeys + tid < pc.L
                           ? load_early(scale + static_cast<int64_t>(id) * kBS * Hk + off)
                           : 0.f;
            };
            float ks = scale_of(p.k_scale, id0, 0), vs = scale_of(p.v_scale, id0, 0);
            int entry = pc.nsteps > 1 ? id1 : -1;  // of this key's block of the next step
#pragma unroll 1
            for (int n = 0; n < pc.nsteps && ok; ++n, ++gs) {
                const int b = gs & 1, kst = gs % KS, vst = gs % VS;
                const int nb = min(kStepBlocks, pc.nblk - n * kStepBlocks);
                const int key0 = (pc.step0 + n) * kStepKeys;
                // keys, once the scores of the step before are done with the
                // tile.  (The softmax is then past the scales kScaleRing steps
                // back: the values of the step before were not converted until
                // the P V of three steps back was done.)
                ok = wait_all(br.k_full(kst), (gs / KS) & 1);
                if (ok && gs >= 1) ok = wait_all(br.s_full(b ^ 1), ((gs - 1) >> 1) & 1);
                if (!ok) break;
                {
                    const int ring = gs % kScaleRing;
                    // (the dot product with a key of infinities is NaN, but its
                    // dot product with the codes times infinity need not be)
                    scales[ring * 3 * kStepKeys + tid] = isfinite(ks) ? ks * p.scale_log2 : NAN;
                    // (a drafted row's scale that is not finite counts as its
                    // non-finite elements do: left out here, added at the end)
                    const bool out = !isfinite(vs) && tid + key0 >= ctx;
                    scales[ring * 3 * kStepKeys + kStepKeys + tid] = out ? 0.f : vs;
                    scales[ring * 3 * kStepKeys + 2 * kStepKeys + tid] =
                        scale_log2(isfinite(vs) ? vs : 0.f);
                    // (the bits of non-negative floats order as they do)
                    const uint32_t top = __reduce_max_sync(
                        0xffffffffu, isfinite(vs) ? __float_as_uint(fabsf(vs)) : 0u);
                    if (lane == 0) tops[ring * kConvertWarps + warp - kConvertWarp] = __uint_as_float(top);
                }
                const bool left_out = !isfinite(vs);
                // the next step's scales, and the one's block after it (after
                // this step's have been used: waiting for a load waits for the
                // ones issued since)
                {
                    const int id_next = checked_id(p, entry, 0, 0, false);
                    ks = scale_of(p.k_scale, id_next, n + 1);
                    vs = scale_of(p.v_scale, id_next, n + 1);
                    const int b2 = (n + 2) * kStepBlocks + b_key;
                    entry = -1;
                    if (b2 < pc.nblk) entry = table_entry(p, pc.seq, pc.step0 * kStepBlocks + b2);
                }
                convert_tile<D, false>(smem + Gm::kOffK + kst * Gm::kStage, smem + Gm::kOffK16,
                                       nb * kBS, false, key0, ctx, pc.L, nullptr);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(br.k16_full());
                    mbar_arrive(br.k_empty(kst));
                }
                // values, once the P V of two steps back is done with the tile
                ok = wait_all(br.v_full(vst), (gs / VS) & 1);
                if (ok && gs >= 2) ok = wait_all(br.pv_done(b), ((gs >> 1) - 1) & 1);
                if (!ok) break;
                const bool tail = key0 + kStepKeys > ctx;
                if (tail && tid + key0 >= ctx && left_out)  // (its stored scale is 0)
                    atomicOr(&my_flags[(tid + key0 - ctx) >> 5], 1u << ((tid + key0 - ctx) & 31));
                convert_tile<D, true>(smem + Gm::kOffV + vst * Gm::kStage,
                                      smem + Gm::kOffV16 + b * Gm::kV, nb * kBS, tail, key0, ctx,
                                      pc.L, my_flags);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(br.v16_full(b));
                    mbar_arrive(br.v_empty(vst));
                }
            }
        }
    } else {
        // =============================== softmax ===============================
        const int wh = (warp - kSoftmaxWarp) >> 2;
        const int quarter = warp & 3;
        const int h = lane >> 4;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32 + wh * 16) << 16);
        int gs = 0;
#pragma unroll 1
        for (int it = 0; ok; ++it) {
            const int rec = it & 1;
            if (!wait_all(br.piece_full(rec), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const PieceHead pc = pieces[rec];
            __syncwarp();
            if (lane == 0) mbar_arrive(br.piece_empty(rec));
            if (pc.done) break;
            const int ctx = pc.L - pc.Q;
            // the tile's row of this warp's first lane (past the tile: none)
            const int r0 = !spread_rows(pc.Q * G) ? quarter * 32 + wh * 16
                           : wh == 0              ? quarter * 16
                                                  : kRows;
            const int r = r0 + (lane & 15);
            const int rr = pc.tile * kRows + r;
            const bool row_ok = rr < pc.Q * G;
            const bool live = __any_sync(0xffffffffu, row_ok);
            const uint64_t *mask =
                row_ok ? p.mask + static_cast<int64_t>(pc.q0 + (rr >> logG)) * p.mask_words
                       : nullptr;
            // bring the row's mask near, for the step that needs it
            if (row_ok) prefetch_l1(mask);
            uint32_t *my_flags = flags + (it % kFlagRing) * kFlagWords;
            float m_used = -INFINITY, l = 0.f;  // l: this thread's keys only

#pragma unroll 1
            for (int n = 0; n < pc.nsteps; ++n, ++gs) {
                const int sbuf = gs & 1;
                const int key0 = (pc.step0 + n) * kStepKeys;
                const bool tail = key0 + kStepKeys > ctx;
                uint64_t vis = ~0ull;
                if (tail) {
                    if constexpr (!FP8) {
                        const int vs = gs % VS;
                        if (!wait_all(br.v_full(vs), (gs / VS) & 1)) {
                            ok = false;
                            break;
                        }
                        clean_values<CH>(smem + Gm::kOffV + vs * Gm::kStage, key0,
                                         min(kStepBlocks, pc.nblk - n * kStepBlocks) * kBS, ctx,
                                         pc.L, my_flags);
                        __syncwarp();
                    }
                    vis = visible(mask, p.mask_words, key0 + kHalfKeys * h, ctx, pc.L);
                }
                if (!wait_all(br.s_full(sbuf), (gs >> 1) & 1)) {
                    ok = false;
                    break;
                }
                if (!live) {
                    // (its rows of the weight buffer hold anything: they reach
                    // its rows of O alone; it keeps pace with the other warps,
                    // or its arrivals would count for their earlier steps)
                    if (lane == 0) mbar_arrive(br.s_free(sbuf));
                    if (gs >= 2 && !wait_all(br.pv_done(sbuf), ((gs >> 1) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive(br.p_full(sbuf));
                    continue;
                }
                tc::fence_after_sync();
                uint32_t sx[kHalfKeys];  // this row's scores of this thread's keys (fp32 bits)
#pragma unroll
                for (int c = 0; c < kHalfKeys / 32; ++c)
                    tc::ld32_halves<kHalfKeys>(tl + kTmemS + 128 * sbuf + 32 * c,
                                               *reinterpret_cast<uint32_t(*)[32]>(sx + 32 * c));
                // the step's blocks that are in range: the key producer's word
                // (the ring is longer than it can be ahead: it stages at most
                // three steps past the scores, and these are at most two ahead
                // of this warp)
                const uint32_t blocks = valid[gs % kValidRing];
                tc::wait_ld();
                landed(*reinterpret_cast<uint32_t(*)[32]>(sx));
                landed(*reinterpret_cast<uint32_t(*)[32]>(sx + 32));
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(br.s_free(sbuf));
                const float *sc = scales + (gs % kScaleRing) * 3 * kStepKeys + kHalfKeys * h;
                float top2 = 0.f;  // log2 of the step's largest value scale
                if constexpr (FP8) {
                    const float *t = tops + (gs % kScaleRing) * kConvertWarps;
                    top2 = scale_log2(fmaxf(fmax3(t[0], t[1], t[2]), t[3]));
#pragma unroll
                    for (int e = 0; e < kHalfKeys; e += 4) {
                        const float4 k4 = *reinterpret_cast<const float4 *>(sc + e);
                        const float2 a = f32x2_split(mul_f32x2(
                            f32x2(__uint_as_float(sx[e]), __uint_as_float(sx[e + 1])), f32x2(k4.x, k4.y)));
                        const float2 b = f32x2_split(mul_f32x2(
                            f32x2(__uint_as_float(sx[e + 2]), __uint_as_float(sx[e + 3])), f32x2(k4.z, k4.w)));
                        sx[e] = __float_as_uint(a.x);
                        sx[e + 1] = __float_as_uint(a.y);
                        sx[e + 2] = __float_as_uint(b.x);
                        sx[e + 3] = __float_as_uint(b.y);
                    }
                }
                // to log2 units, rounded before anything is subtracted: a reference
                // made from a rounded score differs from it exactly, where one that
                // is rounded on its own is off by up to 2^12 at scores of 2^36, more
                // than the weights' range (with the subtraction in one fma instead,
                // which outputs zeros from 2^28 on: 32 x 63 nodes 130.5 against
                // 130.6 us, 128 x 300 tokens 40.2 and 41.0, 64 dims 37.6 and 38.4;
                // FP8, where the key's scale holds the factor, 182.4 and 184.1)
                if constexpr (!FP8) {
                    const uint64_t f2 = f32x2(p.scale_log2, p.scale_log2);
#pragma unroll
                    for (int e = 0; e < kHalfKeys; e += 2) {
                        const float2 a = f32x2_split(mul_f32x2(
                            f32x2(__uint_as_float(sx[e]), __uint_as_float(sx[e + 1])), f2));
                        sx[e] = __float_as_uint(a.x);
                        sx[e + 1] = __float_as_uint(a.y);
                    }
                }
                const bool masked = tail || blocks != 0xffffffffu;
                if (masked) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (!((blocks >> (4 * h + b)) & 1u)) vis &= ~(0xFFFFull << (16 * b));
                    const uint32_t v0 = static_cast<uint32_t>(vis), v1 = static_cast<uint32_t>(vis >> 32);
#pragma unroll
                    for (int e = 0; e < kHalfKeys; ++e)
                        if (!((e < 32 ? v0 : v1) & (1u << (e & 31)))) sx[e] = 0xFF800000u;  // -inf
                }
                float mr[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mr[i] = -INFINITY;
#pragma unroll
                for (int e = 0; e < kHalfKeys / 2; ++e)
                    mr[e & 7] = fmax3(mr[e & 7], __uint_as_float(sx[2 * e]),
                                      __uint_as_float(sx[2 * e + 1]));
                const float mx = fmax3(fmax3(mr[0], mr[1], mr[2]), fmax3(mr[3], mr[4], mr[5]),
                                       fmaxf(mr[6], mr[7]));
                // the row's other half: the thread 16 lanes away
                const float mo = __shfl_xor_sync(0xffffffffu, mx, 16);
                float m_new = fmaxf(mx, mo) + top2;
                // (rounded down, and the reference up: fp16 holds every weight)
                const float bound = __fadd_rd(m_used, kTopLog2);
                bool raise = m_new > bound;
                if constexpr (FP8) {
                    // the largest scale need not be at a key that the row sees,
                    // nor at one with weight: the largest product itself
                    if (__any_sync(0xffffffffu, raise)) {
                        float ex = -INFINITY, ey = -INFINITY;
#pragma unroll
                        for (int e = 0; e < kHalfKeys; e += 4) {
                            const float4 lv =
                                *reinterpret_cast<const float4 *>(sc + 2 * kStepKeys + e);
                            const float2 a = f32x2_split(
                                add_f32x2(f32x2(__uint_as_float(sx[e]), __uint_as_float(sx[e + 1])),
                                          f32x2(lv.x, lv.y)));
                            const float2 b = f32x2_split(add_f32x2(
                                f32x2(__uint_as_float(sx[e + 2]), __uint_as_float(sx[e + 3])),
                                f32x2(lv.z, lv.w)));
                            ex = fmax3(ex, a.x, a.y);
                            ey = fmax3(ey, b.x, b.y);
                        }
                        ex = fmaxf(ex, ey);
                        ex = fmaxf(ex, __shfl_xor_sync(0xffffffffu, ex, 16));
                        m_new = ex;
                        raise = m_new > bound;
                    }
                }
                // O holds this piece's earlier steps relative to m_used: rescale
                // this thread's columns before the reference moves (the
                // previous P V done first)
                m_new = __fsub_ru(m_new, kSetLog2);
                const bool resc = raise && n > 0 && m_used != -INFINITY;
                if (__any_sync(0xffffffffu, resc)) {
                    if (!wait_all(br.pv_done((gs - 1) & 1), ((gs - 1) >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const float alpha = resc ? ex2(m_used - m_new) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < DH / 32; ++c) {
                        uint32_t x[32];
                        tc::ld32_halves<DH>(tl + kTmemO + 32 * c, x);
                        tc::wait_ld();
                        landed(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
                        tc::st32_halves<DH>(tl + kTmemO + 32 * c, x);
                    }
                    tc::wait_st();
                    l *= alpha;
                }
                if (raise) m_used = m_new;
                const float ms = m_used == -INFINITY ? 0.f : m_used;
                // weights 2^(s - m), fp16 pairs; the P V of as many steps back as
                // there are buffers is done with this one
                if (gs >= Gm::kPBuffers) {
                    const int last = gs - Gm::kPBuffers;
                    if (!wait_all(br.pv_done(last & 1), (last >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                }
                const uint64_t nms2 = f32x2(-ms, -ms);
                uint64_t l2[4] = {0ull, 0ull, 0ull, 0ull};
                uint32_t x[32];
                float4 v4;  // FP8: the value scales of four keys
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 t = f32x2_split(add_f32x2(
                        f32x2(__uint_as_float(sx[2 * e]), __uint_as_float(sx[2 * e + 1])), nms2));
                    float p0 = ex2(t.x), p1 = ex2(t.y);
                    l2[e & 3] = add_f32x2(l2[e & 3], f32x2(p0, p1));
                    if constexpr (FP8) {
                        if ((e & 1) == 0) v4 = *reinterpret_cast<const float4 *>(sc + kStepKeys + 2 * e);
                        const float2 w = f32x2_split(mul_f32x2(
                            f32x2(p0, p1), (e & 1) ? f32x2(v4.z, v4.w) : f32x2(v4.x, v4.y)));
                        p0 = w.x;
                        p1 = w.y;
                    }
                    x[e] = pack_half2(p0, p1);
                }
                tc::st32_halves<32>(tl + Gm::kTmemP + Gm::kPApart * sbuf, x);
                const float2 la =
                    f32x2_split(add_f32x2(add_f32x2(l2[0], l2[1]), add_f32x2(l2[2], l2[3])));
                l += la.x + la.y;
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(br.p_full(sbuf));
            }
            if (!ok) break;

            // ---- the piece's output: O / l, or the partial state (m, l, O),
            // this thread's head dimensions
            if (!wait_all(br.pv_done((gs - 1) & 1), ((gs - 1) >> 1) & 1)) {
                ok = false;
                break;
            }
            // The flags of the piece three ahead, whose first ones are set after
            // every warp has read this piece's O (o_free, before the next piece's
            // first P V, before its values or the third piece's are cleaned).
            // Their buffer held the piece before this one's: read by every warp
            // before this piece's first P V.
            if (warp == kSoftmaxWarp && lane < kFlagWords)
                flags[(it + 3) % kFlagRing * kFlagWords + lane] = 0;
            __syncwarp();
            if (live) {
                tc::fence_after_sync();
                uint32_t any = 0;
#pragma unroll
                for (int w = 0; w < kFlagWords; ++w) any |= my_flags[w];
                l += __shfl_xor_sync(0xffffffffu, l, 16);  // the row's sum over both halves' keys
                const bool whole = pc.slot < 0;
                const float inv = l > 0.f ? 1.f / l : l;  // (nothing visible: 0; NaN stays)
                if (!whole && h == 0 && row_ok)
                    p.part_ml[static_cast<int64_t>(pc.slot) * kRows + r] = make_float2(m_used, l);
#pragma unroll 1
                for (int k = 0; k < DH / 32; ++k) {  // 32 dims at a time
                    uint32_t o[32];
                    tc::ld32_halves<DH>(tl + kTmemO + 32 * k, o);
                    tc::wait_ld();
                    landed(o);
                    if (whole) {
                        // exchanged inside groups of four lanes, so that a store
                        // of the warp covers 64 bytes of eight rows (16 bytes of
                        // 32 rows each: 3 us for an item's outputs)
                        uint4 x[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            x[c] = make_uint4(pack_scaled(o[8 * c], o[8 * c + 1], inv),
                                              pack_scaled(o[8 * c + 2], o[8 * c + 3], inv),
                                              pack_scaled(o[8 * c + 4], o[8 * c + 5], inv),
                                              pack_scaled(o[8 * c + 6], o[8 * c + 7], inv));
                        lane_transpose4(x, lane);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int src = (lane & ~3) + c;  // the lane the row came from
                            const int row = pc.tile * kRows + r0 + (src & 15);
                            if (row < pc.Q * G)
                                *reinterpret_cast<uint4 *>(
                                    p.out +
                                    (static_cast<int64_t>(pc.q0 + (row >> logG)) * H + pc.kvh * G +
                                     (row & (G - 1))) * D +
                                    DH * (src >> 4) + 32 * k + 8 * (lane & 3)) = x[c];
                        }
                    } else if (row_ok) {
                        // the rows of a half-warp side by side
                        uint4 *dst = reinterpret_cast<uint4 *>(p.part_o) +
                                     (static_cast<int64_t>(pc.slot) * (D / 4) +
                                      (DH * h + 32 * k) / 4) * kRows + r;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            dst[c * kRows] =
                                make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (any != 0 && row_ok)
                    add_non_finite<D, FP8>(
                        p, pc.seq, pc.kvh, ctx, pc.Q, my_flags, mask, DH * h, DH,
                        whole ? p.out + (static_cast<int64_t>(pc.q0 + (rr >> logG)) * H +
                                         pc.kvh * G + (rr & (G - 1))) * D + DH * h
                              : nullptr,
                        reinterpret_cast<float *>(p.part_o) +
                            ((static_cast<int64_t>(pc.slot) * (D / 4) + DH * h / 4) * kRows + r) * 4);
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(br.o_free());
        }
    }

    if (busy_cta && !ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, cta);
    // every role is done: hand the tensor memory back
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// Merges the partial states of the items that stretch borders cut: block
// (b, y) takes rows kMergeRows y .. of the item that border b + 1 is the first
// to cut.  The item's first piece is the last one of CTA b (its second slot),
// the others the first ones of the CTAs that follow.  A thread takes one row
// and D/4 / 16 groups of four dims, rows side by side as the states lie; the
// result is turned round in shared memory for whole rows of output.  Bound:
// the latency of loads out of L2, so two pieces are asked for before the
// border is known and PIECES at a time after that, the running maximum and sum
// kept as in the tile kernel (maxima first, then four pieces at a time: 2 us
// more for one sequence cut into 19 pieces).
template <int D, int PIECES>
__global__ void __launch_bounds__(kMergeThreads, PIECES == kMergeFew ? 4 : 2)
    tree_merge_kernel(const __grid_constant__ TreeParams p) {
    constexpr int kGroups = kMergeThreads / kMergeRows;  // threads per row
    constexpr int NQ = D / 4 / kGroups;                  // groups of four dims per thread
    __shared__ uint2 turned[kMergeRows][D / 4 + 1];
    // the kernel launched next may start: this one and the tile kernel write
    // the outputs and the workspace alone
    grid_launch_dependents();
    grid_dependency_wait();
    const int c0 = blockIdx.x;
    const int row0 = blockIdx.y * kMergeRows;
    const int rl = threadIdx.x % kMergeRows, g = threadIdx.x / kMergeRows;
    const float2 *ml0 = p.part_ml + static_cast<int64_t>(2 * c0) * kRows + row0 + rl;
    const float4 *o0 = p.part_o + (static_cast<int64_t>(2 * c0) * (D / 4) + g) * kRows + row0 + rl;
    float2 ml[PIECES];
    float4 x[PIECES][NQ];
    auto load = [&](int j, int i) {  // piece i into place j
        const int64_t slot = 2 * i + (i == 0);
        ml[j] = __ldcg(ml0 + slot * kRows);
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            x[j][q] = __ldcg(o0 + (slot * (D / 4) + kGroups * q) * kRows);
    };
    float M = -INFINITY, den = 0.f, o[4 * NQ];
#pragma unroll
    for (int e = 0; e < 4 * NQ; ++e) o[e] = 0.f;
    // adds the first n pieces loaded
    auto add = [&](int n) {
        float top = M;
#pragma unroll
        for (int j = 0; j < PIECES; ++j)
            if (j < n) top = fmaxf(top, ml[j].x);
        // (a piece without a visible finite score weighs nothing, but a NaN in
        // its sum or its O stays)
        const float f = M == -INFINITY ? 1.f : ex2(M - top);
        M = top;
        den *= f;
#pragma unroll
        for (int e = 0; e < 4 * NQ; ++e) o[e] *= f;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            if (j >= n) break;
            const float w = ml[j].x == -INFINITY ? 1.f : ex2(ml[j].x - M);
            den = fmaf(ml[j].y, w, den);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                o[4 * q] = fmaf(x[j][q].x, w, o[4 * q]);
                o[4 * q + 1] = fmaf(x[j][q].y, w, o[4 * q + 1]);
                o[4 * q + 2] = fmaf(x[j][q].z, w, o[4 * q + 2]);
                o[4 * q + 3] = fmaf(x[j][q].w, w, o[4 * q + 3]);
            }
        }
    };
    // an item that was cut has two pieces at least: they are on their way
    // before the border says whether there is one (their slots exist anyway)
    load(0, 0);
    load(1, 1);
    const Border b = p.borders[c0 + 1];
    if (b.pieces == 0 || row0 >= b.rows) return;
    const int G = p.num_heads / p.num_kv_heads, logG = __ffs(G) - 1;
    add(2);
#pragma unroll 1
    for (int i = 2; i < b.pieces; i += PIECES) {
        const int n = min(PIECES, b.pieces - i);
#pragma unroll
        for (int j = 0; j < PIECES; ++j)
            if (j < n) load(j, i + j);
        add(n);
    }
    const float inv = den > 0.f ? 1.f / den : den;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
        turned[rl][g + kGroups * q] = make_uint2(pack_half2(o[4 * q] * inv, o[4 * q + 1] * inv),
                                                 pack_half2(o[4 * q + 2] * inv, o[4 * q + 3] * inv));
    __syncthreads();
    for (int i = threadIdx.x; i < kMergeRows * (D / 4); i += kMergeThreads) {
        const int row = row0 + i / (D / 4);
        if (row >= b.rows) break;
        __half *dst = p.out + (static_cast<int64_t>(b.q0 + (row >> logG)) * p.num_heads +
                               b.kvh * G + (row & (G - 1))) * D;
        reinterpret_cast<uint2 *>(dst)[i % (D / 4)] = turned[i / (D / 4)][i % (D / 4)];
    }
}

struct Scratch {
    int64_t borders, ml, o;  // bytes
    int64_t total() const { return borders + ml + o; }
};

Scratch scratch(int ctas, int D) {
    Scratch z;
    z.borders = dec::align256(static_cast<int64_t>(ctas) * sizeof(Border));
    z.ml = dec::align256(static_cast<int64_t>(2) * ctas * kRows * sizeof(float2));
    z.o = static_cast<int64_t>(2) * ctas * kRows * D * sizeof(float);
    return z;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A tensor map over bytes; returns a PKV status.
int encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
           const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle) {
    // the driver's encoder, found once through the runtime
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiled>(nullptr);
        return reinterpret_cast<EncodeTiled>(f);
    }();
    if (fn == nullptr) {
        set_last_error("cuTensorMapEncodeTiled is not available from the driver");
        return PKV_ERR_CUDA;
    }
    const cuuint32_t ones[4] = {1u, 1u, 1u, 1u};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank),
                          const_cast<void *>(base), dims, strides, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_last_error("cuTensorMapEncodeTiled failed (tree attention)");
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

// fp16 keys [NB * 16][row_bytes] as {128 bytes, 8 rows, chunks, 8-row groups}:
// one copy brings a head's chunks of a block, each 8 rows x 128 bytes -- the
// unit of the MMA's swizzled operand -- on its own, in a uniform order.
int make_key_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int row_bytes, int D) {
    const cuuint64_t row = static_cast<cuuint64_t>(row_bytes);
    const cuuint64_t dims[4] = {128, 8, row / 128, static_cast<cuuint64_t>(num_blocks) * 2};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {128, 8, static_cast<cuuint32_t>(D / 64), 2};
    return encode(map, cache, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Codes [NB * 16][row_bytes] by 16 rows of one head.
int make_code_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int row_bytes, int D) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes),
                                static_cast<cuuint64_t>(num_blocks) * kBS};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(D), kBS};
    return encode(map, cache, 2, dims, strides, box,
                  D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// fp16 values [NB * 16][row_bytes] as {128 bytes, rows, chunks}: 16 rows of a
// head's chunks, chunk by chunk.
int make_value_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int row_bytes, int D) {
    const cuuint64_t row = static_cast<cuuint64_t>(row_bytes);
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(num_blocks) * kBS, row / 128};
    const cuuint64_t strides[2] = {row, 128};
    const cuuint32_t box[3] = {128, kBS, static_cast<cuuint32_t>(D / 64)};
    return encode(map, cache, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Query rows [Tq][heads][D] by 128 bytes of `rows` rows: `group` heads of
// rows/group tokens.
int make_query_map(CUtensorMap *map, const void *q, int64_t tokens, int heads, int D, int group,
                   int rows) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2,
                                   static_cast<cuuint64_t>(heads) * D * 2};
    const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(group),
                               static_cast<cuuint32_t>(rows / group)};
    return encode(map, q, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The tile kernel and its merge, on `stream`.
template <int D, bool FP8>
int launch(TreeParams &p, void *workspace, cudaStream_t stream) {
    using Gm = Geo<D, FP8>;
    const int Hk = p.num_kv_heads;
    const int row_bytes = Hk * D * (FP8 ? 1 : 2);
    int st = FP8 ? make_code_map(&p.tm_k, p.k_cache, p.num_blocks, row_bytes, D)
                 : make_key_map(&p.tm_k, p.k_cache, p.num_blocks, row_bytes, D);
    if (st == PKV_OK)
        st = FP8 ? make_code_map(&p.tm_v, p.v_cache, p.num_blocks, row_bytes, D)
                 : make_value_map(&p.tm_v, p.v_cache, p.num_blocks, row_bytes, D);
    if (st == PKV_OK)
        st = make_query_map(&p.tm_q, p.q, p.num_query_tokens, p.num_heads, D, p.num_heads / Hk,
                            kRows);
    if (st == PKV_OK)
        st = make_query_map(&p.tm_q16, p.q, p.num_query_tokens, p.num_heads, D, p.num_heads / Hk,
                            16);
    if (st != PKV_OK) return st;
    const int ctas = sm_count();
    const Scratch z = scratch(ctas, D);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.borders = reinterpret_cast<Border *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + z.borders);
    p.part_o = reinterpret_cast<float4 *>(ws + z.borders + z.ml);
    using Fn = void (*)(const TreeParams);
    const Fn fn = tree_tile_kernel<D, FP8>;
    const int smem = dec::kTileAlign + Gm::kBytes;
    st = prepare_kernel(reinterpret_cast<const void *>(fn), Gm::kThreads, smem, nullptr);
    if (st != PKV_OK) return st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(Gm::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failure(e, "tree_tile_kernel launch");
    if (ctas == 1) return PKV_OK;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), kRows / kMergeRows);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    // Fewer items than half the CTAs are cut into many pieces (one sequence of
    // 1041 tokens: few in flight 10.7 us, many 10.3; 60000 tokens of one KV head
    // 29 and 27); otherwise into two or three (32 x 63 nodes of groups of 8:
    // 132 and 134; 64 ragged sequences 99.2 and 100.2).
    const int64_t items = static_cast<int64_t>(p.num_seqs) * Hk * p.max_tiles;
    e = cudaLaunchKernelEx(&cfg,
                           2 * items < ctas ? static_cast<Fn>(tree_merge_kernel<D, kMergeMany>)
                                            : static_cast<Fn>(tree_merge_kernel<D, kMergeFew>),
                           p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failure(e, "tree_merge_kernel launch");
}

int tree_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                   const float *k_scale, const float *v_scale, bool fp8,
                   const int32_t *block_tables, const int32_t *seq_lens,
                   const int32_t *query_start, const uint64_t *tree_mask, int32_t mask_words,
                   float scale, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                   int32_t block_size, int32_t num_seqs, int32_t max_blocks_per_seq,
                   int32_t num_query_tokens, int32_t max_query_len, int32_t max_seq_len,
                   int64_t num_blocks, void *workspace, size_t workspace_bytes,
                   pkv_stream_t stream) {
    if (num_seqs < 0 || num_query_tokens < 0) return PKV_ERR_INVALID;
    if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start ||
        !tree_mask || (fp8 && (!k_scale || !v_scale)))
        return PKV_ERR_NULL;
    if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 || head_dim <= 0 ||
        block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || max_query_len <= 0 ||
        max_seq_len <= 0 || mask_words <= 0 ||
        max_query_len > static_cast<int64_t>(mask_words) * 64 || !std::isfinite(scale))
        return PKV_ERR_INVALID;
    const int G = num_heads / num_kv_heads;
    if (!(G == 1 || G == 2 || G == 4 || G == 8)) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != kBS || num_seqs > 65535 || max_query_len > PKV_MAX_TREE_NODES ||
        num_blocks > INT32_MAX / kBS || max_blocks_per_seq > INT32_MAX / kBS)
        return PKV_ERR_UNSUPPORTED;
    // (a step past the last key is a 32-bit position too)
    if (std::min(max_seq_len, max_blocks_per_seq * kBS) > INT32_MAX - kStepKeys)
        return PKV_ERR_UNSUPPORTED;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scale, 16) || !aligned(v_scale, 16) || !aligned(block_tables, 4) ||
        !aligned(seq_lens, 4) || !aligned(query_start, 4) || !aligned(tree_mask, 8) ||
        !aligned(workspace, 16))
        return PKV_ERR_ALIGNMENT;
    const size_t need = pkv_tree_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim,
                                                 num_query_tokens, max_query_len, max_seq_len);
    if (workspace == nullptr || workspace_bytes < need) return PKV_ERR_WORKSPACE;
    TreeParams p{};
    p.out = static_cast<__half *>(out);
    p.q = static_cast<const __half *>(q);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.query_start = query_start;
    p.mask = tree_mask;
    p.mask_words = mask_words;
    // (a scale of zero weighs every finite score alike: so does one this small)
    const double sl2 = static_cast<double>(scale) * 1.4426950408889634;
    p.scale_log2 = static_cast<float>(std::max(std::abs(sl2), 1e-37));
    p.negate = scale < 0.f;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_query_tokens = num_query_tokens;
    p.max_query_len = max_query_len;
    p.max_tiles = (max_query_len * G + kRows - 1) / kRows;
    p.max_seq_len = max_seq_len;
    p.num_blocks = num_blocks;
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (head_dim == 128)
        return fp8 ? launch<128, true>(p, workspace, s) : launch<128, false>(p, workspace, s);
    return fp8 ? launch<64, true>(p, workspace, s) : launch<64, false>(p, workspace, s);
}

}  // namespace
}  // namespace tree
}  // namespace pkv

extern "C" size_t pkv_tree_workspace_bytes(int32_t num_seqs, int32_t num_heads,
                                           int32_t num_kv_heads, int32_t head_dim,
                                           int32_t num_query_tokens, int32_t max_query_len,
                                           int32_t max_seq_len) {
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        num_heads % num_kv_heads != 0 || num_query_tokens < 0 || max_query_len <= 0 ||
        max_seq_len <= 0)
        return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    return static_cast<size_t>(pkv::tree::scratch(pkv::sm_count(), head_dim).total());
}

extern "C" int pkv_tree_attention(void *out, const void *q, const void *k_cache,
                                  const void *v_cache, const int32_t *block_tables,
                                  const int32_t *seq_lens, const int32_t *query_start,
                                  const uint64_t *tree_mask, int32_t mask_words, float scale,
                                  int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t block_size, int32_t num_seqs,
                                  int32_t max_blocks_per_seq, int32_t num_query_tokens,
                                  int32_t max_query_len, int32_t max_seq_len,
                                  int64_t num_blocks, void *workspace, size_t workspace_bytes,
                                  pkv_stream_t stream) {
    return pkv::tree::tree_attention(out, q, k_cache, v_cache, nullptr, nullptr, false,
                                     block_tables, seq_lens, query_start, tree_mask, mask_words,
                                     scale, num_heads, num_kv_heads, head_dim, block_size,
                                     num_seqs, max_blocks_per_seq, num_query_tokens,
                                     max_query_len, max_seq_len, num_blocks, workspace,
                                     workspace_bytes, stream);
}

extern "C" int pkv_tree_attention_fp8(void *out, const void *q, const void *k_cache,
                                      const void *v_cache, const float *k_scale,
                                      const float *v_scale, const int32_t *block_tables,
                                      const int32_t *seq_lens, const int32_t *query_start,
                                      const uint64_t *tree_mask, int32_t mask_words,
                                      float scale, int32_t num_heads, int32_t num_kv_heads,
                                      int32_t head_dim, int32_t block_size, int32_t num_seqs,
                                      int32_t max_blocks_per_seq, int32_t num_query_tokens,
                                      int32_t max_query_len, int32_t max_seq_len,
                                      int64_t num_blocks, void *workspace,
                                      size_t workspace_bytes, pkv_stream_t stream) {
    return pkv::tree::tree_attention(out, q, k_cache, v_cache, k_scale, v_scale, true,
                                     block_tables, seq_lens, query_start, tree_mask, mask_words,
                                     scale, num_heads, num_kv_heads, head_dim, block_size,
                                     num_seqs, max_blocks_per_seq, num_query_tokens,
                                     max_query_len, max_seq_len, num_blocks, workspace,
                                     workspace_bytes, stream);
}
