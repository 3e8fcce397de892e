// pkv_tree.cu -- attention of a tree of drafted tokens per sequence over the
// paged cache (fp16 or FP8).
//
// Sequence i holds L tokens, the last Q of them drafted; query row r sees the
// context 0 .. L-Q-1 and the drafted tokens whose mask bit is set:
//     out = sum_vis 2^(s_j - m) V_j / sum_vis 2^(s_j - m),
//     s_j = scale log2(e) q . K_j,  m the running maximum.
//
// fp16 caches: tree_tile_kernel, on the fifth-generation tensor cores.  The
// rows of a (sequence, KV head) -- drafted token j, head g of the group:
// row j*G + g -- are cut into tiles of 128 (the MMA's M), the cache into steps
// of 128 keys.  The work is the list of (sequence, KV head, tile) items, each
// its steps plus a start-up cost; one persistent CTA per SM takes an equal
// contiguous stretch of the whole list, so a single long sequence fills the
// GPU as well as a batch does.  An item cut by a stretch's border leaves fp32
// partial states (m, l, O) in the workspace, and a second small kernel, whose
// CTAs start as the first one's leave, merges them.  Bound: HBM while a tile's
// 128-key step (64 KB of keys and values) costs less than its bytes, i.e. to
// about 128 rows per KV head; the tensor pipe and the exponentials above.
//
// Per CTA, warp-specialised, every hand-off an mbarrier with a bounded wait:
//  * warp 0 walks the stretch, publishes its pieces and stages their keys
//    (tensor copies of 16 rows x 128 bytes, a 3-step ring); warp 1 stages the
//    values (a 3-step ring);
//  * warp 2 stages a piece's query tile and issues S = Q K^T into one of two
//    score buffers, so the scores of the next step are computed while the
//    softmax works on this one;
//  * warps 3-10, two threads per row: the softmax of the chunk kernel (running
//    reference maximum that moves by more than 2^8 only, fp16 weights back to
//    tensor memory), with the tree's mask;
//  * warp 11 issues O += P V.  Value rows behind the sequence's end hold
//    anything and are zeroed first (by the softmax warps); drafted rows may be
//    masked for some query rows, and 0 x NaN is NaN, so their non-finite
//    elements are zeroed too and added, where visible, when the piece's O is
//    read out.
// Rows of a tile past the last drafted one cost no softmax work: a warp whose
// 16 rows are all past it only passes the barriers on.
//
// FP8 caches: tree_rows_kernel, one warp per (query row, head).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
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
constexpr int kThreads = 128;

struct TreeParams {
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
    float scale_log2;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t num_seqs;
    int32_t max_blocks;
    int32_t num_query_tokens;
    int32_t max_query_len;
    int32_t max_seq_len;
    int64_t num_blocks;
    ErrorRecord *err;
};

template <int D>
__device__ __forceinline__ void load_dims(const void *cache, const float *scale, int64_t row,
                                          int lane, float (&x)[D / 32]) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const int64_t at = row * D + lane + 32 * i;
        __nv_fp8_e4m3 c;
        c.__x = static_cast<const uint8_t *>(cache)[at];
        x[i] = static_cast<float>(c) * scale[row];
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) tree_rows_kernel(const __grid_constant__ TreeParams p) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int H = p.num_heads, Hk = p.num_kv_heads;
    if (w >= static_cast<int64_t>(p.num_query_tokens) * H) return;
    const int r = static_cast<int>(w / H), h = static_cast<int>(w % H), kvh = h / (H / Hk);
    int lo = 0, hi = p.num_seqs - 1;  // the last sequence that starts at or before r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.query_start[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    const int q0 = p.query_start[lo], q1 = p.query_start[lo + 1];
    if (r < q0 || r >= q1) return;
    const int Q = q1 - q0, L = p.seq_lens[lo];
    if (L < 0 || L > p.max_seq_len || L > p.max_blocks * kBS || Q > L || Q > p.max_query_len ||
        q0 < 0 || q1 > p.num_query_tokens) {
        if (lane == 0) record_error(p.err, PKV_DEVERR_SEQ_LEN, lo);
        return;
    }
    float q[D / 32], o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        q[i] = __half2float(p.q[w * D + lane + 32 * i]);
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < L; ++j) {
        if (j >= L - Q) {
            const int b = j - (L - Q);
            if (!((p.mask[static_cast<int64_t>(r) * p.mask_words + b / 64] >> (b % 64)) & 1))
                continue;
        }
        const int64_t entry = static_cast<int64_t>(lo) * p.max_blocks + j / kBS;
        const int64_t id = p.block_tables[entry];
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) record_error(p.err, PKV_DEVERR_BLOCK_ID, entry);
            continue;
        }
        const int64_t row = (id * kBS + j % kBS) * Hk + kvh;
        float x[D / 32], s = 0.f;
        load_dims<D>(p.k_cache, p.k_scale, row, lane, x);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale_log2;
        if (s == -INFINITY) continue;
        const float mn = fmaxf(m, s), a = exp2f(m - mn), pr = exp2f(s - mn);
        load_dims<D>(p.v_cache, p.v_scale, row, lane, x);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = fmaf(o[i], a, pr * x[i]);
        l = fmaf(l, a, pr);
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        p.out[w * D + lane + 32 * i] = __float2half_rn(l == 0.f ? 0.f : o[i] / l);
}

// ---------------------------------------------------------------------------
// The tensor-core kernel.

constexpr int kRows = 128;                    // query rows per tile: the MMA's M
constexpr int kStepBlocks = 8;                // blocks per step
constexpr int kStepKeys = kStepBlocks * kBS;  // 128 keys: the score MMA's N
constexpr int kKStages = 3;                   // key ring depth (steps)
constexpr int kVStages = 3;                   // value ring depth (steps)
// softmax: warp 3 + 4 wh + q takes rows (tensor-memory lanes) 32 q + 16 wh ..
// + 15, two threads per row: lanes 16 h + i take keys 64 h .. of a step and
// the head dimensions (D/2) h .. of O
constexpr int kSoftmaxWarps = 8;
constexpr int kHalfKeys = kStepKeys / 2;
constexpr int kPVWarp = 3 + kSoftmaxWarps;
constexpr int kTileThreads = (4 + kSoftmaxWarps) * 32;
// tensor memory: O in columns [0, head_dim), two score buffers of 128 columns,
// two weight buffers (fp16 pairs) of 64
constexpr int kTmemCols = 512;
constexpr int kTmemO = 0;
constexpr int kTmemS = 128;
constexpr int kTmemP = 384;
constexpr float kRescaleLog2 = 8.f;  // move the reference past 2^8
constexpr int kFlagWords = PKV_MAX_TREE_NODES / 32;
// merge: threads per row, rows per block
constexpr int kMergeThreads = 128;
constexpr int kMergeRows = 8;

// What a stretch's first border says about the item it falls into.
struct Border {
    int32_t pieces;  // of the item; 0: the border cuts none, or is not the
                     // item's first border
    int32_t rows;    // query rows of the tile
    int32_t q0;      // first query token of the tile
    int32_t kvh;
};

struct TileParams {
    CUtensorMap tm_k;  // keys: 128 bytes of 16 rows per copy
    CUtensorMap tm_v;  // values: a head's chunks of 16 rows per copy
    CUtensorMap tm_q;  // query rows: 128 bytes of each row of a 128-row tile
    TreeParams t;
    Border *borders;  // [CTAs]
    float2 *part_ml;  // [2 CTAs][128] (m, l)
    float *part_o;    // [2 CTAs][128][D]
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
constexpr int kValidRing = 8;  // steps whose blocks' validity is kept (see the softmax)

template <int D>
struct Geo {
    static constexpr int kChunks = D / 64;                // 128-byte chunks of a head row
    static constexpr int kQ = kChunks * kRows * 128;      // [chunk][row][128 B]
    static constexpr int kK = kChunks * kStepKeys * 128;  // [chunk][key][128 B]
    static constexpr int kVBlock = kChunks * kBS * 128;   // [chunk][token][128 B]
    static constexpr int kV = kStepBlocks * kVBlock;
    static constexpr int kOffK = kQ;
    static constexpr int kOffV = kOffK + kKStages * kK;
    static constexpr int kOffBar = kOffV + kVStages * kV;
    static constexpr int kBars = 4 + 2 + 2 * kKStages + 2 * kVStages + 4 + 4 + 2;
    static constexpr int kOffPiece = kOffBar + kBars * 8;
    static constexpr int kOffFlags = kOffPiece + 2 * static_cast<int>(sizeof(Piece));
    static constexpr int kOffValid = kOffFlags + 3 * kFlagWords * 4;  // (see the softmax)
    static constexpr int kOffMisc = kOffValid + kValidRing * 4;
    static constexpr int kOffScan = kOffMisc + 16;  // the prologue's words
    static constexpr int kBytes = kOffScan + (kTileThreads / 32 + 4) * 8;
};

int tile_smem_bytes(int D) {
    return dec::kTileAlign + (D == 128 ? Geo<128>::kBytes : Geo<64>::kBytes);
}

// mbarrier addresses (shared space) by role
struct Bars {
    uint32_t b;
    __device__ uint32_t piece_full(int s) const { return b + 8 * s; }
    __device__ uint32_t piece_empty(int s) const { return b + 8 * (2 + s); }
    __device__ uint32_t q_full() const { return b + 8 * 4; }
    __device__ uint32_t q_empty() const { return b + 8 * 5; }
    __device__ uint32_t k_full(int s) const { return b + 8 * (6 + s); }
    __device__ uint32_t k_empty(int s) const { return b + 8 * (6 + kKStages + s); }
    static constexpr int kV0 = 6 + 2 * kKStages;
    __device__ uint32_t v_full(int s) const { return b + 8 * (kV0 + s); }
    __device__ uint32_t v_empty(int s) const { return b + 8 * (kV0 + kVStages + s); }
    static constexpr int kS0 = kV0 + 2 * kVStages;
    __device__ uint32_t s_full(int s) const { return b + 8 * (kS0 + s); }
    __device__ uint32_t s_free(int s) const { return b + 8 * (kS0 + 2 + s); }
    __device__ uint32_t p_full(int s) const { return b + 8 * (kS0 + 4 + s); }
    __device__ uint32_t pv_done(int s) const { return b + 8 * (kS0 + 6 + s); }
    __device__ uint32_t o_free() const { return b + 8 * (kS0 + 8); }
    __device__ uint32_t scanned() const { return b + 8 * (kS0 + 9); }
};

// arrivals that free a piece record: the value producer, the two MMA warps and
// every softmax warp
constexpr int kPieceReaders = 3 + kSoftmaxWarps;

// Every lane waits (bounded); false if any lane gave up.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed fp32 pairs (one instruction for two lanes' worth of fma or add) and
// the three-input maximum.
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
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
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

// Transposes N x N 16-byte elements held by groups of N lanes (N = 4 or 8):
// afterwards element c of lane t of a group is element t of the group's lane c.
template <int N>
__device__ __forceinline__ void lane_transpose(uint4 (&x)[N], int lane) {
#pragma unroll
    for (int m = 1; m < N; m <<= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < N; ++i) {
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

// Units of an item: its steps and kItemUnits for its start-up.
constexpr int kItemUnits = 1;

// The step a place `x` units into an item falls on.
__device__ __forceinline__ int step_at(int64_t x, int steps) {
    const int64_t s = x - kItemUnits;
    return s <= 0 ? 0 : s >= steps ? steps : static_cast<int>(s);
}

// First unit of CTA c's stretch, of `busy` = min(CTAs, units) that have one
// (so no stretch is empty).
__device__ __forceinline__ int64_t stretch(int64_t units, int c, int busy) {
    return units * c / busy;
}

struct SeqGeo {
    int L, Q, q0, tiles, steps;
};

__device__ __forceinline__ SeqGeo make_geo(int L, int Q, int q0, int G) {
    return SeqGeo{L, Q, q0, (Q * G + kRows - 1) / kRows, (L + kStepKeys - 1) / kStepKeys};
}

// Geometry of sequence s; false if it has no rows or is invalid (recorded when
// `report`).
__device__ __forceinline__ bool seq_geo(const TreeParams &p, int s, int G, bool report,
                                        SeqGeo &sg) {
    const int L = __ldg(p.seq_lens + s);
    const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1);
    const int Q = q1 - q0;
    if (L < 0 || L > p.max_seq_len || L > static_cast<int64_t>(p.max_blocks) * kBS || Q < 0 ||
        Q > L || Q > p.max_query_len || q0 < 0 || q1 > p.num_query_tokens) {
        if (report) record_error(p.err, PKV_DEVERR_SEQ_LEN, s);
        return false;
    }
    sg = make_geo(L, Q, q0, G);
    return Q > 0;
}

__device__ __forceinline__ int64_t seq_units(const SeqGeo &sg, int Hk) {
    return static_cast<int64_t>(Hk) * sg.tiles * (sg.steps + kItemUnits);
}

// Sum over the CTA of v, and the exclusive prefix of this thread's (every
// thread calls; `sh` holds one word per warp).
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t *sh, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kTileThreads / 32;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
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

// Byte offset of 16-byte unit i (row-major) of a staged value tile.
template <int CH>
__device__ __forceinline__ int v_unit(int i) {
    const int t = i / (8 * CH), u = i % (8 * CH);
    return (t >> 4) * (CH * kBS * 128) + (u >> 3) * (kBS * 128) + (t & 15) * 128 + (u & 7) * 16;
}

// The fp16 pair w with infinities and NaN zeroed.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
    if ((w & 0x7C00u) == 0x7C00u) w &= 0xFFFF0000u;
    if ((w & 0x7C000000u) == 0x7C000000u) w &= 0x0000FFFFu;
    return w;
}

// The value tile `vb` of a step that reaches past the context: rows at and past
// the sequence's end hold anything and are zeroed; of the drafted rows (key ctx
// on) the non-finite elements are zeroed and the row flagged.  `keys` of the
// step's keys, the first of them key0, are staged; thread i of kScanners.  A
// unit is 16 bytes, kScan of them in flight per thread.
constexpr int kScanners = kSoftmaxWarps * 32;
template <int CH>
__device__ __forceinline__ void clean_values(uint8_t *vb, int key0, int keys, int ctx, int L,
                                             uint32_t *flags, int thread) {
    constexpr int kUnits = 8 * CH;  // units of a row
    constexpr int kScan = 4;
    const int end = keys * kUnits;
    for (int i0 = max(ctx - key0, 0) * kUnits + thread; i0 < end; i0 += kScanners * kScan) {
        uint4 x[kScan];
#pragma unroll
        for (int k = 0; k < kScan; ++k)
            x[k] = *reinterpret_cast<const uint4 *>(vb + v_unit<CH>(min(i0 + kScanners * k, end - 1)));
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            const int i = i0 + kScanners * k;
            const int key = key0 + i / kUnits;
            // all ones in an exponent carry into its sign's place
            const uint32_t bad = (((x[k].x & 0x7C007C00u) + 0x04000400u) |
                                  ((x[k].y & 0x7C007C00u) + 0x04000400u) |
                                  ((x[k].z & 0x7C007C00u) + 0x04000400u) |
                                  ((x[k].w & 0x7C007C00u) + 0x04000400u)) & 0x80008000u;
            if (i >= end || (bad == 0 && key < L)) continue;
            uint4 *at = reinterpret_cast<uint4 *>(vb + v_unit<CH>(i));
            if (key >= L) {
                *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
                *at = make_uint4(finite_halves(x[k].x), finite_halves(x[k].y),
                                 finite_halves(x[k].z), finite_halves(x[k].w));
                atomicOr(&flags[(key - ctx) >> 5], 1u << ((key - ctx) & 31));
            }
        }
    }
    fence_proxy_async_smem();
}

// Block id of entry b of a sequence, or -1 when out of range (recorded when
// `report`).
__device__ __forceinline__ int block_id(const TreeParams &p, int seq, int b, bool report) {
    const int64_t at = static_cast<int64_t>(seq) * p.max_blocks + b;
    const int id = __ldg(p.block_tables + at);
    if (id >= 0 && static_cast<int64_t>(id) < p.num_blocks) return id;
    if (report) record_error(p.err, PKV_DEVERR_BLOCK_ID, at);
    return -1;
}

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    tree_tile_kernel(const __grid_constant__ TileParams tp) {
    using Gm = Geo<D>;
    constexpr int CH = Gm::kChunks;
    constexpr int DH = D / 2;  // the head dimensions (of O) each softmax thread owns
    const TreeParams &p = tp.t;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((dec::kTileAlign - (smem_u32(smem_raw) & (dec::kTileAlign - 1))) &
                                (dec::kTileAlign - 1));
    const uint32_t sb = smem_u32(smem);
    const Bars br{sb + Gm::kOffBar};
    Piece *pieces = reinterpret_cast<Piece *>(smem + Gm::kOffPiece);
    uint32_t *flags = reinterpret_cast<uint32_t *>(smem + Gm::kOffFlags);
    volatile uint32_t *valid = reinterpret_cast<volatile uint32_t *>(smem + Gm::kOffValid);
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + Gm::kOffMisc);
    int64_t *scan = reinterpret_cast<int64_t *>(smem + Gm::kOffScan);
    volatile int64_t *start = scan + kTileThreads / 32;  // sequence, its first unit, L | Q, q0

    const int Hk = p.num_kv_heads, H = p.num_heads;
    const int G = H / Hk, logG = __ffs(G) - 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(br.piece_full(s), 1);
            mbar_init(br.piece_empty(s), kPieceReaders);
            mbar_init(br.s_full(s), 2);
            mbar_init(br.s_free(s), kSoftmaxWarps);
            mbar_init(br.p_full(s), kSoftmaxWarps);
            mbar_init(br.pv_done(s), 1);
        }
        mbar_init(br.q_full(), 1);
        mbar_init(br.q_empty(), 1);
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(br.k_full(s), 1);
            mbar_init(br.k_empty(s), 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(br.v_full(s), 1);
            mbar_init(br.v_empty(s), 1);
        }
        mbar_init(br.o_free(), kSoftmaxWarps);
        mbar_init(br.scanned(), kSoftmaxWarps);
        fence_mbarrier_init();
        prefetch_tensormap(&tp.tm_k);
        prefetch_tensormap(&tp.tm_v);
        prefetch_tensormap(&tp.tm_q);
    }
    if (threadIdx.x < 3 * kFlagWords) flags[threadIdx.x] = 0;
    if (warp == 2) {
        tc::tmem_alloc(sb + Gm::kOffMisc, kTmemCols);
        tc::tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();  // the merge: it waits for this grid

    // ---- the list's length, and where this CTA's stretch starts: the thread
    // that holds the sequence its first unit falls into says so (with more
    // sequences than threads, in a second pass)
    int64_t units = 0;
    const bool one_pass = p.num_seqs <= kTileThreads;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kTileThreads) {
        const int s = s0 + threadIdx.x;
        SeqGeo sg;
        const bool has = s < p.num_seqs && seq_geo(p, s, G, cta == 0, sg);
        int64_t total;
        const int64_t w = has ? seq_units(sg, Hk) : 0;
        const int64_t before = cta_scan(w, scan, total);
        units += total;
        if (one_pass && total > 0) {
            const int64_t u0 = stretch(total, cta, static_cast<int>(min(static_cast<int64_t>(ctas), total)));
            if (w > 0 && before <= u0 && u0 < before + w) {
                start[0] = s;
                start[1] = before;
                start[2] = static_cast<int64_t>(sg.L) << 32 | static_cast<unsigned>(sg.Q);
                start[3] = sg.q0;
            }
        }
    }
    const int busy = static_cast<int>(min(static_cast<int64_t>(ctas), units));  // CTAs with a stretch
    const int64_t u0 = busy ? stretch(units, cta, busy) : 0;
    const int64_t u1 = busy ? stretch(units, cta + 1, busy) : 0;
    if (!one_pass && cta < busy) {
        int64_t run = 0;
        for (int s0 = 0; s0 < p.num_seqs; s0 += kTileThreads) {
            const int s = s0 + threadIdx.x;
            SeqGeo sg;
            const bool has = s < p.num_seqs && seq_geo(p, s, G, false, sg);
            int64_t total;
            const int64_t w = has ? seq_units(sg, Hk) : 0;
            const int64_t before = run + cta_scan(w, scan, total);
            if (w > 0 && before <= u0 && u0 < before + w) {
                start[0] = s;
                start[1] = before;
                start[2] = static_cast<int64_t>(sg.L) << 32 | static_cast<unsigned>(sg.Q);
                start[3] = sg.q0;
            }
            run += total;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = misc[0];
    if (cta >= busy) {
        if (threadIdx.x == 0) tp.borders[cta].pieces = 0;
    } else if (warp == 0) {
        // ===================== pieces, query tiles and keys =====================
        int seq = static_cast<int>(start[0]);
        int64_t first = start[1];  // the sequence's first unit
        int64_t u = u0;
        SeqGeo sg = make_geo(static_cast<int>(start[2] >> 32), static_cast<int>(start[2]),
                             static_cast<int>(start[3]), G);
        // the place of the stretch's start in its item, kept from piece to piece
        int n = sg.steps + kItemUnits;
        int item = static_cast<int>((u - first) / n);
        int x = static_cast<int>(u - first - static_cast<int64_t>(item) * n);
        // the border at u0, for the merge (every CTA writes one, whether or not
        // its stretch holds a step)
        if (lane == 0) {
            Border border;
            const int64_t a = u0 - x;
            const int tile = item % sg.tiles;
            const bool cuts = cta > 0 && step_at(x, sg.steps) > 0 &&
                              step_at(stretch(units, cta - 1, busy) - a, sg.steps) == 0;
            // pieces: the CTA before this one, and those up to the item's last unit
            border.pieces =
                cuts ? static_cast<int>(((a + n) * busy - 1) / units) - (cta - 1) + 1 : 0;
            border.rows = min(kRows, sg.Q * G - tile * kRows);
            border.q0 = sg.q0 + tile * (kRows >> logG);
            border.kvh = item / sg.tiles;
            tp.borders[cta] = border;
        }
        __syncwarp();
        // The next piece of the stretch, and the ids of its first blocks.
        auto next_piece = [&](PieceHead &pc, int &ids) {
            pc.done = 1;
            ids = -1;
            while (u < u1) {
                if (x == n) {  // the next item
                    x = 0;
                    if (++item == Hk * sg.tiles) {  // of the next sequence with rows
                        item = 0;
                        do ++seq;
                        while (seq < p.num_seqs && !seq_geo(p, seq, G, false, sg));
                        if (seq >= p.num_seqs) return;  // (not reached: u1 is inside the list)
                        n = sg.steps + kItemUnits;
                    }
                }
                const int take = static_cast<int>(min(u1 - u, static_cast<int64_t>(n - x)));
                const int s0 = step_at(x, sg.steps), s1 = step_at(x + take, sg.steps);
                u += take;
                x += take;
                if (s1 == s0) continue;
                pc.seq = seq;
                pc.kvh = item / sg.tiles;
                pc.tile = item - pc.kvh * sg.tiles;
                pc.step0 = s0;
                pc.nsteps = s1 - s0;
                pc.nblk = min((sg.L + kBS - 1) / kBS - s0 * kStepBlocks, pc.nsteps * kStepBlocks);
                pc.L = sg.L;
                pc.Q = sg.Q;
                pc.q0 = sg.q0;
                pc.slot = s0 == 0 && s1 == sg.steps ? -1 : 2 * cta + (s0 == 0);
                pc.done = 0;
                if (lane < pc.nblk) ids = block_id(p, seq, s0 * kStepBlocks + lane, true);
                return;
            }
        };
        PieceHead cur;
        int cur_ids;
        next_piece(cur, cur_ids);
        int gs = 0;  // steps staged
        bool ok = true;
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
            // its keys: the ids of 32 blocks at a time, one per lane, the next
            // ones -- of this piece or the next -- looked up a window ahead
            const int b0 = cur.step0 * kStepBlocks;
            PieceHead nxt;
            int nxt_ids = -1, ids = cur_ids, ahead = -1;
            for (int n = 0; n < cur.nsteps; ++n, ++gs) {
                const int ks = gs % kKStages;
                const int at = n * kStepBlocks;
                if ((at & 31) == 0) {
                    if (at != 0) ids = ahead;
                    const int b = at + 32 + lane;
                    ahead = b < cur.nblk ? block_id(p, cur.seq, b0 + b, true) : -1;
                }
                if (gs >= kKStages && !wait_all(br.k_empty(ks), ((gs / kKStages) - 1) & 1)) {
                    ok = false;
                    break;
                }
                const int nb = min(kStepBlocks, cur.nblk - at);
                // lane l: block l / CH of the step, chunk l % CH (a bad block
                // reads rows before the cache: zeros)
                const int b = min(lane / CH, kStepBlocks - 1), c = lane % CH;
                const int id = __shfl_sync(0xffffffffu, ids, (at & 31) + b);
                const uint32_t good = __ballot_sync(0xffffffffu, id >= 0 || lane >= nb * CH);
                if (lane == 0) {
                    valid[gs % kValidRing] = good;
                    mbar_arrive_expect_tx(br.k_full(ks), nb * CH * kBS * 128);
                }
                __syncwarp();
                if (lane < nb * CH)
                    tensor_g2s_3d(sb + Gm::kOffK + ks * Gm::kK + c * (kStepKeys * 128) +
                                      b * (kBS * 128),
                                  &tp.tm_k, 0, id >= 0 ? id * kBS : -kBS, cur.kvh * CH + c,
                                  br.k_full(ks));
                // (when the ring is full: the look-ups wait for memory)
                if (n == min(kKStages, cur.nsteps) - 1) next_piece(nxt, nxt_ids);
            }
            cur = nxt;
            cur_ids = nxt_ids;
        }
        if (!ok) {
            if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, cta);
            // let the last copies land before the CTA can exit
            for (int s = 0; s < kKStages && s < gs; ++s) {
                const int last = gs - 1 - ((gs - 1 - s) % kKStages);
                mbar_wait_bounded(br.k_full(s), (last / kKStages) & 1);
            }
        }
    } else if (warp == 1) {
        // ================================ values ================================
        int gs = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int rec = it & 1;
            if (!wait_all(br.piece_full(rec), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const PieceHead pc = pieces[rec];
            int ids = pieces[rec].ids[lane];
            __syncwarp();
            if (lane == 0) mbar_arrive(br.piece_empty(rec));
            if (pc.done) break;
            const int b0 = pc.step0 * kStepBlocks;
            int ahead = -1;
            for (int n = 0; n < pc.nsteps; ++n, ++gs) {
                const int vs = gs % kVStages;
                const int at = n * kStepBlocks;
                if ((at & 31) == 0) {
                    if (at != 0) ids = ahead;
                    const int b = at + 32 + lane;
                    ahead = b < pc.nblk ? block_id(p, pc.seq, b0 + b, false) : -1;
                }
                if (gs >= kVStages && !wait_all(br.v_empty(vs), ((gs / kVStages) - 1) & 1)) {
                    ok = false;
                    break;
                }
                const int nb = min(kStepBlocks, pc.nblk - at);
                if (lane == 0) mbar_arrive_expect_tx(br.v_full(vs), nb * Gm::kVBlock);
                __syncwarp();
                const int id = __shfl_sync(0xffffffffu, ids, (at & 31) + min(lane, kStepBlocks - 1));
                if (lane < nb)
                    tensor_g2s_3d(sb + Gm::kOffV + vs * Gm::kV + lane * Gm::kVBlock, &tp.tm_v, 0,
                                  id >= 0 ? id * kBS : -kBS, pc.kvh * CH, br.v_full(vs));
            }
        }
        if (!ok) {
            if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, cta);
            for (int s = 0; s < kVStages && s < gs; ++s) {
                const int last = gs - 1 - ((gs - 1 - s) % kVStages);
                mbar_wait_bounded(br.v_full(s), (last / kVStages) & 1);
            }
        }
    } else if (warp == 2) {
        // ==================== query tiles and score MMAs ====================
        int gs = 0, q_staged = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int rec = it & 1;
            if (!wait_all(br.piece_full(rec), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const PieceHead pc = pieces[rec];
            const int nsteps = pc.nsteps, nblk = pc.nblk;
            __syncwarp();
            if (lane == 0) mbar_arrive(br.piece_empty(rec));
            if (pc.done) break;
            // the query tile, once the previous piece's last scores are done
            if (it >= 1) ok = wait_all(br.q_empty(), (it - 1) & 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(br.q_full(), Gm::kQ);
            __syncwarp();
            if (lane < CH)
                tensor_g2s_3d(sb + lane * (kRows * 128), &tp.tm_q, 128 * lane, pc.kvh * G,
                              pc.q0 + pc.tile * (kRows >> logG), br.q_full());
            q_staged = it + 1;
            ok = wait_all(br.q_full(), it & 1);
            for (int n = 0; n < nsteps && ok; ++n, ++gs) {
                const int ks = gs % kKStages, b = gs & 1;
                ok = wait_all(br.k_full(ks), (gs / kKStages) & 1);
                // the softmax has read the scores of two steps back
                if (ok && gs >= 2) ok = wait_all(br.s_free(b), ((gs >> 1) - 1) & 1);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
                    const int nb = min(kStepBlocks, nblk - n * kStepBlocks);
                    const uint32_t idesc = tc::idesc_f16_f32(kRows, nb * kBS, false, false);
                    const uint32_t k_s = sb + Gm::kOffK + ks * Gm::kK;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc::mma_ss(tmem + kTmemS + 128 * b,
                                   tc::smem_desc(sb + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16,
                                                 1024, tc::kSwizzle128B),
                                   tc::smem_desc(k_s + (kk >> 2) * (kStepKeys * 128) + (kk & 3) * 32,
                                                 16, 1024, tc::kSwizzle128B),
                                   idesc, kk > 0);
                    tc::commit(br.s_full(b));
                    mbar_arrive(br.s_full(b));  // passes the step's validity on
                    tc::commit(br.k_empty(ks));
                    if (n == nsteps - 1) tc::commit(br.q_empty());
                }
                __syncwarp();
            }
        }
        if (!ok) {
            if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, cta);
            if (q_staged) mbar_wait_bounded(br.q_full(), (q_staged - 1) & 1);
        }
    } else if (warp == kPVWarp) {
        // ============================= P V MMAs =============================
        constexpr uint32_t kIdescPV = tc::idesc_f16_f32(kRows, D, false, true);
        int gs = 0;
        bool ok = true;
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
            for (int n = 0; n < pc.nsteps && ok; ++n, ++gs) {
                const int vs = gs % kVStages, b = gs & 1;
                const int nb = min(kStepBlocks, pc.nblk - n * kStepBlocks);
                // the previous piece's O has been read
                if (n == 0 && it > 0) ok = wait_all(br.o_free(), (it - 1) & 1);
                if (ok) ok = wait_all(br.v_full(vs), (gs / kVStages) & 1);
                if (!ok) break;
                const uint32_t v_s = sb + Gm::kOffV + vs * Gm::kV;
                ok = wait_all(br.p_full(b), (gs >> 1) & 1);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
                    for (int k = 0; k < nb; ++k)
                        tc::mma_ts(tmem + kTmemO, tmem + kTmemP + 64 * b + 8 * k,
                                   tc::smem_desc(v_s + k * Gm::kVBlock, kBS * 128, 1024,
                                                 tc::kSwizzle128B),
                                   kIdescPV, (n > 0 || k > 0) ? 1u : 0u);
                    tc::commit(br.pv_done(b));
                    tc::commit(br.v_empty(vs));
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, cta);
    } else {
        // =============================== softmax ===============================
        const int wh = (warp - 3) >> 2;
        const int quarter = warp & 3;
        const int h = lane >> 4;
        const int r = quarter * 32 + wh * 16 + (lane & 15);
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32 + wh * 16) << 16);
        const float sl2 = p.scale_log2;
        int gs = 0;
        bool ok = true;
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
            const int rr = pc.tile * kRows + r;
            const bool row_ok = rr < pc.Q * G;
            const bool live = __any_sync(0xffffffffu, row_ok);
            const int j = rr >> logG;
            const uint64_t *mask =
                row_ok ? p.mask + static_cast<int64_t>(pc.q0 + j) * p.mask_words : nullptr;
            // bring the row's mask near, for the step that needs it
            if (row_ok) prefetch_l1(mask);
            uint32_t *my_flags = flags + (it % 3) * kFlagWords;
            float m_used = -INFINITY, l = 0.f;  // l: this thread's keys only

            for (int n = 0; n < pc.nsteps; ++n, ++gs) {
                const int sbuf = gs & 1;
                const int key0 = (pc.step0 + n) * kStepKeys;
                if (key0 + kStepKeys > ctx) {
                    const int vs = gs % kVStages;
                    if (!wait_all(br.v_full(vs), (gs / kVStages) & 1)) {
                        ok = false;
                        break;
                    }
                    clean_values<CH>(smem + Gm::kOffV + vs * Gm::kV, key0,
                                     min(kStepBlocks, pc.nblk - n * kStepBlocks) * kBS, ctx, pc.L,
                                     my_flags, threadIdx.x - 3 * 32);
                    __syncwarp();
                }
                if (n == pc.nsteps - 1 && lane == 0) mbar_arrive(br.scanned());
                if (!wait_all(br.s_full(sbuf), (gs >> 1) & 1)) {
                    ok = false;
                    break;
                }
                // the step's blocks that are in range: the key producer's word,
                // one bit per copy (the ring is longer than it can be ahead:
                // it stages at most kKStages steps past the scores, and these
                // are at most two ahead of this warp)
                const uint32_t copies = valid[gs % kValidRing];
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
                tc::wait_ld();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(br.s_free(sbuf));
                const bool fast = copies == 0xffffffffu && key0 + kStepKeys <= ctx && sl2 >= 0.f;
                if (!fast) {
                    uint64_t vis = visible(mask, p.mask_words, key0 + kHalfKeys * h, ctx, pc.L);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (!((copies >> (CH * (4 * h + b))) & 1u)) vis &= ~(0xFFFFull << (16 * b));
#pragma unroll
                    for (int e = 0; e < kHalfKeys; ++e) {
                        const uint32_t w = e < 32 ? static_cast<uint32_t>(vis)
                                                  : static_cast<uint32_t>(vis >> 32);
                        sx[e] = (w >> (e & 31)) & 1u
                                    ? __float_as_uint(__uint_as_float(sx[e]) * sl2)
                                    : __float_as_uint(-INFINITY);
                    }
                }
                float mr[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mr[i] = -INFINITY;
#pragma unroll
                for (int e = 0; e < kHalfKeys / 2; ++e)
                    mr[e & 7] = fmax3(mr[e & 7], __uint_as_float(sx[2 * e]),
                                      __uint_as_float(sx[2 * e + 1]));
                float mx = fmax3(fmax3(mr[0], mr[1], mr[2]), fmax3(mr[3], mr[4], mr[5]),
                                 fmaxf(mr[6], mr[7]));
                if (fast) mx *= sl2;
                // the row's other half: the thread 16 lanes away
                const float mo = __shfl_xor_sync(0xffffffffu, mx, 16);
                const float m_new = fmaxf(m_used, fmaxf(mx, mo));
                const bool raise = m_new > m_used + kRescaleLog2;
                // O holds this piece's earlier steps relative to m_used: rescale
                // this thread's columns before the reference moves (the
                // previous P V done first)
                const bool resc = raise && n > 0 && m_used != -INFINITY;
                if (__any_sync(0xffffffffu, resc)) {
                    if (!wait_all(br.pv_done((gs - 1) & 1), ((gs - 1) >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const float alpha = resc ? ex2(m_used - m_new) : 1.f;
#pragma unroll
                    for (int c = 0; c < DH / 32; ++c) {
                        uint32_t x[32];
                        tc::ld32_halves<DH>(tl + kTmemO + 32 * c, x);
                        tc::wait_ld();
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
                // weights 2^(s * scale - m) (2^(t - m) for masked steps), fp16
                // pairs; the P V of two steps back is done with this buffer
                const float a = fast ? sl2 : 1.f;
                if (gs >= 2) {
                    if (!wait_all(br.pv_done(sbuf), ((gs >> 1) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                }
                const uint64_t a2 = f32x2(a, a), nms2 = f32x2(-ms, -ms);
                uint64_t l2[4] = {0ull, 0ull, 0ull, 0ull};
                uint32_t x[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 t = f32x2_split(fma_f32x2(
                        f32x2(__uint_as_float(sx[2 * e]), __uint_as_float(sx[2 * e + 1])), a2, nms2));
                    const float p0 = ex2(t.x), p1 = ex2(t.y);
                    l2[e & 3] = add_f32x2(l2[e & 3], f32x2(p0, p1));
                    x[e] = pack_half2(p0, p1);
                }
                tc::st32_halves<32>(tl + kTmemP + 64 * sbuf, x);
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
            if (!wait_all(br.pv_done((gs - 1) & 1), ((gs - 1) >> 1) & 1) ||
                !wait_all(br.scanned(), it & 1)) {
                ok = false;
                break;
            }
            // the flags of the piece after the next one: every warp has read
            // what they held for the previous piece, and none reaches that
            // piece before this warp's arrivals for the next
            if (warp == 3 && lane < kFlagWords) flags[(it + 2) % 3 * kFlagWords + lane] = 0;
            __syncwarp();
            if (!live) {
                if (lane == 0) mbar_arrive(br.o_free());
                continue;
            }
            tc::fence_after_sync();
            float o[DH];
            {
                uint32_t ob[DH];
#pragma unroll
                for (int c = 0; c < DH / 32; ++c)
                    tc::ld32_halves<DH>(tl + kTmemO + 32 * c,
                                        *reinterpret_cast<uint32_t(*)[32]>(ob + 32 * c));
                tc::wait_ld();
#pragma unroll
                for (int d = 0; d < DH; ++d) o[d] = __uint_as_float(ob[d]);
            }
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < kFlagWords; ++w) any |= my_flags[w];
            if (any != 0 && row_ok) {
                // the elements that were left out: a weight times an infinity
                // or a NaN is that, whatever the (positive) weight
                for (int node = 0; node < pc.Q; ++node) {
                    if (!((my_flags[node >> 5] >> (node & 31)) & 1u) ||
                        !((__ldg(mask + (node >> 6)) >> (node & 63)) & 1))
                        continue;
                    const int key = ctx + node;
                    const int id = block_id(p, pc.seq, key / kBS, false);
                    if (id < 0) continue;
                    const __half *v = static_cast<const __half *>(p.v_cache) +
                                      ((static_cast<int64_t>(id) * kBS + key % kBS) * Hk + pc.kvh) * D +
                                      DH * h;
#pragma unroll
                    for (int d = 0; d < DH; ++d) {
                        const float x = __half2float(v[d]);
                        if (!isfinite(x)) o[d] += x;
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(br.o_free());
            l += __shfl_xor_sync(0xffffffffu, l, 16);  // the row's sum over both halves' keys
            // a thread holds DH dims of one row: exchanged inside groups of
            // lanes so that a warp's store covers whole lines of a few rows
            // (stored as they lie, 32 lanes on 32 lines, an item's outputs
            // took 3 us and its partial state 6)
            const int r0 = quarter * 32 + wh * 16;
            if (pc.slot < 0) {
                const float inv = l > 0.f ? 1.f / l : l;  // (no visible key: 0; NaN stays)
                constexpr int NC = DH / 8;  // 16-byte pieces of a thread's fp16 dims
                uint4 x[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    x[c] = make_uint4(pack_half2(o[8 * c] * inv, o[8 * c + 1] * inv),
                                      pack_half2(o[8 * c + 2] * inv, o[8 * c + 3] * inv),
                                      pack_half2(o[8 * c + 4] * inv, o[8 * c + 5] * inv),
                                      pack_half2(o[8 * c + 6] * inv, o[8 * c + 7] * inv));
                lane_transpose<NC>(x, lane);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int src = (lane & ~(NC - 1)) + c;  // the lane the row came from
                    const int row = pc.tile * kRows + r0 + (src & 15);
                    if (row < pc.Q * G)
                        *reinterpret_cast<uint4 *>(
                            p.out + (static_cast<int64_t>(pc.q0 + (row >> logG)) * H + pc.kvh * G +
                                     (row & (G - 1))) * D +
                            DH * (src >> 4) + 8 * (lane & (NC - 1))) = x[c];
                }
            } else {
                const int64_t row0 = static_cast<int64_t>(pc.slot) * kRows;
                if (h == 0 && row_ok) tp.part_ml[row0 + r] = make_float2(m_used, l);
#pragma unroll
                for (int k = 0; k < DH / 32; ++k) {
                    uint4 x[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        x[c] = make_uint4(__float_as_uint(o[32 * k + 4 * c]),
                                          __float_as_uint(o[32 * k + 4 * c + 1]),
                                          __float_as_uint(o[32 * k + 4 * c + 2]),
                                          __float_as_uint(o[32 * k + 4 * c + 3]));
                    lane_transpose<8>(x, lane);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int src = (lane & ~7) + c;
                        const int row = r0 + (src & 15);
                        if (pc.tile * kRows + row < pc.Q * G)
                            *reinterpret_cast<uint4 *>(tp.part_o + (row0 + row) * D +
                                                       DH * (src >> 4) + 32 * k + 4 * (lane & 7)) =
                                x[c];
                    }
                }
            }
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, cta);
    }

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
// to cut.  D/8 threads per row, 8 dims each.  The item's first piece is the
// last one of CTA b (its second slot), the others the first ones of the CTAs
// that follow.
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    tree_merge_kernel(const __grid_constant__ TileParams tp) {
    constexpr int kPerRow = D / 8;
    constexpr int kPass = kMergeThreads / kPerRow;  // rows at a time
    grid_dependency_wait();
    const int c0 = blockIdx.x;
    const Border b = tp.borders[c0 + 1];
    if (b.pieces == 0) return;
    const TreeParams &p = tp.t;
    const int G = p.num_heads / p.num_kv_heads, logG = __ffs(G) - 1;
    for (int rr = blockIdx.y * kMergeRows + threadIdx.x / kPerRow;
         rr < min(b.rows, static_cast<int>(blockIdx.y + 1) * kMergeRows); rr += kPass) {
        const int d0 = 8 * (threadIdx.x % kPerRow);
        float M = -INFINITY, den = 0.f, o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 8
        for (int i = 0; i < b.pieces; ++i) {
            const int64_t row = static_cast<int64_t>(2 * (c0 + i) + (i == 0)) * kRows + rr;
            M = fmaxf(M, __ldcg(tp.part_ml + row).x);
        }
#pragma unroll 4
        for (int i = 0; i < b.pieces; ++i) {
            const int64_t row = static_cast<int64_t>(2 * (c0 + i) + (i == 0)) * kRows + rr;
            const float2 ml = __ldcg(tp.part_ml + row);
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(tp.part_o + row * D + d0));
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(tp.part_o + row * D + d0) + 1);
            // (a piece without a visible finite score weighs nothing, but a NaN
            // in its sum or its O stays)
            const float w = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);
            den = fmaf(ml.y, w, den);
            o[0] = fmaf(x.x, w, o[0]);
            o[1] = fmaf(x.y, w, o[1]);
            o[2] = fmaf(x.z, w, o[2]);
            o[3] = fmaf(x.w, w, o[3]);
            o[4] = fmaf(y.x, w, o[4]);
            o[5] = fmaf(y.y, w, o[5]);
            o[6] = fmaf(y.z, w, o[6]);
            o[7] = fmaf(y.w, w, o[7]);
        }
        const float inv = den > 0.f ? 1.f / den : den;
        __half *dst = p.out + (static_cast<int64_t>(b.q0 + (rr >> logG)) * p.num_heads + b.kvh * G +
                               (rr & (G - 1))) * D + d0;
        *reinterpret_cast<uint4 *>(dst) =
            make_uint4(pack_half2(o[0] * inv, o[1] * inv), pack_half2(o[2] * inv, o[3] * inv),
                       pack_half2(o[4] * inv, o[5] * inv), pack_half2(o[6] * inv, o[7] * inv));
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

// The tensor-core kernel and its merge, on `stream`.
int launch_tiles(const TreeParams &t, int D, void *workspace, cudaStream_t stream) {
    TileParams p{};
    p.t = t;
    const int Hk = t.num_kv_heads;
    const int row_bytes = Hk * D * 2;
    int st = dec::make_kv_tensor_map(&p.tm_k, t.k_cache, t.num_blocks, row_bytes, 1);
    if (st == PKV_OK)
        st = dec::make_kv_tensor_map(&p.tm_v, t.v_cache, t.num_blocks, row_bytes, D * 2 / 128);
    if (st == PKV_OK)
        st = dec::make_q_tensor_map(&p.tm_q, t.q, t.num_query_tokens, t.num_heads, D,
                                    t.num_heads / Hk);
    if (st != PKV_OK) return st;
    const int ctas = sm_count();
    const Scratch z = scratch(ctas, D);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.borders = reinterpret_cast<Border *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + z.borders);
    p.part_o = reinterpret_cast<float *>(ws + z.borders + z.ml);
    using Fn = void (*)(const TileParams);
    const Fn fn = D == 128 ? tree_tile_kernel<128> : tree_tile_kernel<64>;
    const int smem = tile_smem_bytes(D);
    st = prepare_kernel(reinterpret_cast<const void *>(fn), kTileThreads, smem, nullptr);
    if (st != PKV_OK) return st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failure(e, "tree_tile_kernel launch");
    if (ctas == 1) return PKV_OK;
    const Fn merge = D == 128 ? tree_merge_kernel<128> : tree_merge_kernel<64>;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), kRows / kMergeRows);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, merge, p);
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
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_query_tokens = num_query_tokens;
    p.max_query_len = max_query_len;
    p.max_seq_len = max_seq_len;
    p.num_blocks = num_blocks;
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;
    if (!fp8)
        return launch_tiles(p, head_dim, workspace, reinterpret_cast<cudaStream_t>(stream));
    using Fn = void (*)(const TreeParams);
    const Fn fn = head_dim == 128 ? tree_rows_kernel<128> : tree_rows_kernel<64>;
    const int64_t warps = static_cast<int64_t>(num_query_tokens) * num_heads;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((warps + 3) / 4));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failure(e, "tree attention launch");
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
