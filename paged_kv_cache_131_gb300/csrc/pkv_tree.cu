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
//  * warp 0 walks the stretch, publishes its pieces, stages a piece's query
//    tile and its keys (tensor copies of 16 rows x 128 bytes, a 3-step ring);
//    warp 1 stages the values (a 3-step ring);
//  * warp 2 issues S = Q K^T into one of two score buffers, so the scores of
//    the next step are computed while the softmax works on this one;
//  * warps 3-10, two threads per row: the softmax of the chunk kernel (running
//    reference maximum that moves by more than 2^8 only, fp16 weights back to
//    tensor memory), with the tree's mask;
//  * warp 11 issues O += P V.  Value rows behind the sequence's end hold
//    anything and are zeroed first; drafted rows may be masked for some query
//    rows, and 0 x NaN is NaN, so their non-finite elements are zeroed too and
//    added, where visible, when the piece's O is read out.
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
    int64_t item0;  // the item's first unit
    int64_t units;  // units of the whole list
    int32_t steps;  // the item's steps; 0: the border cuts no item, or is not
                    // the item's first border
    int32_t rows;   // query rows of the tile
    int32_t q0;     // first query token of the tile
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
struct Piece {
    int seq, kvh, tile, step0;
    int nsteps, nblk, L, Q;
    int q0, slot, done, pad;  // slot: partial state, or -1 for a whole item
};

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
    static constexpr int kOffMisc = kOffFlags + kFlagWords * 4;
    static constexpr int kOffScan = kOffMisc + 16;  // the prologue's words
    static constexpr int kBytes = kOffScan + (kTileThreads / 32 + 2) * 8;
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

// 32 bytes to global memory (32-byte aligned).
__device__ __forceinline__ void store32(void *dst, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Units of an item: its steps and kItemUnits for its start-up.
constexpr int kItemUnits = 1;

// The step a place `x` units into an item falls on.
__device__ __forceinline__ int step_at(int64_t x, int steps) {
    const int64_t s = x - kItemUnits;
    return s <= 0 ? 0 : s >= steps ? steps : static_cast<int>(s);
}

// First unit of CTA c's stretch.
__device__ __forceinline__ int64_t stretch(int64_t units, int c, int ctas) {
    return units * c / ctas;
}

struct SeqGeo {
    int L, Q, q0, tiles, steps;
};

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
    sg.L = L;
    sg.Q = Q;
    sg.q0 = q0;
    sg.tiles = (Q * G + kRows - 1) / kRows;
    sg.steps = (L + kStepKeys - 1) / kStepKeys;
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
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + Gm::kOffMisc);
    int64_t *scan = reinterpret_cast<int64_t *>(smem + Gm::kOffScan);
    volatile int64_t *start = scan + kTileThreads / 32;  // sequence, its first unit

    const int Hk = p.num_kv_heads, H = p.num_heads;
    const int G = H / Hk, logG = __ffs(G) - 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(br.piece_full(s), 1);
            mbar_init(br.piece_empty(s), kPieceReaders);
            mbar_init(br.s_full(s), 1);
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
        mbar_init(br.scanned(), 1);
        fence_mbarrier_init();
        prefetch_tensormap(&tp.tm_k);
        prefetch_tensormap(&tp.tm_v);
        prefetch_tensormap(&tp.tm_q);
    }
    if (warp == 2) {
        tc::tmem_alloc(sb + Gm::kOffMisc, kTmemCols);
        tc::tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();  // the merge: it waits for this grid

    // ---- the list's length, and where this CTA's stretch starts
    int64_t units = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kTileThreads) {
        const int s = s0 + threadIdx.x;
        SeqGeo sg;
        const bool has = s < p.num_seqs && seq_geo(p, s, G, cta == 0, sg);
        int64_t total;
        const int64_t w = has ? seq_units(sg, Hk) : 0;
        const int64_t before = cta_scan(w, scan, total);
        if (p.num_seqs <= kTileThreads) {  // the usual case: one pass
            const int64_t u0 = stretch(total, cta, ctas);
            if (w > 0 && before <= u0 && u0 < before + w) {
                start[0] = s;
                start[1] = before;
            }
        }
        units += total;
    }
    const int64_t u0 = stretch(units, cta, ctas), u1 = stretch(units, cta + 1, ctas);
    if (p.num_seqs > kTileThreads) {
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
            }
            run += total;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = misc[0];
    const int seq0 = static_cast<int>(start[0]);
    const int64_t seq0_unit = start[1];

    if (units == 0) {
        if (threadIdx.x == 0) tp.borders[cta].steps = 0;
    } else if (warp == 0) {
        // ===================== pieces, query tiles and keys =====================
        int seq = seq0;
        int64_t first = seq0_unit;  // the sequence's first unit
        int64_t u = u0;
        SeqGeo sg;
        seq_geo(p, seq, G, false, sg);
        if (lane == 0) {
            // the border at u0, for the merge
            const int64_t n = sg.steps + kItemUnits;
            const int item = static_cast<int>((u0 - first) / n);
            const int64_t a = first + item * n;
            Border b;
            b.item0 = a;
            b.units = units;
            const bool cuts = step_at(u0 - a, sg.steps) > 0 &&
                              (cta == 0 || step_at(stretch(units, cta - 1, ctas) - a, sg.steps) == 0);
            const int tile = item % sg.tiles;
            b.steps = cuts ? sg.steps : 0;
            b.rows = min(kRows, sg.Q * G - tile * kRows);
            b.q0 = sg.q0 + tile * (kRows >> logG);
            b.kvh = item / sg.tiles;
            tp.borders[cta] = b;
        }
        int gs = 0;  // steps staged
        bool ok = true;
        for (int it = 0; ok;) {
            // the next piece
            Piece pc;
            pc.done = 1;
            while (u < u1) {
                const int64_t n = sg.steps + kItemUnits;
                const int64_t item = (u - first) / n;
                if (item >= static_cast<int64_t>(Hk) * sg.tiles) {  // the next sequence with rows
                    first += seq_units(sg, Hk);
                    do ++seq;
                    while (seq < p.num_seqs && !seq_geo(p, seq, G, false, sg));
                    if (seq >= p.num_seqs) {  // (not reached: u1 is inside the list)
                        u = u1;
                        break;
                    }
                    continue;
                }
                const int64_t a = first + item * n;
                const int64_t end = min(u1, a + n);
                const int s0 = step_at(u - a, sg.steps), s1 = step_at(end - a, sg.steps);
                u = end;
                if (s1 == s0) continue;
                pc.seq = seq;
                pc.kvh = static_cast<int>(item) / sg.tiles;
                pc.tile = static_cast<int>(item) % sg.tiles;
                pc.step0 = s0;
                pc.nsteps = s1 - s0;
                pc.nblk = min((sg.L + kBS - 1) / kBS - s0 * kStepBlocks, pc.nsteps * kStepBlocks);
                pc.L = sg.L;
                pc.Q = sg.Q;
                pc.q0 = sg.q0;
                pc.slot = s0 == 0 && s1 == sg.steps ? -1 : 2 * cta + (s0 == 0);
                pc.done = 0;
                break;
            }
            const int rec = it & 1;
            if (it >= 2 && !wait_all(br.piece_empty(rec), ((it >> 1) - 1) & 1)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                pieces[rec] = pc;
                mbar_arrive(br.piece_full(rec));
            }
            if (pc.done) break;
            // its query tile, once the previous piece's last scores are done
            if (it >= 1 && !wait_all(br.q_empty(), (it - 1) & 1)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(br.q_full(), Gm::kQ);
            __syncwarp();
            if (lane < CH)
                tensor_g2s_3d(sb + lane * (kRows * 128), &tp.tm_q, 128 * lane, pc.kvh * G,
                              pc.q0 + pc.tile * (kRows >> logG), br.q_full());
            ++it;
            // its keys: the ids of 32 blocks at a time, one per lane
            const int b0 = pc.step0 * kStepBlocks;
            int ids = lane < pc.nblk ? block_id(p, pc.seq, b0 + lane, true) : -1;
            for (int n = 0; n < pc.nsteps; ++n, ++gs) {
                const int ks = gs % kKStages;
                const int at = n * kStepBlocks;
                if (at != 0 && (at & 31) == 0)
                    ids = at + lane < pc.nblk ? block_id(p, pc.seq, b0 + at + lane, true) : -1;
                if (gs >= kKStages && !wait_all(br.k_empty(ks), ((gs / kKStages) - 1) & 1)) {
                    ok = false;
                    break;
                }
                const int nb = min(kStepBlocks, pc.nblk - at);
                if (lane == 0) mbar_arrive_expect_tx(br.k_full(ks), nb * CH * kBS * 128);
                __syncwarp();
                // lane l: block l / CH of the step, chunk l % CH (a bad block
                // reads rows before the cache: zeros)
                const int b = min(lane / CH, kStepBlocks - 1), c = lane % CH;
                const int id = __shfl_sync(0xffffffffu, ids, (at & 31) + b);
                if (lane < nb * CH)
                    tensor_g2s_3d(sb + Gm::kOffK + ks * Gm::kK + c * (kStepKeys * 128) +
                                      b * (kBS * 128),
                                  &tp.tm_k, 0, id >= 0 ? id * kBS : -kBS, pc.kvh * CH + c,
                                  br.k_full(ks));
            }
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
            const Piece pc = pieces[rec];
            __syncwarp();
            if (lane == 0) mbar_arrive(br.piece_empty(rec));
            if (pc.done) break;
            const int b0 = pc.step0 * kStepBlocks;
            int ids = lane < pc.nblk ? block_id(p, pc.seq, b0 + lane, false) : -1;
            for (int n = 0; n < pc.nsteps; ++n, ++gs) {
                const int vs = gs % kVStages;
                const int at = n * kStepBlocks;
                if (at != 0 && (at & 31) == 0)
                    ids = at + lane < pc.nblk ? block_id(p, pc.seq, b0 + at + lane, false) : -1;
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
        // ============================ score MMAs ============================
        int gs = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int rec = it & 1;
            if (!wait_all(br.piece_full(rec), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const int done = pieces[rec].done, nsteps = pieces[rec].nsteps, nblk = pieces[rec].nblk;
            __syncwarp();
            if (lane == 0) mbar_arrive(br.piece_empty(rec));
            if (done) break;
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
                    tc::commit(br.k_empty(ks));
                    if (n == nsteps - 1) tc::commit(br.q_empty());
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, cta);
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
            const Piece pc = pieces[rec];
            __syncwarp();
            if (lane == 0) mbar_arrive(br.piece_empty(rec));
            if (pc.done) break;
            const int ctx = pc.L - pc.Q;
            for (int n = 0; n < pc.nsteps && ok; ++n, ++gs) {
                const int vs = gs % kVStages, b = gs & 1;
                const int nb = min(kStepBlocks, pc.nblk - n * kStepBlocks);
                // the previous piece's O and flags have been read
                if (n == 0) {
                    if (it > 0) ok = wait_all(br.o_free(), (it - 1) & 1);
                    if (!ok) break;
                    if (lane < kFlagWords) flags[lane] = 0;
                    __syncwarp();
                }
                ok = wait_all(br.v_full(vs), (gs / kVStages) & 1);
                if (!ok) break;
                const uint32_t v_s = sb + Gm::kOffV + vs * Gm::kV;
                const int key0 = (pc.step0 + n) * kStepKeys;
                if (key0 + nb * kBS > ctx) {
                    // rows at and past the end: zeroed; drafted rows: their
                    // non-finite elements zeroed and the row flagged
                    uint8_t *vb = smem + Gm::kOffV + vs * Gm::kV;
                    const int r0 = max(ctx - key0, 0);
                    constexpr int kUnits = 8 * CH;  // 16-byte units of a row
                    for (int i = r0 * kUnits + lane; i < nb * kBS * kUnits; i += 32) {
                        const int t = i / kUnits, un = i % kUnits;
                        uint4 *at = reinterpret_cast<uint4 *>(
                            vb + (t >> 4) * Gm::kVBlock + (un >> 3) * (kBS * 128) + (t & 15) * 128 +
                            (un & 7) * 16);
                        const int key = key0 + t;
                        if (key >= pc.L) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        } else {
                            uint4 x = *at;
                            uint32_t *w = reinterpret_cast<uint32_t *>(&x);
                            bool bad = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((w[e] & 0x7C00u) == 0x7C00u) {
                                    w[e] &= 0xFFFF0000u;
                                    bad = true;
                                }
                                if ((w[e] & 0x7C000000u) == 0x7C000000u) {
                                    w[e] &= 0x0000FFFFu;
                                    bad = true;
                                }
                            }
                            if (bad) {
                                *at = x;
                                atomicOr(&flags[(key - ctx) >> 5], 1u << ((key - ctx) & 31));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (n == pc.nsteps - 1 && lane == 0) mbar_arrive(br.scanned());
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
            const Piece pc = pieces[rec];
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
            float m_used = -INFINITY, l = 0.f;  // l: this thread's keys only

            for (int n = 0; n < pc.nsteps; ++n, ++gs) {
                const int sbuf = gs & 1;
                const int at = n * kStepBlocks;
                const int nb = min(kStepBlocks, pc.nblk - at);
                const int key0 = (pc.step0 + n) * kStepKeys;
                // the step's blocks in range, and this thread's visible keys:
                // looked up while the scores are computed
                const bool good = lane >= nb || block_id(p, pc.seq, pc.step0 * kStepBlocks + at + min(lane, nb - 1), false) >= 0;
                const uint32_t blocks = __ballot_sync(0xffffffffu, good);
                const bool fast = blocks == 0xffffffffu && key0 + kStepKeys <= ctx && sl2 >= 0.f;
                uint64_t vis = ~0ull;
                if (!fast && live) {
                    vis = visible(mask, p.mask_words, key0 + kHalfKeys * h, ctx, pc.L);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (!((blocks >> (4 * h + b)) & 1u)) vis &= ~(0xFFFFull << (16 * b));
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
                tc::wait_ld();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(br.s_free(sbuf));
                if (!fast) {
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
            uint32_t flagged[kFlagWords];
            bool any = false;
#pragma unroll
            for (int w = 0; w < kFlagWords; ++w) {
                flagged[w] = flags[w];
                any = any || flagged[w] != 0;
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(br.o_free());
            l += __shfl_xor_sync(0xffffffffu, l, 16);  // the row's sum over both halves' keys
            if (any && row_ok) {
                // the elements that were left out: a weight times an infinity
                // or a NaN is that, whatever the (positive) weight
                for (int w = 0; w < kFlagWords; ++w)
                    for (uint32_t bits = flagged[w]; bits; bits &= bits - 1) {
                        const int node = 32 * w + __ffs(bits) - 1;
                        if (!((__ldg(mask + node / 64) >> (node & 63)) & 1)) continue;
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
            if (!row_ok) continue;
            if (pc.slot < 0) {
                const float inv = l > 0.f ? 1.f / l : l;  // (no visible key: 0; NaN stays)
                __half *dst = p.out + (static_cast<int64_t>(pc.q0 + j) * H + pc.kvh * G +
                                       (rr & (G - 1))) * D + DH * h;
#pragma unroll
                for (int c = 0; c < DH / 16; ++c) {
                    uint32_t x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = pack_half2(o[16 * c + 2 * e] * inv, o[16 * c + 2 * e + 1] * inv);
                    *reinterpret_cast<uint4 *>(dst + 16 * c) = make_uint4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<uint4 *>(dst + 16 * c + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                }
            } else {
                const int64_t row = static_cast<int64_t>(pc.slot) * kRows + r;
                if (h == 0) tp.part_ml[row] = make_float2(m_used, l);
                float *dst = tp.part_o + row * D + DH * h;
#pragma unroll
                for (int c = 0; c < DH / 8; ++c) {
                    uint32_t x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(o[8 * c + e]);
                    store32(dst + 8 * c, x);
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
// to cut.  D/8 threads per row, 8 dims each; the item's pieces are those of the
// CTAs from b on whose stretch holds some of its steps.
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    tree_merge_kernel(const __grid_constant__ TileParams tp, int ctas) {
    constexpr int kPerRow = D / 8;
    constexpr int kPass = kMergeThreads / kPerRow;  // rows at a time
    grid_dependency_wait();
    const int c0 = blockIdx.x;  // the CTA that holds the item's first steps
    const Border b = tp.borders[c0 + 1];
    if (b.steps == 0) return;
    const TreeParams &p = tp.t;
    const int G = p.num_heads / p.num_kv_heads, logG = __ffs(G) - 1;
    const int last = static_cast<int>(((b.item0 + b.steps + kItemUnits) * ctas - 1) / b.units);
    for (int rr = blockIdx.y * kMergeRows + threadIdx.x / kPerRow;
         rr < min(b.rows, static_cast<int>(blockIdx.y + 1) * kMergeRows); rr += kPass) {
        const int d0 = 8 * (threadIdx.x % kPerRow);
        float M = -INFINITY, den = 0.f, o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
        // pieces c0 .. last; the first one's state is in its CTA's second slot
        for (int c = c0; c <= last; ++c) {
            const int s0 = step_at(stretch(b.units, c, ctas) - b.item0, b.steps);
            const int s1 = step_at(stretch(b.units, c + 1, ctas) - b.item0, b.steps);
            if (s0 == s1) continue;
            const int64_t row = static_cast<int64_t>(2 * c + (s0 == 0)) * kRows + rr;
            M = fmaxf(M, __ldcg(tp.part_ml + row).x);
        }
        for (int c = c0; c <= last; ++c) {
            const int s0 = step_at(stretch(b.units, c, ctas) - b.item0, b.steps);
            const int s1 = step_at(stretch(b.units, c + 1, ctas) - b.item0, b.steps);
            if (s0 == s1) continue;
            const int64_t row = static_cast<int64_t>(2 * c + (s0 == 0)) * kRows + rr;
            const float2 ml = __ldcg(tp.part_ml + row);
            // (a piece without a visible finite score weighs nothing, but a NaN
            // in its sum or its O stays)
            const float w = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);
            den = fmaf(ml.y, w, den);
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(tp.part_o + row * D + d0));
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(tp.part_o + row * D + d0) + 1);
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
    using MergeFn = void (*)(const TileParams, int);
    const MergeFn merge = D == 128 ? tree_merge_kernel<128> : tree_merge_kernel<64>;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), kRows / kMergeRows);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, merge, p, ctas);
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
        !aligned(workspace, 32))
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
