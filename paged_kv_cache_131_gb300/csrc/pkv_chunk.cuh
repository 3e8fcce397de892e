// pkv_chunk.cuh -- the tile kernel (instantiated by pkv_chunk.cu, and under score
// rules by pkv_chunk_rules.cu) of attention of a chunk of new tokens per sequence over the
// paged cache, causal within the new tokens ("vLLM 技术内幕" §3.2: chunked
// prefill, prompt and output tokens scheduled alike; §7.4: draft tokens
// verified together).  Sequence i holds L tokens, the last Q of them new;
// new token j (position L - Q + j) attends to positions 0 .. L - Q + j.
//
// Sequences whose new tokens times the group size fit the balanced decode
// schedule's query columns (8 or 16: MmaColsPolicy) run there -- the same
// streaming of whole token rows as a decode; the others run here, on the
// fifth-generation tensor cores (tcgen05) with accumulators in tensor memory.
//
// The work is a list of items (query tile of 128 rows, KV head, KV
// partition of 4096 tokens, sequence), built on the device by a one-CTA plan
// kernel for the sequences this kernel takes (partitions past a tile's
// causal range are not items).  Persistent CTAs (one per SM) pull items in
// list order from an atomic counter, so tiles with more keys and tiles with
// fewer balance out.  A row is (new token j, query head g of the KV head's
// group): row = j*G + g, so a tile covers 128/G consecutive new tokens.
// When both kernels have work, the plan kernel also estimates each one's
// share and picks how many SMs the balanced schedule gets; this kernel's
// last that-many CTAs leave at once and the balanced grid uses only its
// first that-many, so the two run side by side on disjoint SMs.
//
// Per CTA, warp-specialised, all hand-offs through mbarriers:
//  * warp 0 takes the items (the next one when the current one's last step
//    is staged; the longest items are handed out first), stages the tile's
//    query rows into shared memory and the partition's
//    keys, 8 blocks (128 keys) per step, one tensor copy per block and
//    64-dimension chunk, into a 4-step ring laid out [chunk][key][128 B] so
//    the 128 keys form one MMA operand;
//  * warp 1 stages the values, one tensor copy per block, into a 2-step ring;
//  * warp 2 (one thread) copies the query tile into tensor memory (two
//    tiles in flight) and issues per step S = Q K^T (M = 128 rows, N = 128
//    keys, one MMA per 16-dimension k step, A read from tensor memory) into
//    a 128-column score buffer; warp 11 (one thread) issues O += P V
//    (N = head_dim, 16 keys per MMA) with the weights P read from tensor
//    memory (two buffers).  An MMA that depends on the previous one holds
//    its issuer back, so each chain has its own issuing warp;
//  * warps 3-10 run the softmax, two threads of one warp per query row,
//    each with half of each step's keys (tensor-memory loads of two 16-lane
//    halves): they read the row's scores, mask keys past the row's position
//    (and past the sequence or in a bad block), combine the two half-row
//    maxima with one shuffle, keep the row's running maximum m and the sums
//    l in the log2 domain and write the fp16 weights P = 2^(s - m) back to
//    tensor memory.  The reference m moves only when the maximum grows by
//    more than 2^8 (the weights stay <= 256): then each thread rescales its
//    half of the row's O in tensor memory first.  The result O / l does not
//    depend on which reference was used.
// A tile whose range fits one partition writes fp16 out; otherwise
// every partition leaves fp32 partial states (m, l, O) and, per softmax warp,
// the last CTA of the tile to take a ticket merges them with a log-sum-exp
// rescale.  No CTA waits for another.
//
// Under score rules (pkv_score_rules) the same, but
//  * a tile's keys are a list of blocks (Span): the prefix's, then those from the
//    first row's window on; partitions of 8192 tokens divide that list, and an item
//    whose partition the list does not reach is passed over when it is taken;
//  * the softmax applies the rules to the scores (rule_scores); most steps are seen
//    whole by every row (Clear) and pass the masks over;
//  * a step that is not has its value blocks' elements that are not finite zeroed
//    before the MMAs and added at the end by the rows that see them.
// What bounds it (4 x 2048 new tokens of up to 8192, H 32, Hk 8, D 128, clock reads in
// a copy, cycles a step of 2700 with a cap): the softmax warps, two a scheduler: the
// scores' extremes 700, weights 1150 (690 without a cap: its polynomial is four packed
// multiply-adds a pair), scores' load 190, votes and waits 300, an item's output 430;
// issue slots 39% busy, tensor pipe 28%.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/pagedkv.h"
#include "pkv_decode_common.cuh"
#include "pkv_decode_host.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace chunk {

using dec::kBS;
using dec::kNegInf;

constexpr int kRows = 128;                     // query rows per tile: the MMA's M
constexpr int kStepBlocks = 8;                 // blocks per step
constexpr int kStepKeys = kStepBlocks * kBS;   // 128 keys: the score MMA's N
constexpr int kKStages = 4;                    // key ring depth (steps)
constexpr int kVStages = 2;                    // value ring depth (steps)
constexpr int kPartTokens = 4096;              // KV partition
constexpr int kClaimLead = 1;                  // steps staged after the next item is claimed
constexpr int kPartBlocks = kPartTokens / kBS;
// under rules partitions are twice as long: an item that leaves a partial state costs
// its softmax warps about 8 us (stores, ticket, merge), a tenth of a partition's steps
constexpr int kRulePartBlocks = 2 * kPartBlocks;
template <bool kRules>
constexpr int part_blocks = kRules ? kRulePartBlocks : kPartBlocks;
// softmax: eight warps; warp 3 + 4 wh + q takes the rows (tensor-memory
// lanes) 32 q + 16 wh .. + 15, two threads per row: lanes 16 h + i take keys
// 64 h .. 64 h + 63 of a step and the head dimensions (D/2) h .. of O
constexpr int kSoftmaxWarps = 8;
constexpr int kGroupKeys = kStepKeys / 2;
constexpr int kPVWarp = 3 + kSoftmaxWarps;  // issues the P V MMAs (warp 2 the score MMAs)
constexpr int kThreads = (4 + kSoftmaxWarps) * 32;
// tensor memory: O in columns [0, head_dim), the scores in [128, 256), the
// weights (fp16 pairs) in two buffers of 64 columns, the query tile (fp16
// pairs, copied from shared memory) in two buffers of 64 columns
constexpr int kTmemCols = 512;
constexpr int kTmemO = 0;
constexpr int kTmemS = 128;
constexpr int kTmemP = 256;
constexpr int kTmemQ = 384;
constexpr float kRescaleLog2 = 8.f;            // move the reference past 2^8
// Under score rules the weights stand 2^7 higher (2^7 to 2^15, the row's largest):
// fp16 then is off by 2^-32 of the largest at most where it loses bits (a capped or
// biased row can spread much of its mass over many small weights).  Standing 2^11
// higher and moving past 2^4 instead cost a tenth of the time: with 5000 normal
// scores every fourth row's maximum grows by that, and a warp waits for any of its 16.
constexpr float kRuleShiftLog2 = 7.f;
// rates of the split between the call's two kernels (see the plan kernel)
// (single precision: this GPU's double-precision rate is low)
constexpr float kHbmBytesPerUs = 6.0e6f;        // decode stream, whole GPU
constexpr float kSmBytesPerUs = 58.0e3f;        // decode stream per SM
constexpr float kTileStepUs = 1.3f;             // one 128-key step of a tile

struct ChunkParams {
    CUtensorMap tm_k;  // keys: one 128-byte chunk of 16 rows per copy
    CUtensorMap tm_v;  // values: a head's chunks of 16 rows per copy
    CUtensorMap tm_q;  // query rows: 128 bytes of each row of a 128-row tile
    __half *out;
    const __half *q;
    const int32_t *block_tables;
    const int32_t *seq_lens;
    const int32_t *query_start;
    float scale_log2;
    int num_heads;
    int num_kv_heads;
    int max_blocks_per_seq;
    int max_query_len;
    int max_seq_len;
    int num_tiles;  // tiles per (sequence, kv head) the tickets are sized for
    int num_parts;  // KV partitions the partial states are sized for
    int num_query_tokens;
    int min_rows;   // sequences with fewer rows (new tokens x group) are not ours
    int num_seqs;
    int head_dim;
    int num_ctas;    // CTAs the tile kernel is launched with
    int max_cols;    // rows the balanced schedule takes per (sequence, kv head); 0: none
    // work list: the sequences taken here (big_seq[k]) and the exclusive
    // prefix of their item counts (big_cum[k], big_cum[n_big] = total items);
    // *work is the next item to hand out
    int *big_seq;
    int *big_cum;
    int *n_big;
    int *work;
    // SMs left to the balanced schedule's share of the call (written by the
    // plan kernel; that many tile CTAs exit at once)
    int *split;
    int64_t num_blocks;
    int *counters;    // [S][Hk][num_tiles][8] tickets (one per softmax warp), zero between calls
    // partial states, row index R = kv_head * Tq * G + query_start * G + tile
    // row (the rows of a half-warp are consecutive): (m, l) [2 halves][parts][R]
    // (each half-warp keeps a copy), O [parts][D][R]
    float2 *part_ml;
    float *part_o;
    ErrorRecord *err;
    // score rules (the kernels under rules only)
    dec::RuleParams rules;
    const __half *v_cache;
};

// An item as the producer hands it to the other warps.
struct ItemInfo {
    int seq, part, kvh, tile;
    int nsteps, nblk, L, Q;
    int q0, nparts, done, prefix;
    uint32_t valid[kPartBlocks / 32];  // one bit per block of the partition: id in range
    int pb, skip;    // (under rules) see Span
    int all_valid;   // (under rules) every id in range
    int pad;
};

// Shared memory (from a 1024-aligned base): the query tile being staged,
// the key ring, the value ring, the mbarriers, two item records and a few
// words.
template <int D>
struct Geo {
    static constexpr int kChunks = D / 64;                   // 128-byte chunks of a head row
    static constexpr int kQ = kChunks * kRows * 128;         // [chunk][row][128 B]
    static constexpr int kK = kChunks * kStepKeys * 128;     // [chunk][key][128 B]
    static constexpr int kVBlock = kChunks * kBS * 128;      // [chunk][token][128 B]
    static constexpr int kV = kStepBlocks * kVBlock;
    static constexpr int kOffK = kQ;
    static constexpr int kOffV = kOffK + kKStages * kK;
    static constexpr int kOffBar = kOffV + kVStages * kV;
    static constexpr int kBars = 2 + 2 + 1 + 1 + 2 * kKStages + 2 * kVStages + 1 + 1 + 2 + 2 + 1;
    static constexpr int kOffInfo = kOffBar + kBars * 8;
    static constexpr int kOffMisc = kOffInfo + 2 * static_cast<int>(sizeof(ItemInfo));
    static constexpr int kBytes = kOffMisc + 16;
};

inline int smem_bytes(int D) {
    return dec::kTileAlign + (D == 128 ? Geo<128>::kBytes : Geo<64>::kBytes);
}

// mbarrier addresses (shared space) by role
struct Bars {
    uint32_t b;
    // item records: published / read by every role
    __device__ uint32_t q_full(int s) const { return b + 8 * s; }
    __device__ uint32_t q_empty(int s) const { return b + 8 * (2 + s); }
    // the query tile in shared memory: landed / copied to tensor memory
    __device__ uint32_t qs_full() const { return b + 8 * 4; }
    __device__ uint32_t qs_empty() const { return b + 8 * 5; }
    __device__ uint32_t k_full(int s) const { return b + 8 * (6 + s); }
    __device__ uint32_t k_empty(int s) const { return b + 8 * (6 + kKStages + s); }
    __device__ uint32_t v_full(int s) const { return b + 8 * (6 + 2 * kKStages + s); }
    __device__ uint32_t v_empty(int s) const { return b + 8 * (6 + 2 * kKStages + kVStages + s); }
    static constexpr int kS = 6 + 2 * kKStages + 2 * kVStages;
    __device__ uint32_t s_full() const { return b + 8 * kS; }
    __device__ uint32_t s_free() const { return b + 8 * (kS + 1); }
    __device__ uint32_t p_full(int s) const { return b + 8 * (kS + 2 + s); }
    __device__ uint32_t pv_done(int s) const { return b + 8 * (kS + 4 + s); }
    __device__ uint32_t o_free() const { return b + 8 * (kS + 6); }
};

// arrivals that free an item record: the value producer, the two MMA warps
// and every softmax warp, once each has read it
constexpr int kQEmptyArrivals = 3 + kSoftmaxWarps;

// Every lane waits (bounded); false if any lane gave up.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed fp32 pairs (the f32x2 forms of sm_100 and later: one instruction for
// two lanes' worth of fma or add) and the three-input maximum.

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

// a * b + c per lane, round to nearest
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
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

__device__ __forceinline__ float fmin3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Geometry of sequence s for this kernel; false if the sequence is not
// ours (too few rows) or invalid (recorded when `report`, which the plan passes; the
// items' takers look at listed sequences alone).
struct SeqGeo {
    int L, Q, q0, rows, tiles, parts;
    int prefix;  // (under rules) positions below are seen by every token, <= L
};

template <bool kRules>
__device__ __forceinline__ bool seq_geo(const ChunkParams &p, int s, int G, bool report,
                                        SeqGeo &sg) {
    const int L = __ldg(p.seq_lens + s);
    const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1);
    const bool in = q0 >= 0 && q1 >= q0 && q1 <= p.num_query_tokens;  // (so q1 - q0 fits)
    const int Q = in ? q1 - q0 : 0;
    if (in && L == 0) return false;  // left out of the call, whatever its rows
    if (!in || L < 0 || L > p.max_blocks_per_seq * kBS || L > p.max_seq_len || Q > L ||
        Q > p.max_query_len ||
        (report && dec::starts_fall(p.query_start, s, q0, p.num_query_tokens))) {
        if (report) record_error(p.err, PKV_DEVERR_SEQ_LEN, s);
        return false;
    }
    sg.L = L;
    sg.Q = Q;
    sg.q0 = q0;
    sg.rows = Q * G;
    if (sg.rows < p.min_rows || sg.rows == 0) return false;
    sg.tiles = (sg.rows + kRows - 1) / kRows;
    constexpr int kTokens = part_blocks<kRules> * kBS;
    sg.parts = (L + kTokens - 1) / kTokens;
    sg.prefix = 0;
    if constexpr (kRules) {
        if (p.rules.prefix_lens != nullptr)
            sg.prefix = max(0, min(L, __ldg(p.rules.prefix_lens + s)));
        if (p.rules.window < L) {
            // a tile's window spans window + 128 / G - 1 positions at most
            const int most = (sg.prefix + kBS - 1) / kBS +
                             (p.rules.window + kRows / G) / kBS + 2;
            sg.parts = min(sg.parts, (most + kRulePartBlocks - 1) / kRulePartBlocks);
        }
    }
    return true;
}

// Under rules: the blocks that some row of a tile sees, in order -- the first pb
// (the prefix's) and, `skip` blocks later, those from the first row's window to
// the last row's position; nblk in all.  Partitions divide this list.
struct Span {
    int pb, skip, nblk;
};

__device__ __forceinline__ int span_block(int pb, int skip, int v) { return v < pb ? v : v + skip; }

__device__ __forceinline__ Span tile_span(const SeqGeo &sg, int tile, int G, int window) {
    const int a0 = sg.L - sg.Q + tile * (kRows / G);  // positions of the first
    const int a1 = sg.L - sg.Q + (min(sg.rows, (tile + 1) * kRows) - 1) / G;  // and last row
    Span sp;
    sp.pb = (sg.prefix + kBS - 1) / kBS;
    const int end = a1 / kBS + 1, w0 = max(0, a0 - window + 1) / kBS;
    sp.skip = max(0, w0 - sp.pb);
    sp.nblk = sp.skip > 0 ? sp.pb + end - w0 : max(end, sp.pb);
    return sp;
}

// Whether every row of a tile (positions a0 .. a1) sees all keys of the block
// that starts at kp.
__device__ __forceinline__ bool seen_whole(int kp, int a0, int a1, int window, int prefix) {
    return kp + kBS <= prefix || (kp + kBS - 1 <= a0 && a1 - kp < window);
}

// The same for places of the tile's list at once: every row sees the blocks at places
// [from, to) whole, and those below `prefix` whole; `past` as `to` for the latter's
// blocks that no row is before.
struct Clear {
    int from, to, prefix, past;
    __device__ __forceinline__ bool has(int v, int n) const {
        return (v >= from && v + n <= to) || v + n <= prefix;
    }
    __device__ __forceinline__ bool has_past(int v, int n) const {
        return (v >= from && v + n <= to) || v + n <= past;
    }
};

__device__ __forceinline__ Clear clear_of(int pb, int skip, int a0, int a1, int window,
                                          int prefix) {
    Clear c;
    const int low = a1 >= window ? (a1 - window + 1 + kBS - 1) / kBS - skip : 0;
    c.from = skip > 0 ? max(pb, low) : low;
    c.to = (a0 + 1) / kBS - skip;
    c.prefix = prefix / kBS;
    c.past = min(c.prefix, (a0 + 1) / kBS);
    return c;
}

// First query tile that needs KV partition `part` (its last token reaches
// the partition): tile t's last token j_last(t) = (min(rows, 128(t+1)) - 1)/G
// sees keys up to L - Q + j_last(t).
__device__ __forceinline__ int first_tile(const SeqGeo &sg, int part, int G) {
    const int x = part * kPartTokens - (sg.L - sg.Q);  // j_last must reach x
    if (x <= 0) return 0;
    const int t = (x * G + 1 + kRows - 1) / kRows - 1;
    return min(sg.tiles - 1, max(0, t));
}

template <bool kRules>
__device__ __forceinline__ int seq_items(const SeqGeo &sg, int G, int Hk) {
    // (under rules: every partition of every tile; the empty ones are passed over
    // when they are taken)
    if constexpr (kRules) return sg.parts * sg.tiles * Hk;
    int n = 0;
    for (int pt = 0; pt < sg.parts; ++pt) n += sg.tiles - first_tile(sg, pt, G);
    return n * Hk;
}

// One CTA: the list of the sequences this kernel takes and their item counts.
template <bool kRules>
__global__ void __launch_bounds__(1024) chunk_plan_kernel(const __grid_constant__ ChunkParams p,
                                                          int G) {
    __shared__ int wsum[32];
    __shared__ int run[2];  // sequences listed, items listed
    // work of the two kernels of the call: key/value blocks the balanced
    // schedule streams, and 128-key steps of the tile kernel's items
    __shared__ unsigned long long dec_blocks;
    __shared__ float tile_steps;
    // sequences of several partitions, whose tiles' tickets are set to zero here: the
    // workspace may hold another call's partial states there
    __shared__ int cut_seq[1024], cut_tiles[1024], cuts;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        run[0] = run[1] = 0;
        cuts = 0;
        dec_blocks = 0ull;
        tile_steps = 0.f;
    }
    __syncthreads();
    for (int s0 = 0; s0 < p.num_seqs; s0 += blockDim.x) {
        const int s = s0 + threadIdx.x;
        SeqGeo sg;
        const bool mine = s < p.num_seqs && seq_geo<kRules>(p, s, G, true, sg);
        const int cnt = mine ? seq_items<kRules>(sg, G, p.num_kv_heads) : 0;
        if (mine && sg.parts > 1) {
            const int e = atomicAdd(&cuts, 1);
            cut_seq[e] = s;
            cut_tiles[e] = sg.tiles;
        }
        float my_steps = 0.f;
        unsigned long long my_dec = 0;
        if (mine) {
            // 128-key steps of the sequence's items, estimated in closed form:
            // tile t (128/G new tokens each, the last one clipped) sees
            // L - Q + min(Q, (t + 1) 128/G) keys, plus on average half a step
            // of rounding per (tile, partition) item
            const float R = static_cast<float>(kRows / G), nt = static_cast<float>(sg.tiles);
            const float keys = nt * static_cast<float>(sg.L - sg.Q) +
                               R * nt * (nt - 1.f) * 0.5f + static_cast<float>(sg.Q);
            my_steps = keys * (1.f / kStepKeys) * static_cast<float>(p.num_kv_heads) +
                       0.5f * static_cast<float>(cnt);
            if constexpr (kRules) {
                // from the first, middle and last tile's blocks
                const int w = p.rules.window;
                const float b = static_cast<float>(tile_span(sg, 0, G, w).nblk) +
                                4.f * static_cast<float>(tile_span(sg, sg.tiles / 2, G, w).nblk) +
                                static_cast<float>(tile_span(sg, sg.tiles - 1, G, w).nblk);
                my_steps = nt * static_cast<float>(p.num_kv_heads) *
                           (b * (1.f / (6.f * kStepBlocks)) + 0.5f);
            }
        } else if (s < p.num_seqs && p.max_cols > 0) {
            const int L = __ldg(p.seq_lens + s);
            const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1);
            const int Q = q0 >= 0 && q1 >= q0 && q1 <= p.num_query_tokens ? q1 - q0 : 0;
            if (Q > 0 && Q <= L && Q <= p.max_cols / G && L <= p.max_blocks_per_seq * kBS)
                my_dec = static_cast<unsigned long long>((L + kBS - 1) / kBS);
            if constexpr (kRules) {
                if (my_dec > 0) {
                    const int pl = p.rules.prefix_lens != nullptr
                                       ? max(0, min(L, __ldg(p.rules.prefix_lens + s)))
                                       : 0;
                    my_dec -= max(0, max(0, L - Q - p.rules.window + 1) / kBS -
                                         (pl + kBS - 1) / kBS);
                }
            }
        }
        // one shared atomic per warp and counter
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            my_steps += __shfl_xor_sync(0xffffffffu, my_steps, o);
            my_dec += __shfl_xor_sync(0xffffffffu, my_dec, o);
        }
        if (lane == 0 && my_steps > 0.f) atomicAdd(&tile_steps, my_steps);
        if (lane == 0 && my_dec) atomicAdd(&dec_blocks, my_dec);
        // two exclusive scans at once: (is listed, items) packed in one int2
        int a = mine ? 1 : 0, c = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int ya = __shfl_up_sync(0xffffffffu, a, o);
            const int yc = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o) {
                a += ya;
                c += yc;
            }
        }
        __shared__ int wa[32];
        if (lane == 31) {
            wa[warp] = a;
            wsum[warp] = c;
        }
        __syncthreads();
        if (warp == 0) {
            const int nw = blockDim.x >> 5;
            int va = lane < nw ? wa[lane] : 0, vc = lane < nw ? wsum[lane] : 0;
            int ia = va, ic = vc;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int ya = __shfl_up_sync(0xffffffffu, ia, o);
                const int yc = __shfl_up_sync(0xffffffffu, ic, o);
                if (lane >= o) {
                    ia += ya;
                    ic += yc;
                }
            }
            if (lane < nw) {
                wa[lane] = ia - va;
                wsum[lane] = ic - vc;
            }
        }
        __syncthreads();
        const int ea = run[0] + wa[warp] + a - (mine ? 1 : 0);
        const int ec = run[1] + wsum[warp] + c - cnt;
        // launched as a programmatic dependent: the lengths and offsets above
        // may be read while the previous kernel (the cache write) finishes,
        // but nothing is written before it has completed -- which also makes
        // this kernel's completion imply that kernel's for the ones after it
        if (s0 == 0) grid_dependency_wait();
        if (mine) {
            p.big_seq[ea] = s;
            p.big_cum[ea] = ec;
        }
        // (a warp takes a sequence's KV head: 32 bytes a tile)
        for (int i = warp; i < cuts * p.num_kv_heads; i += static_cast<int>(blockDim.x >> 5)) {
            const int e = i / p.num_kv_heads, kvh = i - e * p.num_kv_heads;
            uint4 *at = reinterpret_cast<uint4 *>(
                p.counters + (static_cast<int64_t>(cut_seq[e]) * p.num_kv_heads + kvh) *
                                 p.num_tiles * kSoftmaxWarps);
            for (int j = lane; j < cut_tiles[e] * (kSoftmaxWarps / 4); j += 32)
                at[j] = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncthreads();
        if (threadIdx.x == blockDim.x - 1) {
            run[0] = ea + (mine ? 1 : 0);
            run[1] = ec + cnt;
            cuts = 0;
        }
        __syncthreads();
    }
    grid_dependency_wait();  // (returns at once if the loop waited already)
    if (threadIdx.x == 0) {
        p.big_cum[run[0]] = run[1];
        *p.n_big = run[0];
        *p.work = 0;
    }
    // SMs for the balanced schedule: the split that evens the two kernels'
    // estimated times when they run side by side.  Decode: its bytes at
    // min(HBM rate, SMs x per-SM rate); tile: its steps at a per-step cost
    // over the remaining SMs, plus half an average item for the last wave.
    // Rates measured on this GPU (chunked prefill beside decodes: the decode
    // kernel streams ~58 GB/s per SM when it shares the GPU; a tile step
    // costs ~1-1.5 us beside it, 1.2-1.3 gave the shortest calls, 1.1 far
    // longer ones).  Thread i tries 2 + 2i SMs; the smallest estimate wins
    // (ties: fewer SMs).
    __shared__ unsigned long long best_w[32];
    unsigned long long key = ~0ull;
    if (dec_blocks > 0) {
        const int b = 2 + 2 * static_cast<int>(threadIdx.x);
        if (b < p.num_ctas) {
            const float dec_bytes = static_cast<float>(dec_blocks) * kBS * p.num_kv_heads *
                                    p.head_dim * 2 * 2;
            const float steps = tile_steps;
            const float items = fmaxf(1.f, static_cast<float>(run[1]));
            const float tail = 0.5f * __fdividef(steps, items) * kTileStepUs;
            const float t_dec = __fdividef(dec_bytes, fminf(kHbmBytesPerUs, b * kSmBytesPerUs));
            const float t_tile =
                __fdividef(steps * kTileStepUs, static_cast<float>(p.num_ctas - b)) + tail;
            // (non-negative floats order as their bits)
            key = (static_cast<unsigned long long>(__float_as_uint(fmaxf(t_dec, t_tile))) << 32) |
                  static_cast<unsigned>(b);
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const unsigned long long y = __shfl_xor_sync(0xffffffffu, key, o);
        key = y < key ? y : key;
    }
    if (lane == 0) best_w[warp] = key;
    __syncthreads();
    if (warp == 0) {
        unsigned long long k = lane < static_cast<int>(blockDim.x >> 5) ? best_w[lane] : ~0ull;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const unsigned long long y = __shfl_xor_sync(0xffffffffu, k, o);
            k = y < k ? y : k;
        }
        if (lane == 0) *p.split = k == ~0ull ? 0 : static_cast<int>(k & 0xffffffffu);
    }
}

// Block ids of an item's partition: lane l holds blocks l, 32 + l, .. of it; -1 past
// the item or out of range (recorded when `report`).
// (pb, skip: under rules the list of blocks is a tile's Span.)
template <int W>
__device__ __forceinline__ void load_ids(const ChunkParams &p, int seq, int blo, int nblk,
                                         int lane, bool report, int (&ids)[W], int pb = 0,
                                         int skip = 0) {
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int b = w * 32 + lane;
        int id = -1;
        if (b < nblk) {
            const int64_t at = static_cast<int64_t>(seq) * p.max_blocks_per_seq +
                               span_block(pb, skip, blo + b);
            id = __ldg(p.block_tables + at);
            if (id < 0 || static_cast<int64_t>(id) >= p.num_blocks) {
                if (report) record_error(p.err, PKV_DEVERR_BLOCK_ID, at);
                id = -1;
            }
        }
        ids[w] = id;
    }
}

// Block b's id (every lane calls).
template <int W>
__device__ __forceinline__ int id_of(const int (&ids)[W], int b) {
    int v = -1;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int x = __shfl_sync(0xffffffffu, ids[w], b & 31);
        if ((b >> 5) == w) v = x;
    }
    return v;
}

// The (partition, kv head, tile) of item `local` of a sequence: partition-
// major, then tile (the last first), then kv head.
__device__ __forceinline__ int3 decode_item(const SeqGeo &sg, int local, int G, int Hk) {
    for (int pt = 0; pt < sg.parts; ++pt) {
        const int t0 = first_tile(sg, pt, G);
        const int nt = sg.tiles - t0;
        // a partition's tiles longest first (a later tile sees more keys),
        // every KV head of a tile together, so the CTAs that finish first
        // take the short ones at the end
        if (local < nt * Hk) return make_int3(pt, local % Hk, sg.tiles - 1 - local / Hk);
        local -= nt * Hk;
    }
    return make_int3(-1, -1, -1);
}

// An item as the key producer takes it from the list (every lane holds the
// scalars; block ids are spread over the lanes).
template <bool kRules>
struct Fetched {
    int done, seq, part, kvh, tile, nsteps, nblk, L, Q, q0, nparts;
    int prefix, pb, skip, all_valid;  // (under rules)
    int ids[part_blocks<kRules> / 32];
    uint32_t valid[kPartBlocks / 32];  // (without)
};

template <bool kRules>
__device__ __forceinline__ void fetch_item(const ChunkParams &p, int n_big, int total, int G,
                                           int logG, int lane, Fetched<kRules> &f) {
    if constexpr (kRules) {
        // items in list order until one has blocks (the list ends every search)
        for (;;) {
            int item = 0;
            if (lane == 0) item = atomicAdd(p.work, 1);
            item = __shfl_sync(0xffffffffu, item, 0);
            f.done = item >= total;
            if (f.done) return;
            int lo = 0, hi = n_big - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (__ldcg(p.big_cum + mid) <= item) lo = mid;
                else hi = mid - 1;
            }
            const int seq = __ldcg(p.big_seq + lo);
            SeqGeo sg;
            seq_geo<true>(p, seq, G, false, sg);
            const int local = item - __ldcg(p.big_cum + lo), per = sg.tiles * p.num_kv_heads;
            const int part = local / per, rest = local - part * per;
            const int tile = sg.tiles - 1 - rest / p.num_kv_heads;
            const Span sp = tile_span(sg, tile, G, p.rules.window);
            const int blo = part * kRulePartBlocks;
            if (blo >= sp.nblk) continue;
            f.seq = seq;
            f.part = part;
            f.kvh = rest % p.num_kv_heads;
            f.tile = tile;
            f.nblk = min(kRulePartBlocks, sp.nblk - blo);
            f.nsteps = (f.nblk + kStepBlocks - 1) / kStepBlocks;
            f.L = sg.L;
            f.Q = sg.Q;
            f.q0 = sg.q0;
            f.nparts = (sp.nblk + kRulePartBlocks - 1) / kRulePartBlocks;
            f.prefix = sg.prefix;
            f.pb = sp.pb;
            f.skip = sp.skip;
            load_ids(p, seq, blo, f.nblk, lane, true, f.ids, sp.pb, sp.skip);
            bool all = true;
#pragma unroll
            for (int w = 0; w < kRulePartBlocks / 32; ++w)
                all = all && (f.ids[w] >= 0 || 32 * w + lane >= f.nblk);
            f.all_valid = __all_sync(0xffffffffu, all);
            return;
        }
    } else {
    int item = 0;
    if (lane == 0) item = atomicAdd(p.work, 1);
    item = __shfl_sync(0xffffffffu, item, 0);
    f.done = item >= total;
    if (f.done) return;
    // the listed sequence holding the item (every lane searches alike)
    int lo = 0, hi = n_big - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldcg(p.big_cum + mid) <= item) lo = mid;
        else hi = mid - 1;
    }
    const int seq = __ldcg(p.big_seq + lo);
    SeqGeo sg;
    seq_geo<false>(p, seq, G, false, sg);  // (the plan listed it: valid)
    const int3 d = decode_item(sg, item - __ldcg(p.big_cum + lo), G, p.num_kv_heads);
    const int j_last = (min(sg.rows, (d.z + 1) * kRows) - 1) >> logG;
    const int kv_end = sg.L - sg.Q + j_last + 1;  // keys [0, kv_end) for the tile
    const int k1 = min(kv_end, (d.x + 1) * kPartTokens);
    const int blo = d.x * kPartBlocks;
    f.seq = seq;
    f.part = d.x;
    f.kvh = d.y;
    f.tile = d.z;
    f.nblk = (k1 + kBS - 1) / kBS - blo;  // >= 1
    f.nsteps = (f.nblk + kStepBlocks - 1) / kStepBlocks;
    f.L = sg.L;
    f.Q = sg.Q;
    f.q0 = sg.q0;
    f.nparts = (kv_end + kPartTokens - 1) / kPartTokens;
    load_ids(p, seq, blo, f.nblk, lane, true, f.ids);
#pragma unroll
    for (int w = 0; w < kPartBlocks / 32; ++w) f.valid[w] = __ballot_sync(0xffffffffu, f.ids[w] >= 0);
    }
}

// What a kernel's scores follow: nothing more than the causal order, or rules, of
// which the window and the prefix are numbers and the cap and the bias by distance
// are compiled in or left out (4 x 2048 new tokens of up to 8192, H 32, Hk 8, D 128:
// one kernel with all of it took 740 us with a bias and 903 with both where these
// take 693 and 808, the rest being equal).
constexpr int kPlain = 0, kRuled = 1, kCapped = 2, kBiased = 4;

// Step n of an item, as its place in the item's list of steps: under a bias by
// distance from the newest keys to the oldest, so that the first step sets the rows'
// references (the other way round a steep slope moves them, and O, at every step).
template <int kMode>
__device__ __forceinline__ int place_of(int n, int nsteps) {
    return (kMode & kBiased) != 0 ? nsteps - 1 - n : n;
}

constexpr float kNear = -1.f;

// tanh of a pair of values of at most 1 in size (dec::tanh_near).
__device__ __forceinline__ uint64_t tanh_near2(uint64_t y) {
    const uint64_t t = mul_f32x2(y, y);
    uint64_t r = f32x2(dec::kTanh6, dec::kTanh6);
    r = fma_f32x2(t, r, f32x2(dec::kTanh5, dec::kTanh5));
    r = fma_f32x2(t, r, f32x2(dec::kTanh4, dec::kTanh4));
    r = fma_f32x2(t, r, f32x2(dec::kTanh3, dec::kTanh3));
    r = fma_f32x2(t, r, f32x2(dec::kTanh2, dec::kTanh2));
    r = fma_f32x2(t, r, f32x2(dec::kTanh1, dec::kTanh1));
    r = fma_f32x2(t, r, f32x2(dec::kTanh0, dec::kTanh0));
    return mul_f32x2(y, r);
}

// The n lowest of 16 bits (n may be anything).
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n >= kBS ? 0xFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// The row's scores of this thread's 64 keys under the rules: mx their maximum in log2
// units, and in sx either those scores (masked ones minus infinity; returns 1), or
// them in units of 1/a (returns a > 0), or raw ones far below the cap (returns kNear;
// the weights' loop caps them).  The keys are four blocks of the tile's list from
// place v0 on, nbg of them there, bad ones not in vmask.
// usual (the same for the whole warp): its rows see every key of the step, none of them
// behind their positions under a bias.
template <int kMode>
__device__ __forceinline__ float rule_scores(const ChunkParams &p, uint32_t (&sx)[kGroupKeys],
                                             bool usual, int nbg, uint32_t vmask, int v0, int pb,
                                             int skip, int prefix, int pos, float slope,
                                             float sl2, float &mx) {
    constexpr bool kCap = (kMode & kCapped) != 0, kBias = (kMode & kBiased) != 0;
    const float cap = p.rules.cap_log2, cs = p.rules.cap_scale;
    const float c2 = cs * (2.f * dec::kLog2e);
    const bool exp_form = cap <= dec::kExpCapLog2;
    float mr[8], most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) mr[i] = kNegInf;
    if constexpr (kCap || !kBias) {
#pragma unroll
        for (int e = 0; e < kGroupKeys / 2; ++e)
            mr[e & 7] = fmax3(mr[e & 7], __uint_as_float(sx[2 * e]), __uint_as_float(sx[2 * e + 1]));
        mx = fmax3(fmax3(mr[0], mr[1], mr[2]), fmax3(mr[3], mr[4], mr[5]), fmaxf(mr[6], mr[7]));
    }
    if constexpr (kCap) {
        // (a NaN score does not move the extremes; the polynomial keeps it)
        float lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[i] = mx;
#pragma unroll
        for (int e = 0; e < kGroupKeys / 2; ++e)
            lo[e & 3] = fmin3(lo[e & 3], __uint_as_float(sx[2 * e]), __uint_as_float(sx[2 * e + 1]));
        most = fmaxf(mx, -fminf(fmin3(lo[0], lo[1], lo[2]), lo[3]));
    }
    usual = usual && (kCap ? cs : sl2) > 0.f;
    if constexpr (kCap) {
        if (usual && !__all_sync(0xffffffffu, most <= p.rules.near_most)) {
            usual = false;
            if (!kBias && exp_form) {
                // scores near the cap or past it: tanh in place, that of the largest the
                // largest
                if (__all_sync(0xffffffffu, most * cs <= 1.f)) {
                    const uint64_t cs2 = f32x2(cs, cs);
#pragma unroll
                    for (int e = 0; e < kGroupKeys / 2; ++e) {
                        const float2 v = f32x2_split(tanh_near2(mul_f32x2(
                            f32x2(__uint_as_float(sx[2 * e]), __uint_as_float(sx[2 * e + 1])), cs2)));
                        sx[2 * e] = __float_as_uint(v.x);
                        sx[2 * e + 1] = __float_as_uint(v.y);
                    }
                    mx = cap * dec::tanh_near(mx * cs);
                } else {
#pragma unroll
                    for (int e = 0; e < kGroupKeys; ++e)
                        sx[e] = __float_as_uint(dec::tanh_exp(__uint_as_float(sx[e]) * c2));
                    mx = cap * dec::tanh_exp(mx * c2);
                }
                return cap;
            }
        }
    }
    if (usual) {
        if constexpr (!kCap && !kBias) {
            mx *= sl2;
            return sl2;
        }
        const float n0 = p.rules.near[0], n1 = p.rules.near[1], n2 = p.rules.near[2],
                    n3 = p.rules.near[3];
        if constexpr (kCap && !kBias) {
            // (the capping rises with the score: the largest is that of the largest)
            const float t = mx * mx;
            mx *= fmaf(t, fmaf(t, fmaf(t, n3, n2), n1), n0);
            return kNear;
        }
        // keys at and before the row: the distance falls by one per key
        const uint64_t k0 = f32x2(n0, n0), k1 = f32x2(n1, n1), k2 = f32x2(n2, n2),
                       k3 = f32x2(n3, n3), a2 = f32x2(sl2, sl2), slope2 = f32x2(slope, slope),
                       two = f32x2(2.f, 2.f);
        const float d0 = static_cast<float>(span_block(pb, skip, v0) * kBS - pos);
        uint64_t d2 = f32x2(d0, d0 + 1.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) mr[i] = kNegInf;
#pragma unroll
        for (int e = 0; e < kGroupKeys / 2; ++e) {
            const uint64_t x = f32x2(__uint_as_float(sx[2 * e]), __uint_as_float(sx[2 * e + 1]));
            uint64_t r = a2;
            if constexpr (kCap) {
                const uint64_t t = mul_f32x2(x, x);
                r = fma_f32x2(t, k3, k2);
                r = fma_f32x2(t, r, k1);
                r = fma_f32x2(t, r, k0);
            }
            const float2 v = f32x2_split(fma_f32x2(x, r, mul_f32x2(slope2, d2)));
            d2 = add_f32x2(d2, two);  // (whole numbers below 2^24: exact)
            sx[2 * e] = __float_as_uint(v.x);
            sx[2 * e + 1] = __float_as_uint(v.y);
            mr[e & 7] = fmax3(mr[e & 7], v.x, v.y);
        }
        mx = fmax3(fmax3(mr[0], mr[1], mr[2]), fmax3(mr[3], mr[4], mr[5]), fmaxf(mr[6], mr[7]));
        return 1.f;
    }

    // ---- steps with masks, with prefix keys behind the row under a bias, or with
    // scores near the cap under both
#pragma unroll
    for (int i = 0; i < 8; ++i) mr[i] = kNegInf;
#pragma unroll
    for (int b = 0; b < kGroupKeys / kBS; ++b) {
        // bits of the block's keys that the row sees: up to its position, from its
        // window's start on, or in the prefix
        const int kp = span_block(pb, skip, v0 + b) * kBS, d = pos - kp;
        uint32_t seen = low_bits(d + 1);
        if (d >= p.rules.window) seen &= ~low_bits(d - p.rules.window + 1);
        seen |= low_bits(prefix - kp);
        if (b >= nbg || !((vmask >> b) & 1u)) seen = 0u;
        if (kCap && !exp_form) {
#pragma unroll
            for (int i = 0; i < kBS; ++i) {
                uint32_t &x = sx[b * kBS + i];
                const float y = __uint_as_float(x) * cs;
                x = __float_as_uint(fabsf(y) <= 1.f ? dec::tanh_near(y)
                                                    : dec::tanh_exp(y * (2.f * dec::kLog2e)));
            }
        }
        const float d0 = static_cast<float>(d);
#pragma unroll
        for (int i = 0; i < kBS; ++i) {
            uint32_t &x = sx[b * kBS + i];
            float t = __uint_as_float(x);
            if constexpr (kCap) t = cap * (exp_form ? dec::tanh_exp(t * c2) : t);
            else t *= sl2;
            if constexpr (kBias) t = fmaf(-slope, fabsf(d0 - static_cast<float>(i)), t);
            // (all ones where the bit is set)
            const uint32_t m = static_cast<uint32_t>(static_cast<int32_t>(seen << (31 - i)) >> 31);
            x = (__float_as_uint(t) & m) | (0xFF800000u & ~m);
        }
#pragma unroll
        for (int i = 0; i < kBS / 2; ++i)
            mr[i] = fmax3(mr[i], __uint_as_float(sx[b * kBS + 2 * i]),
                          __uint_as_float(sx[b * kBS + 2 * i + 1]));
    }
    mx = fmax3(fmax3(mr[0], mr[1], mr[2]), fmax3(mr[3], mr[4], mr[5]), fmaxf(mr[6], mr[7]));
    return 1.f;
}

// Value block `vb` ([chunk][token][128 B]): rows from `end` on zeroed, and of the
// others the elements that are not finite.  Bit 0: there were any; bit 1: this lane
// wrote something.  (Every load before the first check: one warp does this, between
// the copies' arrival and the MMAs.)
template <int CH>
__device__ __forceinline__ uint32_t clean_block(uint8_t *vb, int end, int lane) {
    constexpr int kUnits = CH * kBS * 8 / 32;
    uint4 x[kUnits];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) x[j] = *reinterpret_cast<uint4 *>(vb + (32 * j + lane) * 16);
    uint32_t out = 0;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const int token = ((32 * j + lane) >> 3) & (kBS - 1);
        uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        // an exponent of all ones carries into its half's sign bit
        uint32_t bad = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) bad |= (w[k] & 0x7C007C00u) + 0x04000400u;
        if (token >= end || (bad & 0x80008000u) != 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (token >= end || (w[k] & 0x7C00u) == 0x7C00u) w[k] &= 0xFFFF0000u;
                if (token >= end || (w[k] & 0x7C000000u) == 0x7C000000u) w[k] &= 0xFFFFu;
            }
            *reinterpret_cast<uint4 *>(vb + (32 * j + lane) * 16) =
                make_uint4(w[0], w[1], w[2], w[3]);
            out |= token >= end ? 2u : 3u;
        }
    }
    return out;
}

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkParams p) {
    constexpr bool kRules = kMode != kPlain;
    using Gm = Geo<D>;
    constexpr int CH = Gm::kChunks;
    constexpr int DH = D / 2;  // the head dimensions (of O) each softmax thread owns
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((dec::kTileAlign - (smem_u32(smem_raw) & (dec::kTileAlign - 1))) &
                                (dec::kTileAlign - 1));
    const uint32_t sb = smem_u32(smem);
    const Bars br{sb + Gm::kOffBar};
    ItemInfo *info = reinterpret_cast<ItemInfo *>(smem + Gm::kOffInfo);
    // misc: [0] tensor-memory base, [1], [2] (under rules) 1 + the last item of
    // either parity whose values were not all finite where some row is masked
    volatile int *misc = reinterpret_cast<volatile int *>(smem + Gm::kOffMisc);

    const int Hk = p.num_kv_heads, H = p.num_heads;
    const int G = H / Hk, logG = __ffs(G) - 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(br.q_full(s), 1);
            mbar_init(br.q_empty(s), kQEmptyArrivals);
            mbar_init(br.p_full(s), kSoftmaxWarps);
            mbar_init(br.pv_done(s), 1);
        }
        mbar_init(br.qs_full(), 1);
        mbar_init(br.qs_empty(), 1);
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(br.k_full(s), 1);
            mbar_init(br.k_empty(s), 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(br.v_full(s), 1);
            mbar_init(br.v_empty(s), 1);
        }
        mbar_init(br.s_full(), 1);
        mbar_init(br.s_free(), kSoftmaxWarps);
        mbar_init(br.o_free(), kSoftmaxWarps);
        misc[1] = misc[2] = 0;
        fence_mbarrier_init();
    }
    // the work list, the caches and the outputs are written by earlier
    // kernels of the stream
    grid_dependency_wait();
    // the last `split` CTAs leave their SMs to the balanced schedule
    if (static_cast<int>(blockIdx.x) >= static_cast<int>(gridDim.x) - __ldcg(p.split)) return;
    // the kernel launched next (the decode schedule's share of the call)
    // needs nothing from this one: let its CTAs take the SMs this grid leaves
    grid_launch_dependents();
    if (warp == 2) {
        tc::tmem_alloc(sb + Gm::kOffMisc, kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);

    if (warp == 0) {
        // ===================== items, query tiles and keys =====================
        const int n_big = __ldcg(p.n_big);
        const int total = __ldcg(p.big_cum + n_big);
        int gs = 0;  // steps staged
        bool ok = true;
        Fetched<kRules> cur;
        fetch_item<kRules>(p, n_big, total, G, logG, lane, cur);
        for (int it = 0; ok; ++it) {
            const int slot = it & 1;
            if (it >= 2 && !wait_all(br.q_empty(slot), ((it >> 1) - 1) & 1)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                ItemInfo &in = info[slot];
                in.done = cur.done;
                if (!cur.done) {
                    in.seq = cur.seq;
                    in.part = cur.part;
                    in.kvh = cur.kvh;
                    in.tile = cur.tile;
                    in.nsteps = cur.nsteps;
                    in.nblk = cur.nblk;
                    in.L = cur.L;
                    in.Q = cur.Q;
                    in.q0 = cur.q0;
                    in.nparts = cur.nparts;
                    if constexpr (kRules) {
                        in.prefix = cur.prefix;
                        in.pb = cur.pb;
                        in.skip = cur.skip;
                        in.all_valid = cur.all_valid;
                    } else {
#pragma unroll
                        for (int w = 0; w < kPartBlocks / 32; ++w) in.valid[w] = cur.valid[w];
                    }
                }
                mbar_arrive(br.q_full(slot));
            }
            if (cur.done) break;
            // the query tile, into the staging buffer once the previous tile
            // has been copied to tensor memory
            if (it >= 1 && !wait_all(br.qs_empty(), (it - 1) & 1)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(br.qs_full(), Gm::kQ);
            __syncwarp();
            if (lane < CH)
                tensor_g2s_3d(sb + lane * (kRows * 128), &p.tm_q, 128 * lane, cur.kvh * G,
                              cur.q0 + cur.tile * (kRows >> logG), br.qs_full());
            // the next item is taken when this one's last steps are staged,
            // a ring's depth before its softmax ends: the CTAs that finish
            // first take the next items (its lookups overlap those steps)
            Fetched<kRules> nxt;
            nxt.done = 1;
            const int fetch_at = max(cur.nsteps - kClaimLead, 0);
            for (int n = 0; n < cur.nsteps; ++n, ++gs) {
                const int ks = gs % kKStages;
                if (gs >= kKStages && !wait_all(br.k_empty(ks), ((gs / kKStages) - 1) & 1)) {
                    ok = false;
                    break;
                }
                const int sn = place_of<kMode>(n, cur.nsteps);
                const int nb = min(kStepBlocks, cur.nblk - sn * kStepBlocks);
                if (lane == 0) mbar_arrive_expect_tx(br.k_full(ks), nb * CH * kBS * 128);
                __syncwarp();
                // lane l: block l / CH of the step, chunk l % CH (a bad block
                // reads rows before the cache: zeros)
                const int b = min(lane / CH, kStepBlocks - 1), c = lane % CH;
                const int id = id_of(cur.ids, sn * kStepBlocks + b);
                if (lane < nb * CH)
                    tensor_g2s_3d(sb + Gm::kOffK + ks * Gm::kK + c * (kStepKeys * 128) +
                                      b * (kBS * 128),
                                  &p.tm_k, 0, id >= 0 ? id * kBS : -kBS, cur.kvh * CH + c,
                                  br.k_full(ks));
                if (n == fetch_at) fetch_item<kRules>(p, n_big, total, G, logG, lane, nxt);
            }
            cur = nxt;
        }
        if (!ok) {
            if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, blockIdx.x);
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
            const int slot = it & 1;
            if (!wait_all(br.q_full(slot), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const ItemInfo &in = info[slot];
            const int done = in.done, seq = in.seq, part = in.part, kvh = in.kvh;
            const int nsteps = in.nsteps, nblk = in.nblk;
            const int pb = kRules ? in.pb : 0, skip = kRules ? in.skip : 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(br.q_empty(slot));
            if (done) break;
            int ids[part_blocks<kRules> / 32];
            load_ids(p, seq, part * part_blocks<kRules>, nblk, lane, false, ids, pb, skip);
            for (int n = 0; n < nsteps; ++n, ++gs) {
                const int vs = gs % kVStages;
                if (gs >= kVStages && !wait_all(br.v_empty(vs), ((gs / kVStages) - 1) & 1)) {
                    ok = false;
                    break;
                }
                const int sn = place_of<kMode>(n, nsteps);
                const int nb = min(kStepBlocks, nblk - sn * kStepBlocks);
                if (lane == 0) mbar_arrive_expect_tx(br.v_full(vs), nb * Gm::kVBlock);
                __syncwarp();
                const int id = id_of(ids, sn * kStepBlocks + min(lane, kStepBlocks - 1));
                if (lane < nb)
                    tensor_g2s_3d(sb + Gm::kOffV + vs * Gm::kV + lane * Gm::kVBlock, &p.tm_v, 0,
                                  id >= 0 ? id * kBS : -kBS, kvh * CH, br.v_full(vs));
            }
        }
        if (!ok) {
            if (lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, blockIdx.x);
            for (int s = 0; s < kVStages && s < gs; ++s) {
                const int last = gs - 1 - ((gs - 1 - s) % kVStages);
                mbar_wait_bounded(br.v_full(s), (last / kVStages) & 1);
            }
        }
    } else if (warp == 2) {
        // ============================ score MMAs ============================
        // (one issuing thread; inside this kernel each MMA held its issuer
        // back ~110-140 cycles, so the scores and the P V products have one
        // issuing warp each and their chains overlap in the tensor pipe)
        int gs = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int slot = it & 1;
            if (!wait_all(br.q_full(slot), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const ItemInfo &in = info[slot];
            const int done = in.done, nsteps = in.nsteps, nblk = in.nblk;
            __syncwarp();
            if (lane == 0) mbar_arrive(br.q_empty(slot));
            if (done) break;
            // the query tile into tensor memory (the MMAs read A from there);
            // copies and MMAs of this thread run in issue order
            const uint32_t q_t = tmem + kTmemQ + 64 * slot;
            ok = wait_all(br.qs_full(), it & 1);
            if (!ok) break;
            tc::fence_after_sync();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc::cp_128x256b(q_t + 8 * kk,
                                    tc::smem_desc(sb + (kk >> 2) * (kRows * 128) + (kk & 3) * 32,
                                                  16, 1024, tc::kSwizzle128B));
                tc::commit(br.qs_empty());
            }
            __syncwarp();
            for (int n = 0; n < nsteps && ok; ++n) {
                const int g = gs + n, ks = g % kKStages;
                ok = wait_all(br.k_full(ks), (g / kKStages) & 1);
                // the softmax has read the previous step's scores
                if (ok && g >= 1) ok = wait_all(br.s_free(), (g - 1) & 1);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
                    // one MMA per k step over the step's keys (an MMA of
                    // N 64 or less costs the issuing thread about as much as
                    // one of N 128, so fewer and wider ones are faster)
                    const int nb = min(kStepBlocks, nblk - place_of<kMode>(n, nsteps) * kStepBlocks);
                    const uint32_t idesc = tc::idesc_f16_f32(kRows, nb * kBS, false, false);
                    const uint32_t k_s = sb + Gm::kOffK + ks * Gm::kK;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc::mma_ts(tmem + kTmemS, q_t + 8 * kk,
                                   tc::smem_desc(k_s + (kk >> 2) * (kStepKeys * 128) + (kk & 3) * 32,
                                                 16, 1024, tc::kSwizzle128B),
                                   idesc, kk > 0);
                    tc::commit(br.s_full());
                    tc::commit(br.k_empty(ks));
                }
                __syncwarp();
            }
            gs += nsteps;
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, blockIdx.x);
    } else if (warp == kPVWarp) {
        // ============================= P V MMAs =============================
        constexpr uint32_t kIdescPV = tc::idesc_f16_f32(kRows, D, false, true);
        int gs = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int slot = it & 1;
            if (!wait_all(br.q_full(slot), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const ItemInfo &in = info[slot];
            const int done = in.done, nsteps = in.nsteps, nblk = in.nblk, L = in.L;
            const int blo = in.part * part_blocks<kRules>;
            int pb = 0, skip = 0, prefix = 0, a0 = 0, a1 = 0;
            if constexpr (kRules) {
                pb = in.pb;
                skip = in.skip;
                prefix = in.prefix;
                a0 = L - in.Q + in.tile * (kRows >> logG);
                a1 = min(a0 + (kRows >> logG), L) - 1;
            }
            const Clear clear = clear_of(pb, skip, a0, a1, kRules ? p.rules.window : 0, prefix);
            __syncwarp();
            if (lane == 0) mbar_arrive(br.q_empty(slot));
            if (done) break;
            for (int m = 0; m < nsteps && ok; ++m) {
                const int g = gs + m, vs = g % kVStages;
                const int sm = place_of<kMode>(m, nsteps);
                const int nb = min(kStepBlocks, nblk - sm * kStepBlocks);
                ok = wait_all(br.v_full(vs), (g / kVStages) & 1);
                if (!ok) break;
                const uint32_t v_s = sb + Gm::kOffV + vs * Gm::kV;
                if constexpr (kRules) {
                    // blocks that some row does not see whole: value rows past the
                    // sequence's end zeroed, and the others' elements that are not
                    // finite (0 * NaN is not 0), which the rows that see them add
                    // at the end
                    if (!clear.has(blo + sm * kStepBlocks, nb)) {
                        uint32_t found = 0;
                        const int mine = span_block(pb, skip, blo + sm * kStepBlocks + lane) * kBS;
                        uint32_t part_seen = __ballot_sync(
                            0xffffffffu,
                            lane < nb && !seen_whole(mine, a0, a1, p.rules.window, prefix));
                        for (; part_seen != 0; part_seen &= part_seen - 1) {
                            const int b = __ffs(part_seen) - 1;
                            const int kp = __shfl_sync(0xffffffffu, mine, b);
                            uint8_t *vb = smem + Gm::kOffV + vs * Gm::kV + b * Gm::kVBlock;
                            found |= clean_block<CH>(vb, L - kp, lane);
                        }
                        if (found != 0) fence_proxy_async_smem();
                        if (__any_sync(0xffffffffu, found & 1u) && lane == 0) misc[1 + (it & 1)] = it + 1;
                        __syncwarp();
                    }
                } else if (m == nsteps - 1) {
                    // value rows at and past the sequence end hold anything
                    // (their weights are 0, but 0 * NaN is not): zero them
                    const int t0 = L - (blo + m * kStepBlocks + nb - 1) * kBS;
                    if (t0 < kBS) {
                        const int units = (kBS - t0) * 8;  // 16-byte units per chunk
                        uint8_t *vb = smem + Gm::kOffV + vs * Gm::kV + (nb - 1) * Gm::kVBlock;
                        for (int i = lane; i < units * CH; i += 32) {
                            const int c = i / units, r = i % units;
                            *reinterpret_cast<uint4 *>(vb + c * (kBS * 128) +
                                                       (t0 + (r >> 3)) * 128 + (r & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                ok = wait_all(br.p_full(g & 1), (g >> 1) & 1);
                // the previous item's O has been read out
                if (ok && m == 0 && it > 0) ok = wait_all(br.o_free(), (it - 1) & 1);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
                    for (int b = 0; b < nb; ++b)
                        tc::mma_ts(tmem + kTmemO, tmem + kTmemP + 64 * (g & 1) + 8 * b,
                                   tc::smem_desc(v_s + b * Gm::kVBlock, kBS * 128, 1024,
                                                 tc::kSwizzle128B),
                                   kIdescPV, (m > 0 || b > 0) ? 1u : 0u);
                    tc::commit(br.pv_done(g & 1));
                    tc::commit(br.v_empty(vs));
                }
                __syncwarp();
            }
            gs += nsteps;
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, blockIdx.x);
    } else {
        // =============================== softmax ===============================
        // two threads per row: lane 16 h + i of warp 3 + 4 wh + q holds row
        // 32 q + 16 wh + i, keys 64 h .. of each step and head dimensions
        // DH h .. of O; a warp reaches tensor-memory lanes 32 * (warp % 4) ..
        const int wh = (warp - 3) >> 2;
        const int quarter = warp & 3;
        const int h = lane >> 4;
        const int r = quarter * 32 + wh * 16 + (lane & 15);
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32 + wh * 16) << 16);
        const int64_t Tq = p.num_query_tokens;
        const float sl2 = p.scale_log2;
        int gs = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int slot = it & 1;
            if (!wait_all(br.q_full(slot), (it >> 1) & 1)) {
                ok = false;
                break;
            }
            const ItemInfo &in = info[slot];
            const int done = in.done, seq = in.seq, part = in.part, kvh = in.kvh, tile = in.tile;
            const int nsteps = in.nsteps, nblk = in.nblk, L = in.L, Q = in.Q, q0 = in.q0;
            const int nparts = in.nparts;
            const int in_pb = in.pb, in_skip = in.skip, in_prefix = in.prefix;
            uint32_t valid[kPartBlocks / 32];
            // every block of the item in range (the usual case): the steps
            // need no look-up in the array above (under rules: in the table)
            bool all_valid = true;
            if constexpr (kRules) {
                all_valid = in.all_valid != 0;
            } else {
#pragma unroll
                for (int w = 0; w < kPartBlocks / 32; ++w) valid[w] = in.valid[w];
#pragma unroll
                for (int w = 0; w < kPartBlocks / 32; ++w) {
                    const int nbw = min(max(nblk - 32 * w, 0), 32);
                    const uint32_t need = nbw == 32 ? 0xffffffffu : ((1u << nbw) - 1u);
                    all_valid = all_valid && (valid[w] & need) == need;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(br.q_empty(slot));
            if (done) break;
            const int rows = Q * G;
            const int rr = tile * kRows + r;
            const bool row_ok = rr < rows;
            const int j = rr >> logG;
            const int lim = row_ok ? L - Q + j : -1;  // last key position this row sees
            int pb = 0, skip = 0, prefix = 0, pos = 0;
            float slope = 0.f;
            if constexpr (kRules) {
                pb = in_pb;
                skip = in_skip;
                prefix = in_prefix;
                pos = L - Q + min(j, Q - 1);  // (rows past the last: as it, not written)
                if ((kMode & kBiased) != 0)
                    slope = __ldg(p.rules.slopes + kvh * G + (rr & (G - 1))) * dec::kLog2e;
            }
            const int64_t orow = static_cast<int64_t>(q0 + j) * H + kvh * G + (rr & (G - 1));
            const Clear clear =
                clear_of(pb, skip, L - Q + tile * (kRows >> logG),
                         min(L - Q + (tile + 1) * (kRows >> logG), L) - 1,
                         kRules ? p.rules.window : 0, prefix);
            float m_used = kNegInf, l = 0.f;  // l: this thread's keys only

            for (int n = 0; n < nsteps; ++n) {
                const int g = gs + n;
                if (!wait_all(br.s_full(), g & 1)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                uint32_t sx[kGroupKeys];  // this row's scores of this thread's keys (fp32 bits)
#pragma unroll
                for (int c = 0; c < kGroupKeys / 32; ++c)
                    tc::ld32_halves<kGroupKeys>(tl + kTmemS + 32 * c,
                                                *reinterpret_cast<uint32_t(*)[32]>(sx + 32 * c));
                tc::wait_ld();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(br.s_free());
                const int sn = place_of<kMode>(n, nsteps);
                const int nb = min(kStepBlocks, nblk - sn * kStepBlocks);
                const int nbg = min(max(nb - 4 * h, 0), 4);  // this thread's blocks
                const int kbase = part * kPartTokens + n * kStepKeys + kGroupKeys * h;
                const int b0 = n * kStepBlocks + 4 * h;
                uint32_t vmask = 0xFu;
                if constexpr (kRules) {
                    if (!all_valid) {
                        vmask = 0u;
                        for (int b = 0; b < nbg; ++b) {
                            const int64_t id = __ldg(
                                p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq +
                                span_block(pb, skip, part * kRulePartBlocks + sn * kStepBlocks + 4 * h + b));
                            if (id >= 0 && id < p.num_blocks) vmask |= 1u << b;
                        }
                    }
                } else if (!all_valid) {
                    vmask = (valid[b0 >> 5] >> (b0 & 31)) & 0xFu;
                }
                // the maximum of the raw scores first (independent of the
                // masks, so the two overlap); it stands, scaled once, when
                // every key of the warp is visible and the scale is not
                // negative, else the scores are scaled and masked and their
                // maximum taken again
                float mx, a;
                if constexpr (kRules) {
                    const int v = part * kRulePartBlocks + sn * kStepBlocks;
                    bool usual = all_valid && nb == kStepBlocks;
                    if (usual && !((kMode & kBiased) != 0 ? clear.has_past(v, kStepBlocks)
                                                          : clear.has(v, kStepBlocks))) {
                        // (not for the tile, but maybe for this warp's 16 rows)
                        const int v0 = v + 4 * h, kp = span_block(pb, skip, v0) * kBS;
                        const bool past = kp + kGroupKeys - 1 <= pos;
                        usual = __all_sync(
                            0xffffffffu,
                            (v0 >= pb || v0 + 4 <= pb) &&
                                ((past && pos - kp < p.rules.window) ||
                                 (kp + kGroupKeys <= prefix && (past || (kMode & kBiased) == 0))));
                    }
                    a = rule_scores<kMode>(p, sx, usual, nbg, vmask, v + 4 * h, pb, skip, prefix,
                                           pos, slope, sl2, mx);
                } else {
                    const bool fast = __all_sync(0xffffffffu, nbg == 4 && vmask == 0xFu &&
                                                                  kbase + kGroupKeys - 1 <= lim &&
                                                                  sl2 >= 0.f);
                    float mr[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) mr[i] = kNegInf;
#pragma unroll
                    for (int e = 0; e < kGroupKeys / 2; ++e)
                        mr[e & 7] = fmax3(mr[e & 7], __uint_as_float(sx[2 * e]),
                                          __uint_as_float(sx[2 * e + 1]));
                    mx = fmax3(fmax3(mr[0], mr[1], mr[2]), fmax3(mr[3], mr[4], mr[5]),
                                     fmaxf(mr[6], mr[7]));
                    if (!fast) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) mr[i] = kNegInf;
#pragma unroll
                        for (int e = 0; e < kGroupKeys; ++e) {
                            const bool vis = e < nbg * kBS && ((vmask >> (e >> 4)) & 1u) && kbase + e <= lim;
                            const float t = vis ? __uint_as_float(sx[e]) * sl2 : kNegInf;
                            sx[e] = __float_as_uint(t);
                            mr[e & 7] = fmaxf(mr[e & 7], t);
                        }
                        mx = fmax3(fmax3(mr[0], mr[1], mr[2]), fmax3(mr[3], mr[4], mr[5]),
                                   fmaxf(mr[6], mr[7]));
                    } else {
                        mx *= sl2;
                    }
                    a = fast ? sl2 : 1.f;
                }
                // the row's other half: the thread 16 lanes away
                const float mo = __shfl_xor_sync(0xffffffffu, mx, 16);
                const float m_new = fmaxf(m_used, fmaxf(mx, mo));
                const bool raise = m_new > m_used + kRescaleLog2;
                // O holds this item's earlier steps relative to m_used: rescale
                // this thread's columns before the reference moves (the
                // previous P V done first)
                const bool resc = raise && n > 0 && m_used != kNegInf;
                if (__any_sync(0xffffffffu, resc)) {
                    if (!wait_all(br.pv_done((g - 1) & 1), ((g - 1) >> 1) & 1)) {
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
                const float ms = m_used == kNegInf ? 0.f : m_used;
                // weights 2^(s * scale - m) (2^(t - m) for the masked scores),
                // fp16 pairs: column 32 h + i of the buffer holds keys
                // 64 h + 2i, 2i+1; the P V of two steps back must be done
                // with this buffer
                const int pb = g & 1;
                if (g >= 2) {
                    if (!wait_all(br.pv_done(pb), ((g - 2) >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                }
                // key pairs in packed fp32 lanes: one fma and one add per pair
                const float nms = kRules ? kRuleShiftLog2 - ms : -ms;
                const uint64_t a2 = f32x2(a, a), nms2 = f32x2(nms, nms);
                uint64_t l2[4] = {0ull, 0ull, 0ull, 0ull};
                uint32_t x[32];
                if ((kMode & kCapped) != 0 && (kMode & kBiased) == 0 && a == kNear) {
                    // capped scores far below the cap: x (n0 + n1 x^2 + ..) - m
                    const float n0 = p.rules.near[0], n1 = p.rules.near[1],
                                n2 = p.rules.near[2], n3 = p.rules.near[3];
                    const uint64_t k0 = f32x2(n0, n0), k1 = f32x2(n1, n1), k2 = f32x2(n2, n2),
                                   k3 = f32x2(n3, n3);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint64_t y = f32x2(__uint_as_float(sx[2 * e]),
                                                 __uint_as_float(sx[2 * e + 1]));
                        const uint64_t t2 = mul_f32x2(y, y);
                        uint64_t r = fma_f32x2(t2, k3, k2);
                        r = fma_f32x2(t2, r, k1);
                        r = fma_f32x2(t2, r, k0);
                        const float2 t = f32x2_split(fma_f32x2(y, r, nms2));
                        const float p0 = ex2(t.x), p1 = ex2(t.y);
                        l2[e & 3] = add_f32x2(l2[e & 3], f32x2(p0, p1));
                        x[e] = pack_half2(p0, p1);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 t = f32x2_split(fma_f32x2(
                            f32x2(__uint_as_float(sx[2 * e]), __uint_as_float(sx[2 * e + 1])), a2,
                            nms2));
                        const float p0 = ex2(t.x), p1 = ex2(t.y);
                        l2[e & 3] = add_f32x2(l2[e & 3], f32x2(p0, p1));
                        x[e] = pack_half2(p0, p1);
                    }
                }
                tc::st32_halves<32>(tl + kTmemP + 64 * pb, x);
                const float2 la = f32x2_split(add_f32x2(add_f32x2(l2[0], l2[1]), add_f32x2(l2[2], l2[3])));
                l += la.x + la.y;
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(br.p_full(pb));
            }
            if (!ok) break;
            gs += nsteps;

            // ---- the item's output: O / l, or the partial state (m, l, O),
            // this thread's head dimensions
            if (!wait_all(br.pv_done((gs - 1) & 1), ((gs - 1) >> 1) & 1)) {
                ok = false;
                break;
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
            if constexpr (kRules) {
                // values that are not finite, left out of the MMAs where some row is
                // masked: added here by the rows that see them
                if (misc[1 + (it & 1)] == it + 1) {
                    const int a0 = L - Q + tile * (kRows >> logG);
                    const int a1 = min(a0 + (kRows >> logG), L) - 1;
                    for (int b = 0; b < nblk; ++b) {
                        const int blk = span_block(pb, skip, part * kRulePartBlocks + b);
                        const int kp = blk * kBS;
                        if (seen_whole(kp, a0, a1, p.rules.window, prefix)) continue;
                        const int64_t id = __ldg(p.block_tables +
                                                 static_cast<int64_t>(seq) * p.max_blocks_per_seq + blk);
                        if (id < 0 || id >= p.num_blocks) continue;
                        for (int t = 0; t < min(kBS, L - kp); ++t) {
                            if (!dec::rule_sees(pos, kp + t, p.rules.window, prefix)) continue;
                            const __half *v = p.v_cache + ((id * kBS + t) * Hk + kvh) * D + DH * h;
#pragma unroll
                            for (int d = 0; d < DH; ++d) {
                                const float x = __half2float(v[d]);
                                if (!isfinite(x)) o[d] += x;
                            }
                        }
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(br.o_free());
            l += __shfl_xor_sync(0xffffffffu, l, 16);  // the row's sum over both halves' keys
            if (nparts == 1) {
                if (row_ok) {
                    const float inv = l > 0.f ? 1.f / l : 0.f;
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + orow * D + DH * h);
#pragma unroll
                    for (int c = 0; c < DH / 8; ++c)
                        dst[c] = make_uint4(pack_half2(o[8 * c] * inv, o[8 * c + 1] * inv),
                                            pack_half2(o[8 * c + 2] * inv, o[8 * c + 3] * inv),
                                            pack_half2(o[8 * c + 4] * inv, o[8 * c + 5] * inv),
                                            pack_half2(o[8 * c + 6] * inv, o[8 * c + 7] * inv));
                }
                continue;
            }
            // partial state, dimension-major so the rows of a half-warp are
            // consecutive words; each half keeps its own copy of (m, l)
            const int64_t NR = Tq * H;
            const int64_t R = static_cast<int64_t>(kvh) * Tq * G + static_cast<int64_t>(q0) * G + rr;
            const int64_t parts_total = p.num_parts;
            float2 *ml = p.part_ml + h * parts_total * NR;
            if (row_ok) {
                ml[part * NR + R] = make_float2(m_used, l);
                float *dst = p.part_o + (static_cast<int64_t>(part) * D + DH * h) * NR + R;
#pragma unroll
                for (int d = 0; d < DH; ++d) dst[d * NR] = o[d];
            }
            // a ticket per (sequence, kv head, tile, softmax warp): the warp
            // that brings the last partition of its rows merges them.  The
            // warp barrier orders every lane's partial before lane 0's
            // releasing ticket; the last taker acquires the other
            // partitions' partials.
            __syncwarp();
            int last = 0;
            if (lane == 0) {
                int *ticket = p.counters +
                              ((static_cast<int64_t>(seq) * Hk + kvh) * p.num_tiles + tile) *
                                  kSoftmaxWarps +
                              (warp - 3);
                last = atom_add_acq_rel_gpu(ticket, 1) == nparts - 1;
            }
            last = __shfl_sync(0xffffffffu, last, 0);
            __syncwarp();  // memory order: lane 0's acquire before every lane's loads
            if (!last || !row_ok) continue;
            // the tile's last partition: merge every partition's partial row
            float M = kNegInf;
            for (int pp = 0; pp < nparts; ++pp) M = fmaxf(M, __ldcg(ml + pp * NR + R).x);
            float den = 0.f;
#pragma unroll
            for (int d = 0; d < DH; ++d) o[d] = 0.f;
            for (int pp = 0; pp < nparts; ++pp) {
                const float2 v = __ldcg(ml + pp * NR + R);
                const float w = v.x == kNegInf ? 0.f : ex2(v.x - M);
                den = fmaf(v.y, w, den);
                const float *src = p.part_o + (static_cast<int64_t>(pp) * D + DH * h) * NR + R;
#pragma unroll
                for (int d = 0; d < DH; ++d) o[d] = fmaf(__ldcg(src + d * NR), w, o[d]);
            }
            const float inv = den > 0.f ? 1.f / den : 0.f;
            uint4 *dst = reinterpret_cast<uint4 *>(p.out + orow * D + DH * h);
#pragma unroll
            for (int c = 0; c < DH / 8; ++c)
                dst[c] = make_uint4(pack_half2(o[8 * c] * inv, o[8 * c + 1] * inv),
                                    pack_half2(o[8 * c + 2] * inv, o[8 * c + 3] * inv),
                                    pack_half2(o[8 * c + 4] * inv, o[8 * c + 5] * inv),
                                    pack_half2(o[8 * c + 6] * inv, o[8 * c + 7] * inv));
        }
        if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_TIMEOUT, blockIdx.x);
    }

    // every role is done: hand the tensor memory back
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

using ChunkFn = void (*)(const ChunkParams);
// The kernel under score rules (pkv_chunk_rules.cu), or null.
ChunkFn select_chunk_rules(int D, bool capped, bool biased);

}  // namespace chunk
}  // namespace pkv
