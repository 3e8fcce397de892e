/*
 * pagedkv.h -- C ABI of libpagedkv, the GB300 (sm_103a) hot path of paged
 * KV-cache attention: the paged cache write and paged decode attention.
 *
 * Conventions for every entry point:
 *  - Pointers named *_cache, q, out, k, v, slot_mapping, block_tables,
 *    seq_lens and workspace are DEVICE pointers owned by the caller; the
 *    library never allocates, frees or retains them beyond the call.
 *  - Every call is asynchronous on `stream` (NULL = the legacy default
 *    stream) and never synchronises, except pkv_get_device_error.
 *  - Every call first validates its arguments on the host; an invalid call
 *    returns a negative pkv_status and launches nothing.  A failed launch
 *    returns PKV_ERR_CUDA (pkv_last_error_string() has the CUDA message).
 *  - Bad DATA found on the device (a slot or block id out of range, a
 *    sequence longer than its block table) never faults: the offending item
 *    is skipped and the first one is recorded; read it with
 *    pkv_get_device_error.
 *  - fp16 means IEEE binary16 (CUDA __half).
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *pkv_stream_t;

typedef enum pkv_status {
    PKV_OK = 0,
    PKV_ERR_NULL = -1,        /* a required pointer is NULL                        */
    PKV_ERR_INVALID = -2,     /* a size, stride or count is out of its domain      */
    PKV_ERR_UNSUPPORTED = -3, /* valid but not built: head_dim, group size, bs ... */
    PKV_ERR_ALIGNMENT = -4,   /* a pointer or stride breaks a required alignment   */
    PKV_ERR_WORKSPACE = -5,   /* split-KV needs a (larger) workspace               */
    PKV_ERR_CUDA = -6         /* a CUDA runtime call or launch failed              */
} pkv_status;

/* Kinds recorded by the device-side error word (pkv_get_device_error). */
typedef enum pkv_device_error {
    PKV_DEVERR_NONE = 0,
    PKV_DEVERR_SLOT = 1,     /* slot >= num_blocks*block_size; index = token          */
    PKV_DEVERR_BLOCK_ID = 2, /* block id outside [0, num_blocks);
                                index = seq * max_blocks_per_seq + logical block     */
    PKV_DEVERR_SEQ_LEN = 3,  /* seq_len < 0, or more tokens than the block table or
                                max_seq_len allow; index = seq                         */
    PKV_DEVERR_TIMEOUT = 4,  /* a staging wait gave up (about 2 s); index = CTA id   */
    PKV_DEVERR_POSITION = 5, /* position outside [0, max_position); index = token    */
    PKV_DEVERR_PATH = 6,     /* accepted path not ascending or past the block table;
                                index = seq                                           */
    PKV_DEVERR_FREE_LIST = 7, /* the free list's count outside [0, capacity], or more
                                blocks given back than it has room for; index = count */
    PKV_DEVERR_TREE = 8      /* drafted token outside the vocabulary, or a parent that
                                does not come before its node; index = node's row     */
} pkv_device_error;

/*
 * One cache view ("vLLM KV Cache Layout 可视化" -- 核心, KVCacheTensor): a
 * group of same-shaped layers inside one byte allocation.  The byte address
 * of slot `s` of layer `layer` is
 *     offset + layer*layer_stride + (s / block_size)*block_stride
 *            + (s % block_size)*row_width.
 * Layer-outer layouts (LBHNC, LBNHC) have block_stride = page and
 * layer_stride = page*num_blocks; block-outer layouts (BLHNC, BLNHC, BHLNC)
 * have layer_stride = page and block_stride = the bytes of one whole block
 * (page = block_size*row_width) ("layout 是什么").
 */
typedef struct pkv_view {
    int64_t offset;       /* bytes from the cache pointer to layer 0, block 0   */
    int64_t layer_stride; /* bytes between the same block of adjacent layers    */
    int64_t block_stride; /* bytes between adjacent physical blocks of a layer  */
    int64_t row_width;    /* bytes of one token row (one slot)                  */
    int32_t layer;        /* the layer this call writes                         */
} pkv_view;

/*
 * Paged KV-cache write ("vLLM KV Cache Layout 可视化" -- 查一个 token and
 * kernel 那一侧; "deep-dive-into-vllm-05" §2: prefill writes many slots,
 * decode appends one per sequence).
 *
 * For every token t in [0, num_tokens): slot = slot_mapping[t] is split back
 * into block = slot / block_size and position = slot % block_size, and the
 * row_width bytes at k + t*row_width are copied to
 *     k_cache + offset + layer*layer_stride + block*block_stride
 *             + position*row_width
 * (and likewise v -> v_cache, at the same address, when v != NULL).
 *
 *  k, v          device, num_tokens rows of view.row_width bytes, contiguous.
 *                v may be NULL (single-cache write); then v_cache must be NULL.
 *  slot_mapping  device int64 [num_tokens].  A negative slot is padding and is
 *                skipped.  slot >= num_blocks*block_size is skipped and
 *                recorded (PKV_DEVERR_SLOT).  Two tokens with the same slot
 *                in one call: which row lands is unspecified.
 *  k_cache, v_cache  device byte allocations holding the view; the caller
 *                guarantees every slot in [0, num_blocks*block_size) of the
 *                view lies inside them.  Bytes no token addresses are not
 *                touched.
 *  Rows are copied byte for byte (no conversion); 16-byte vectors are used
 *  when every address and stride allows, else 8, 4, 2 or 1 byte.
 *  Returns PKV_OK (num_tokens == 0 launches nothing), PKV_ERR_NULL,
 *  PKV_ERR_INVALID (block_size <= 0, num_blocks <= 0, row_width <= 0 or
 *  > 2^30, block_stride <= 0, offset/layer/layer_stride < 0), PKV_ERR_CUDA.
 */
int pkv_cache_write(const void *k, const void *v, const int64_t *slot_mapping,
                    int64_t num_tokens, void *k_cache, void *v_cache, pkv_view view,
                    int32_t block_size, int64_t num_blocks, pkv_stream_t stream);

/* One (source rows, cache, view) triple of pkv_cache_write_multi. */
typedef struct pkv_write_desc {
    const void *src; /* device: num_tokens rows of view.row_width bytes      */
    void *cache;     /* device byte allocation holding the view              */
    pkv_view view;   /* includes the layer written                           */
} pkv_write_desc;

#define PKV_MAX_WRITE_DESCS 32

/*
 * Several cache writes that share one slot_mapping, in one launch: for every
 * token t and descriptor d, the row at d.src + t*d.view.row_width goes to the
 * address of slot_mapping[t] in d's view, exactly as pkv_cache_write does.
 * This is how every layer and cache of one block table is written at once:
 * the two caches (MLA and indexer) of "vLLM KV Cache Layout 可视化" --
 * 两种 cache 共用一张 block table share one slot number per token (查一个
 * token).
 *  descs       HOST array of num_descs (0..PKV_MAX_WRITE_DESCS) descriptors;
 *              read during the call only.  Rows of different descriptors must
 *              not overlap in memory (which lands is then unspecified).
 *  Other arguments, slot rules and errors as pkv_cache_write.
 */
int pkv_cache_write_multi(const pkv_write_desc *descs, int32_t num_descs,
                          const int64_t *slot_mapping, int64_t num_tokens, int32_t block_size,
                          int64_t num_blocks, pkv_stream_t stream);

/*
 * Copy whole physical blocks within one cache view ("vLLM 技术内幕" §2.2,
 * copy on write: a sequence about to write into a block whose ref_cnt is
 * above one gets a new block holding a copy of the old one).
 * For each pair p in [0, num_pairs), with src = block_mapping[2p] and dst =
 * block_mapping[2p+1], and each layer l in [view.layer, view.layer +
 * num_layers): the page of block_size*row_width bytes at
 *     offset + l*layer_stride + src*block_stride
 * is copied to the same place of block dst.
 *  cache          device byte allocation holding the view.
 *  block_mapping  device int64 [num_pairs][2].  A pair with an id outside
 *                 [0, num_blocks) is skipped and recorded (PKV_DEVERR_BLOCK_ID,
 *                 index = pair); src == dst is a no-op.  A block must not be
 *                 both a source and a destination, nor a destination twice
 *                 (the result is then unspecified).
 *  Returns PKV_OK (nothing to copy launches nothing), PKV_ERR_NULL,
 *  PKV_ERR_INVALID, PKV_ERR_ALIGNMENT, PKV_ERR_CUDA.
 */
int pkv_copy_blocks(void *cache, pkv_view view, int32_t num_layers, int32_t block_size,
                    const int64_t *block_mapping, int64_t num_pairs, int64_t num_blocks,
                    pkv_stream_t stream);

/*
 * Paged decode attention ("deep-dive-into-vllm-05" §2 read loop and §3.2
 * GQA; "vLLM 技术内幕" §2.1: the query is dotted with the keys of each
 * physical block in turn and values are accumulated block by block).
 *
 * For sequence i (length L = seq_lens[i]) and query head h, with G =
 * num_heads/num_kv_heads and kv = h / G (consecutive heads share a KV head):
 *     s_j  = scale * q[i,h,:] . K_j,   K_j = k_cache[bt[i, j/bs], j%bs, kv, :]
 *     out[i,h,:] = sum_j exp(s_j - max s) V_j / sum_j exp(s_j - max s),
 * j in [0, L).  Computed block by block with an online (running max / sum)
 * softmax in fp32; a sequence whose blocks are spread over several CTAs
 * leaves partial (max, sum, weighted values) that are merged with a
 * log-sum-exp rescale inside the same launch.  L == 0 gives zeros.
 *
 * Two schedules (pkv_decode_options.schedule):
 *  - balanced (default): one wave of persistent CTAs, each owning an equal
 *    share of all (KV head group, sequence, block) triples -- a CTA serves up
 *    to 8 KV heads of one group, so more KV heads make more groups; needs a
 *    workspace of pkv_decode_workspace_bytes(...) bytes;
 *  - grid: one CTA per (kv head, sequence, partition of 512 tokens); needs a
 *    workspace only when max_seq_len > 512.
 * With AUTO the balanced schedule runs when the shape and the workspace
 * allow it, else the grid schedule.
 *
 *  out           device fp16 [num_seqs, num_heads, head_dim] (written).
 *  q             device fp16 [num_seqs, num_heads, head_dim].
 *  k_cache, v_cache  device fp16 [num_blocks, block_size, num_kv_heads,
 *                head_dim] ("deep-dive-into-vllm-05" §1.2), 16-byte aligned.
 *  block_tables  device int32 [num_seqs, max_blocks_per_seq]; entries past a
 *                sequence's ceil(L/block_size) blocks are ignored.  An id
 *                outside [0, num_blocks) is skipped and recorded.
 *  seq_lens      device int32 [num_seqs].  A length beyond the block table
 *                (or, on the grid schedule, beyond max_seq_len) is truncated
 *                and recorded (PKV_DEVERR_SEQ_LEN).
 *  max_seq_len   host hint: an upper bound of seq_lens (sizes the grid
 *                schedule's partitions).
 *  workspace     device scratch, 16-byte aligned, of at least
 *                pkv_decode_workspace_bytes(...) bytes (or NULL, see above).
 *                It must be zero-filled before its first use (e.g. by
 *                pkv_decode_workspace_init), and again after a call that records
 *                PKV_DEVERR_TIMEOUT.  Otherwise decode and chunk calls of any kind
 *                and shape, FP8 and under score rules, may follow one another
 *                on it; what anything else writes into it (pkv_tree_attention,
 *                whose scratch is its own) has to be zeroed again.
 *                Calls that share a workspace must not overlap on the GPU.
 *  Ordering: the launch may overlap the previous kernel in the stream when
 *  that kernel signals programmatic launch completion (pkv_cache_write does).
 *  Before that kernel's completion the call reads only q, block_tables and
 *  seq_lens; it reads the caches and writes out/workspace only after.  So a
 *  preceding kernel that signals early must not write q, block_tables or
 *  seq_lens (kernels that never signal are waited for in full, as usual).
 *  Supported: head_dim in {64, 128}; G in {1, 2, 4, 8}; block_size == 16;
 *  num_seqs <= 65535.
 *  Returns PKV_OK (num_seqs == 0 launches nothing), PKV_ERR_NULL,
 *  PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED, PKV_ERR_ALIGNMENT,
 *  PKV_ERR_WORKSPACE, PKV_ERR_CUDA.
 */
int pkv_decode_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                         const int32_t *block_tables, const int32_t *seq_lens, float scale,
                         int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                         int32_t block_size, int32_t num_seqs, int32_t max_blocks_per_seq,
                         int32_t max_seq_len, int64_t num_blocks, void *workspace,
                         size_t workspace_bytes, pkv_stream_t stream);

/* How the per-block arithmetic of pkv_decode_attention_ex runs. */
typedef enum pkv_compute {
    PKV_COMPUTE_AUTO = 0, /* the measured-fastest path (MMA)                     */
    PKV_COMPUTE_SIMT = 1, /* fp32 FMA on CUDA cores, warp-shuffle reductions     */
    PKV_COMPUTE_MMA = 2   /* the GQA group packed into 16x8x16 fp16 MMAs, fp32
                             accumulate                                           */
} pkv_compute;

/* Which CTA schedule pkv_decode_attention_ex uses. */
typedef enum pkv_schedule {
    PKV_SCHEDULE_AUTO = 0,     /* balanced when possible, else grid           */
    PKV_SCHEDULE_GRID = 1,     /* one CTA per (kv head, sequence, partition)  */
    PKV_SCHEDULE_BALANCED = 2  /* persistent CTAs over equal block ranges     */
} pkv_schedule;

typedef struct pkv_decode_options {
    int32_t partition_size; /* grid schedule: tokens per partition, a multiple
                               of block_size in [16, 8192]; 0 = 512          */
    int32_t compute;        /* a pkv_compute value                           */
    int32_t schedule;       /* a pkv_schedule value                          */
} pkv_decode_options;

/* pkv_decode_attention with explicit options (opts may be NULL = defaults).
 * Asking for the balanced schedule when it cannot run returns
 * PKV_ERR_WORKSPACE (workspace too small) or PKV_ERR_UNSUPPORTED. */
int pkv_decode_attention_ex(void *out, const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *block_tables, const int32_t *seq_lens, float scale,
                            int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                            int32_t block_size, int32_t num_seqs, int32_t max_blocks_per_seq,
                            int32_t max_seq_len, int64_t num_blocks, void *workspace,
                            size_t workspace_bytes, const pkv_decode_options *opts,
                            pkv_stream_t stream);

/* Workspace bytes for any schedule of pkv_decode_attention on the current
 * device (its SM count sizes the balanced schedule's partials; without a
 * device, a 256-SM bound is used).  0 for invalid arguments. */
size_t pkv_decode_workspace_bytes(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t max_seq_len);

/* Same, for a grid-schedule partition size (0 = 512). */
size_t pkv_decode_workspace_bytes_ex(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t max_seq_len,
                                     int32_t partition_size);

/*
 * FP8 KV cache ("deep-dive-into-vllm-05" §3.4: quantize on write -- the KV is
 * stored at low precision when written -- and dequantize on read inside the
 * attention kernel; the scales stay with the blocks).  Format: E4M3 (OCP
 * FP8: 4 exponent bits, bias 7, 3 mantissa bits, largest finite 448), one
 * fp32 scale per (token, KV head) row -- the pages' indexer rows carry one
 * FP32 scale per 128 FP8 values ("vLLM KV Cache Layout 可视化").
 *
 * Caches: k_cache, v_cache uint8 [num_blocks, block_size, num_kv_heads,
 * head_dim]; k_scale, v_scale fp32 [num_blocks, block_size, num_kv_heads].
 *
 * pkv_cache_write_fp8 quantizes fp16 rows k, v [num_tokens, num_kv_heads,
 * head_dim] into their slots, in fp32: amax = max |x| of the row,
 * s = amax / 448, code = round-to-nearest-even(x / s) saturated to +-448
 * (s == 0 gives zero codes).  Slot rules and errors as pkv_cache_write;
 * head_dim in {64, 128}; v, v_cache, v_scale all NULL or all set.
 */
int pkv_cache_write_fp8(const void *k, const void *v, const int64_t *slot_mapping,
                        int64_t num_tokens, void *k_cache, void *v_cache, float *k_scale,
                        float *v_scale, int32_t num_kv_heads, int32_t head_dim,
                        int32_t block_size, int64_t num_blocks, pkv_stream_t stream);

/*
 * pkv_decode_attention over FP8 caches (balanced schedule, MMA policy): keys
 * and values are dequantized as value(code) * scale of their row; the result
 * is the attention of pkv_decode_attention on those values.  Needs
 * 16-byte aligned caches and scales and a workspace of
 * pkv_decode_workspace_bytes(...) bytes (zero-filled before its first use, as for
 * pkv_decode_attention).  Other arguments and errors as pkv_decode_attention.
 */
int pkv_decode_attention_fp8(void *out, const void *q, const void *k_cache, const void *v_cache,
                             const float *k_scale, const float *v_scale,
                             const int32_t *block_tables, const int32_t *seq_lens, float scale,
                             int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                             int32_t block_size, int32_t num_seqs, int32_t max_blocks_per_seq,
                             int32_t max_seq_len, int64_t num_blocks, void *workspace,
                             size_t workspace_bytes, pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention of a chunk of new tokens per sequence ("vLLM 技术内幕" §3.2: V1
 * schedules prompt and output tokens alike -- {request: num_tokens} per step
 * -- and cuts a long prompt into chunks that run beside the decodes; §7.4:
 * draft tokens are scheduled with their request and verified together).
 *
 * Sequence i holds seq_lens[i] = L tokens in the cache, this step's new
 * tokens included (write them first, e.g. with pkv_cache_write); its last
 * Q = query_start[i+1] - query_start[i] tokens are the new ones.  New token
 * j (0 <= j < Q) sits at position L - Q + j and attends causally to the
 * cache positions 0 .. L - Q + j.  A chunk of one token is a decode.
 *   out, q          fp16 [num_query_tokens, num_heads, head_dim]; query row r
 *                   is new token r - query_start[i] of the sequence i with
 *                   query_start[i] <= r < query_start[i+1]
 *   k_cache, v_cache, block_tables, seq_lens, scale, num_heads,
 *   num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks:
 *                   as for pkv_decode_attention
 *   query_start     int32 [num_seqs + 1], device: query_start[0] = 0,
 *                   non-decreasing, query_start[num_seqs] <= num_query_tokens
 *                   (rows behind it are left as they are)
 *   max_query_len   host bound on every Q (sizes the launch)
 *   max_seq_len     host bound on every L (sizes the launch and workspace)
 *   workspace       pkv_chunk_workspace_bytes(...) bytes, zeroed once
 *                   (pkv_decode_workspace_init), as for pkv_decode_attention
 *                   and with the same calls
 * Ordering: as for pkv_decode_attention, the launch may overlap a previous
 * kernel that signals programmatic launch completion (pkv_cache_write does);
 * before that kernel's completion the call reads only seq_lens, query_start,
 * q and block_tables, so such a kernel must not write those.
 * Supported: head_dim 64 or 128, block_size 16, group size 1, 2, 4 or 8.
 * Rows of a sequence whose Q exceeds max_query_len or L, whose L exceeds
 * its block table or max_seq_len, whose starts lie outside the rows or fall, or
 * that starts below the sequence before it, are skipped and recorded as
 * PKV_DEVERR_SEQ_LEN; a bad block id is skipped and recorded.  A sequence of
 * length 0 is left out of the call: its rows, however many, are not written, and
 * nothing is recorded.
 * Returns PKV_ERR_WORKSPACE when the workspace is missing or too small. */
int pkv_chunk_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *block_tables, const int32_t *seq_lens,
                        const int32_t *query_start, float scale, int32_t num_heads,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                        int32_t num_seqs, int32_t max_blocks_per_seq, int32_t num_query_tokens,
                        int32_t max_query_len, int32_t max_seq_len, int64_t num_blocks,
                        void *workspace, size_t workspace_bytes, pkv_stream_t stream);

/* Workspace bytes pkv_chunk_attention needs for these bounds (0 for an
 * invalid shape): the short chunks' scratch, the work list, tickets, and,
 * when max_seq_len exceeds one 4096-token KV partition, fp32 partial states
 * of every query row for each partition. */
size_t pkv_chunk_workspace_bytes(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t num_query_tokens,
                                 int32_t max_query_len, int32_t max_seq_len);

/* ------------------------------------------------------------------------
 * Attention whose scores follow rules of the model: capped, biased by distance,
 * limited to a window, with a prefix that every token sees. */

/*
 * With s = scale * q . k of a token at position a and a key at position b:
 *     s' = softcap * tanh(s / softcap)              if softcap > 0
 *     s'' = s' - slopes[h] * |a - b|                for query head h, if slopes
 * and the token sees the key if b <= a and (window > 0) a - b < window, or if
 * b < prefix_lens[i] (of sequence i; later positions than its own included, up
 * to the sequence's length).
 */
typedef struct pkv_score_rules {
    float softcap;              /* >= 0, finite; 0: not capped                    */
    int32_t window;             /* >= 0; 0: every earlier position                */
    const float *slopes;        /* device fp32 [num_heads], or NULL: no bias      */
    const int32_t *prefix_lens; /* device int32 [num_seqs], or NULL: no prefix;
                                   negative counts as 0                           */
} pkv_score_rules;

/*
 * pkv_decode_attention under score rules: each sequence's one query token is at
 * position L - 1.  Blocks that no rule lets the token see are not read.  Scores,
 * maxima, sums and outputs are fp32; softmax weights are rounded to fp16 (each by
 * 2^-11 of itself or, where that is more, by 2^-39 of the row's largest) and
 * the sum they are divided by holds them rounded.  A block whose id is outside
 * [0, num_blocks) is skipped and recorded.  What a position that the token does not
 * see holds, infinities and NaN included, does not reach its output.
 *  rules      HOST pointer, read during the call only; not NULL
 *  workspace  pkv_decode_workspace_bytes(...) bytes, as for
 *             pkv_decode_attention: zero-filled before its first use
 * Runs on the balanced schedule alone: shapes that it does not take (num_seqs
 * whose lengths do not fit shared memory beside two stages, or num_seqs *
 * max_blocks_per_seq above 2^31 - 1) return PKV_ERR_UNSUPPORTED.  Other
 * arguments, shapes, ordering and errors as pkv_decode_attention; slopes and
 * prefix_lens are read before an earlier kernel that signals early has
 * completed, like seq_lens.
 */
int pkv_decode_attention_scored(void *out, const void *q, const void *k_cache,
                                const void *v_cache, const int32_t *block_tables,
                                const int32_t *seq_lens, float scale, int32_t num_heads,
                                int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                int32_t num_seqs, int32_t max_blocks_per_seq,
                                int32_t max_seq_len, int64_t num_blocks, void *workspace,
                                size_t workspace_bytes, const pkv_score_rules *rules,
                                pkv_stream_t stream);

/* The same over FP8 caches (layout of pkv_cache_write_fp8; caches and scales
 * 16-byte aligned); a weight is rounded to fp16 times its value's scale, and summed
 * as it was. */
int pkv_decode_attention_scored_fp8(void *out, const void *q, const void *k_cache,
                                    const void *v_cache, const float *k_scale,
                                    const float *v_scale, const int32_t *block_tables,
                                    const int32_t *seq_lens, float scale, int32_t num_heads,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                    int32_t num_seqs, int32_t max_blocks_per_seq,
                                    int32_t max_seq_len, int64_t num_blocks, void *workspace,
                                    size_t workspace_bytes, const pkv_score_rules *rules,
                                    pkv_stream_t stream);

/* pkv_chunk_attention under score rules: new token j of a sequence is at
 * position L - Q + j.  What a position holds does not reach the rows that do not see
 * it.  Chunks of more than 16 rows (new tokens times group size; 8 where max_query_len
 * allows for such chunks) have their weights rounded by 2^-32 of the row's largest
 * instead of 2^-39, against a sum that holds them as they were; the last bits of their
 * results may depend on the other rows of the call.  Workspace (pkv_chunk_workspace_bytes), other arguments,
 * shapes, ordering and errors as pkv_chunk_attention. */
int pkv_chunk_attention_scored(void *out, const void *q, const void *k_cache,
                               const void *v_cache, const int32_t *block_tables,
                               const int32_t *seq_lens, const int32_t *query_start, float scale,
                               int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, int32_t num_seqs, int32_t max_blocks_per_seq,
                               int32_t num_query_tokens, int32_t max_query_len,
                               int32_t max_seq_len, int64_t num_blocks, void *workspace,
                               size_t workspace_bytes, const pkv_score_rules *rules,
                               pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * A step's bookkeeping on the device. */

/* Largest num_seqs of pkv_resize_sequences. */
#define PKV_MAX_RESIZE_SEQS 8192

/*
 * Block tables, slot maps and the free list of a step, from the lengths that
 * the sequences have (L = seq_lens[i]) and are to have (N = new_lens[i]): a
 * scheduler's allocation, decided on the device, in one launch.  With
 * have = ceil(L / block_size) and want = ceil(N / block_size), over the
 * sequences in order:
 *  - shrinking (N < L: drafts taken back, or with N = 0 a finished request):
 *    blocks have > k >= want go back on the free list, the first of them (in
 *    order of sequence and k) on top.  Their table entries are left as they
 *    were; entries past a sequence's length are never read.
 *  - growing (N > L): new blocks come off the top of the list (blocks given back
 *    in the same call first) into entries have .. want - 1, and each new token
 *    gets a row: token L + j is row query_start[i] + j, with
 *        positions[row] = L + j,  slot_mapping[row] = id * block_size + offset.
 *    A sequence is granted its tokens if the rows up to its last one fit
 *    max_tokens and, where it needs blocks, the blocks needed up to it fit the
 *    list; else it keeps its length and entries, and its rows get slot -1.
 *  - out_lens[i] = N if granted (or N <= L), else L: compare with new_lens.
 *    A refused sequence's rows hold no tokens of it.  The write skips them (slot
 *    -1); the attention behind it is given length 0 for that sequence, e.g.
 *    out_lens[i] == new_lens[i] ? out_lens[i] : 0, which leaves it out, and
 *    pkv_tree_accept a path of -1 (its table entries past L are not its own).
 *    With its kept length L the rows would be taken for its last Q tokens, or,
 *    if there are not so many, be recorded as an error.
 *  - query_start[i] = new tokens asked for by the sequences before i, at most
 *    max_tokens; rows from query_start[num_seqs] on get slot -1 and position 0,
 *    so the writes of a step captured for max_tokens rows skip them.
 * Taking a step back (the same call with the two lengths exchanged) leaves the
 * free list as it was.
 *  block_tables    device int32 [num_seqs, max_blocks_per_seq], updated.  A
 *                  sequence must not give back blocks that another one uses: a
 *                  finished request with a shared prefix shrinks to the prefix,
 *                  not to 0.
 *  seq_lens, new_lens, out_lens  device int32 [num_seqs]; out_lens may be
 *                  seq_lens.  A length outside [0, max_blocks_per_seq *
 *                  block_size] leaves its sequence as it was, recorded
 *                  (PKV_DEVERR_SEQ_LEN).
 *  free_blocks     device int32 [free_capacity]: the list, its top at
 *                  free_count[0] - 1; entries from out_free_count[0] on hold
 *                  nothing of use afterwards.
 *  free_count, out_free_count  device int32 [1]; may be the same.  A count
 *                  outside [0, free_capacity] is clamped, blocks past the
 *                  capacity are dropped, both recorded (PKV_DEVERR_FREE_LIST).
 *  query_start     device int32 [num_seqs + 1], written.
 *  slot_mapping, positions  device int64 [max_tokens], written; positions may be
 *                  NULL.  A block id outside [0, num_blocks), from the table or
 *                  the list, gives slot -1, recorded (PKV_DEVERR_BLOCK_ID).
 * Other buffers must not overlap.  Any block_size; num_seqs at most
 * PKV_MAX_RESIZE_SEQS; max_tokens and free_capacity below 2^30.  Ordering as
 * pkv_norm_rope_write.  Returns PKV_OK (num_seqs == 0 launches nothing),
 * PKV_ERR_NULL, PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED, PKV_ERR_ALIGNMENT (4
 * bytes; 8 for int64), PKV_ERR_CUDA.
 */
int pkv_resize_sequences(int32_t *block_tables, const int32_t *seq_lens,
                         const int32_t *new_lens, int32_t *out_lens, int32_t *free_blocks,
                         const int32_t *free_count, int32_t *out_free_count,
                         int32_t *query_start, int64_t *slot_mapping, int64_t *positions,
                         int32_t num_seqs, int32_t max_blocks_per_seq, int32_t max_tokens,
                         int32_t free_capacity, int32_t block_size, int64_t num_blocks,
                         pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * One speculative step around the cache: the new tokens' queries, keys and
 * values leave the QKV product (pkv_norm_rope_write), a tree of drafted tokens
 * is verified against the cache (pkv_tree_attention), and the accepted path's
 * rows move to the positions they will keep (pkv_tree_accept).  The first one
 * serves decode and prefill steps alike. */

/* Norm and rotation of pkv_norm_rope_write. */
typedef struct pkv_norm_rope {
    const void *q_weight;  /* device fp16 [head_dim], or NULL: queries not normed */
    const void *k_weight;  /* device fp16 [head_dim], or NULL: keys not normed    */
    float eps;             /* added to the mean square, >= 0                      */
    const float *cos_sin;  /* device fp32 [max_position][rot_dim]: rot_dim/2 cosines,
                              then rot_dim/2 sines; NULL iff rot_dim == 0         */
    int64_t max_position;  /* rows of cos_sin                                     */
    int32_t rot_dim;       /* leading dims of each head rotated: a multiple of 16
                              in [0, head_dim]                                    */
    int32_t interleaved;   /* pairs: 0 (d, d + rot_dim/2); 1 (2i, 2i + 1)         */
} pkv_norm_rope;

/*
 * Per-head norm of queries and keys, rotation by position, and the cache
 * write, in one pass over the QKV product's rows.  For every token t with
 * slot_mapping[t] >= 0, every head row x of q and k:
 *     n_d = x_d * w_d / sqrt(mean_d x_d^2 + eps)       (n = x without a weight)
 *     a' = a cos_i - b sin_i,  b' = b cos_i + a sin_i   for pair i = (a, b) of n
 *                                                       at positions[t]
 * computed in fp32 and rounded once.  Rotated queries go to q_out; rotated
 * keys, and values as they are, to the slot's rows of k_cache and v_cache.
 *  q, k, v       device fp16, token t's rows at t*stride elements, its heads
 *                packed [num_heads | num_kv_heads][head_dim]: the three may be
 *                slices of one packed row.  Strides are multiples of 8.
 *  q_out         device fp16 [num_tokens, num_heads, head_dim]; may be q itself
 *                when q is packed (q_stride == num_heads*head_dim), and must not
 *                overlap the inputs otherwise.
 *  positions     device int64 [num_tokens].  A position outside [0,
 *                max_position) skips its token, recorded (PKV_DEVERR_POSITION);
 *                not read when rot_dim == 0 (then it may be NULL).
 *  slot_mapping  as pkv_cache_write: a negative slot is padding -- the token is
 *                skipped, its q_out row left as it was -- and a slot past the
 *                cache skips the token, recorded (PKV_DEVERR_SLOT).
 *  k_cache, v_cache  fp16 [num_blocks, block_size, num_kv_heads, head_dim].
 * Ordering: the call may start before an earlier kernel of the stream that
 * signals programmatic launch completion has finished, and waits for it before
 * it reads or writes anything; it never signals early itself, so a decode or
 * tree attention after it sees its queries.
 * Supported: head_dim 64 or 128.  Returns PKV_OK (num_tokens == 0 launches
 * nothing), PKV_ERR_NULL, PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED,
 * PKV_ERR_ALIGNMENT (16-byte pointers; 8 for int64), PKV_ERR_CUDA.
 */
int pkv_norm_rope_write(void *q_out, const void *q, const void *k, const void *v,
                        int64_t q_stride, int64_t k_stride, int64_t v_stride,
                        const pkv_norm_rope *norm_rope, const int64_t *positions,
                        const int64_t *slot_mapping, int64_t num_tokens, void *k_cache,
                        void *v_cache, int32_t num_heads, int32_t num_kv_heads,
                        int32_t head_dim, int32_t block_size, int64_t num_blocks,
                        pkv_stream_t stream);

/* The same into FP8 caches (layout and quantisation of pkv_cache_write_fp8):
 * keys are quantised from their fp32 values, not rounded to fp16 first. */
int pkv_norm_rope_write_fp8(void *q_out, const void *q, const void *k, const void *v,
                            int64_t q_stride, int64_t k_stride, int64_t v_stride,
                            const pkv_norm_rope *norm_rope, const int64_t *positions,
                            const int64_t *slot_mapping, int64_t num_tokens, void *k_cache,
                            void *v_cache, float *k_scale, float *v_scale, int32_t num_heads,
                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                            int64_t num_blocks, pkv_stream_t stream);

/*
 * Rows of an FP8 cache read back in 16 bits (the inverse of
 * pkv_cache_write_fp8): row t of k (and v) is value(code) * scale of slot
 * slot_mapping[t], rounded to fp16 once.  A negative slot leaves its rows as
 * they were; a slot past the cache too, recorded (PKV_DEVERR_SLOT).  Several
 * tokens may read one slot.
 *  k, v   device fp16 [num_tokens, num_kv_heads, head_dim], written; v, v_cache
 *         and v_scale all NULL or all set.
 * head_dim 64 or 128.  Ordering as pkv_norm_rope_write.  Returns PKV_OK,
 * PKV_ERR_NULL, PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED, PKV_ERR_ALIGNMENT (rows
 * 32, caches 16, slots 8, scales 4 bytes), PKV_ERR_CUDA.
 */
int pkv_cache_read_fp8(void *k, void *v, const int64_t *slot_mapping, int64_t num_tokens,
                       const void *k_cache, const void *v_cache, const float *k_scale,
                       const float *v_scale, int32_t num_kv_heads, int32_t head_dim,
                       int32_t block_size, int64_t num_blocks, pkv_stream_t stream);

/* Largest max_query_len of pkv_tree_attention. */
#define PKV_MAX_TREE_NODES 256

/*
 * Attention of a tree of drafted tokens per sequence over the paged cache.
 * As pkv_chunk_attention, sequence i's last Q = query_start[i+1] -
 * query_start[i] tokens are the drafted ones, already in the cache; but which
 * of them a drafted token sees is given by a mask instead of their order:
 * query row r sees every position 0 .. L-Q-1 and drafted token j (position
 * L-Q+j) exactly when bit j % 64 of tree_mask[r*mask_words + j/64] is set
 * (bits at and past Q are ignored; a token sees itself only if its own bit is
 * set).  A row that sees nothing gives zeros, and so does a row whose visible
 * scores are all minus infinity, where its visible values are finite.  What a
 * masked position holds -- infinities and NaN included -- does not reach the
 * rows that do not see it.  Scores, maxima, sums and outputs are fp32; the
 * softmax weights (FP8: times their value's scale) are rounded to fp16 for the
 * product with the values, each by 2^-11 of itself or, where that is more, by
 * 2^-36 of the row's largest one; the sum they are divided by holds them as
 * they were.
 *   tree_mask      device uint64 [num_query_tokens][mask_words], with
 *                  max_query_len <= 64*mask_words
 *   max_query_len  host bound on every Q, at most PKV_MAX_TREE_NODES
 *   out            may be q itself (each row is read before it is written),
 *                  and must not overlap the inputs otherwise
 *   workspace      pkv_tree_workspace_bytes(...) bytes of device scratch,
 *                  16-byte aligned; its contents need no preparation and carry nothing from call to
 *                  call.  Calls that share a workspace must not overlap.
 *   other arguments, supported shapes, skipped sequences and blocks as
 *   pkv_chunk_attention; max_seq_len or the block table's length stays
 *   below 2^31 - 128 tokens.
 * Ordering: the call may start before an earlier kernel that signals
 * programmatic launch completion has finished, and waits for it before it
 * reads or writes anything.  It signals early itself: a following kernel that
 * is launched with programmatic serialization must not read out before its
 * own wait (so out is not to be the q of a pkv_decode_attention or a
 * pkv_chunk_attention that follows, which read q before theirs).
 * Returns PKV_OK (no sequence or no query token launches nothing),
 * PKV_ERR_NULL, PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED, PKV_ERR_ALIGNMENT (16
 * bytes; 8 for the mask, 4 for int32), PKV_ERR_WORKSPACE, PKV_ERR_CUDA.
 */
int pkv_tree_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                       const int32_t *block_tables, const int32_t *seq_lens,
                       const int32_t *query_start, const uint64_t *tree_mask,
                       int32_t mask_words, float scale, int32_t num_heads,
                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                       int32_t num_seqs, int32_t max_blocks_per_seq, int32_t num_query_tokens,
                       int32_t max_query_len, int32_t max_seq_len, int64_t num_blocks,
                       void *workspace, size_t workspace_bytes, pkv_stream_t stream);

/* The same over FP8 caches, read as value(code) * scale of their rows (layout
 * of pkv_cache_write_fp8; caches and scales 16-byte aligned).  A key whose
 * scale is not finite makes the rows that see it NaN. */
int pkv_tree_attention_fp8(void *out, const void *q, const void *k_cache, const void *v_cache,
                           const float *k_scale, const float *v_scale,
                           const int32_t *block_tables, const int32_t *seq_lens,
                           const int32_t *query_start, const uint64_t *tree_mask,
                           int32_t mask_words, float scale, int32_t num_heads,
                           int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                           int32_t num_seqs, int32_t max_blocks_per_seq,
                           int32_t num_query_tokens, int32_t max_query_len,
                           int32_t max_seq_len, int64_t num_blocks, void *workspace,
                           size_t workspace_bytes, pkv_stream_t stream);

/* Workspace bytes of either tree attention for these bounds on the current
 * device (0 for an invalid shape). */
size_t pkv_tree_workspace_bytes(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t num_query_tokens,
                                int32_t max_query_len, int32_t max_seq_len);

/* One cache of pkv_tree_accept. */
typedef struct pkv_cache_desc {
    void *cache;   /* device byte allocation holding the view              */
    pkv_view view; /* view.layer is the first layer moved                  */
} pkv_cache_desc;

#define PKV_MAX_ACCEPT_DEPTH 256

/*
 * Keep an accepted path of every sequence's drafted tree: with ctx =
 * ctx_lens[i] tokens before the tree, the row of drafted token path[i][d]
 * (position ctx + path[i][d]) moves to position ctx + d, for d = 0, 1, ...
 * until the first negative entry, in every cache of descs and each of
 * num_layers layers from view.layer on -- as if every row were read before any
 * is written.  Rows are moved byte for byte.
 *  descs         HOST array of num_descs (0..PKV_MAX_WRITE_DESCS); read during
 *                the call only.  Quantised caches pass their scales as caches
 *                of their own (row_width 4*num_kv_heads).
 *                Rows of different descriptors must not overlap in memory; one
 *                that names a layer of another again is refused
 *                (PKV_ERR_INVALID).
 *  path          device int32 [num_seqs, max_depth]; its entries before the
 *                first negative one must ascend strictly, and their positions
 *                lie inside the block table: else the sequence is left as it
 *                was and recorded (PKV_DEVERR_PATH).  A sequence that names a
 *                block outside [0, num_blocks) for one of these positions is
 *                left as it was and recorded (PKV_DEVERR_BLOCK_ID).
 *  ctx_lens      device int32 [num_seqs].
 *  block_tables  device int32 [num_seqs, max_blocks_per_seq].  Sequences must
 *                not share the blocks that rows move in.
 * Any block_size.  max_depth at most PKV_MAX_ACCEPT_DEPTH.  Ordering as
 * pkv_norm_rope_write.  Returns PKV_OK (nothing to move launches nothing),
 * PKV_ERR_NULL, PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED, PKV_ERR_ALIGNMENT,
 * PKV_ERR_CUDA.
 */
int pkv_tree_accept(const pkv_cache_desc *descs, int32_t num_descs, int32_t num_layers,
                    const int32_t *path, int32_t max_depth, const int32_t *ctx_lens,
                    const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                    int32_t block_size, int64_t num_blocks, pkv_stream_t stream);

/*
 * Verification of drafted trees (a chain is a tree) against the target's
 * probabilities, from given random numbers: the accepted path of each sequence,
 * as pkv_tree_accept takes it, and its next token, distributed as the target
 * alone would have drawn them.
 *
 * Sequence i's nodes are rows query_start[i] .. query_start[i+1]-1; node 0 is the
 * last token known before the step, always accepted.  parents[row] is a node's
 * parent as an index within its sequence, smaller than its own (node 0's is not
 * read; another node with a negative parent is padding).  p = target_probs[row]
 * is the target's distribution after a node, q = draft_probs[row] the one that
 * its children were drawn from, independently.  From node 0 on, the children x
 * of the current node, in order, with W = 1 and C = 0 at first:
 *     R(t) = max(p(t) - C q(t), 0)
 *     accept x if accept_uniforms[x] * W * q(token x) < R(token x): x is the
 *     current node next;  else C += W, W = sum_t R(t) with the new C.
 * Without draft_probs a child is a fixed guess (q is 1 at its token): accept if
 * accept_uniforms[x] * W < R(token x), else W -= R(token x) and R(token x) = 0.
 * Where no child is accepted, the next token is the lowest index at which the
 * running sum of R passes sample_uniforms[i] times its whole sum; an empty R
 * (W = 0) stands back for the last one that was not.  A path of max_depth nodes
 * ends there, with the next token drawn from p.
 * An element of R is rounded to 32 bits (two fused multiply-adds), four
 * neighbours are added in 32 bits, and from there sums, masses and tests are
 * carried in pairs of fp32 (47 bits): a sum of R is off by 2^-22 of itself at most,
 * and by what such errors of the earlier masses, as C, take from its elements.  A
 * result can differ from the definition's only where a comparison is closer to its
 * border than that.
 *  path           device int32 [num_seqs, max_depth], written: the accepted
 *                 nodes, then -1
 *  path_lens      device int32 [num_seqs], written: accepted nodes, node 0
 *                 counted; 0 (and next token -1) for a sequence without nodes
 *  next_tokens    device int32 [num_seqs], written; -1 where p is zero everywhere
 *  draft_tokens, parents  device int32 [num_nodes].  A token outside [0,
 *                 vocab_size) or a parent that is not smaller leaves its node out
 *                 as if it were padding, recorded (PKV_DEVERR_TREE).
 *  target_probs   device fp32 [num_nodes] rows of vocab_size at target_stride
 *                 elements (>= vocab_size); rows sum to 1 up to rounding.
 *                 Negative values and NaN count as 0; infinities are not handled.
 *                 Where a node's two rows do not start at the same place within 16
 *                 bytes (strides of four elements and aligned bases see to it) they
 *                 are read element by element, with the same results.
 *  draft_probs    the same at draft_stride, or NULL; leaves' rows are not read
 *  accept_uniforms, sample_uniforms  device fp32 [num_nodes], [num_seqs], in
 *                 [0, 1) (others are taken as the nearest of these)
 *  A sequence with more than PKV_MAX_TREE_NODES nodes, or whose rows are not
 *  inside [0, num_nodes), is recorded (PKV_DEVERR_SEQ_LEN) and treated as
 *  without nodes.
 * max_depth at most PKV_MAX_ACCEPT_DEPTH.  Ordering as pkv_norm_rope_write.
 * Returns PKV_OK (num_seqs == 0 launches nothing), PKV_ERR_NULL,
 * PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED, PKV_ERR_ALIGNMENT (4 bytes),
 * PKV_ERR_CUDA.
 */
int pkv_tree_verify(int32_t *path, int32_t max_depth, int32_t *path_lens, int32_t *next_tokens,
                    const int32_t *draft_tokens, const int32_t *parents,
                    const int32_t *query_start, const float *target_probs,
                    int64_t target_stride, const float *draft_probs, int64_t draft_stride,
                    const float *accept_uniforms, const float *sample_uniforms,
                    int32_t num_seqs, int32_t num_nodes, int32_t vocab_size,
                    pkv_stream_t stream);

/* Bytes of the built-in scratch of pkv_decode_attention_noalloc (16 MiB). */
#define PKV_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

/*
 * pkv_decode_attention without a workspace, for callers that cannot allocate
 * device memory: a plugin inside a host runtime that owns the device-memory
 * budget and passes in only inputs and outputs, or a latency-critical loop
 * that must never call cudaMalloc (which can synchronise the device).  The
 * pages have no counterpart; it computes exactly what pkv_decode_attention
 * computes, with the same arguments minus the workspace.
 *
 * Its scratch is a device array of PKV_NOALLOC_SCRATCH_BYTES built into the
 * library: every device that loads the library holds it until the process
 * exits.  The call allocates nothing (no cudaMalloc, cudaFree or allocating
 * library routine).
 *  - The first call on a device, with that device current, looks up the
 *    array's device address (cudaGetSymbolAddress); make that first call
 *    before any stream capture.
 *  - Every call clears the array's tickets on `stream` before the kernel
 *    (a call that gave up may have left some taken).
 *  - All calls share the one array: calls that overlap on the GPU (other
 *    streams, other threads) race and corrupt each other's results.
 *  - A shape whose scratch need exceeds PKV_NOALLOC_SCRATCH_BYTES is refused
 *    with PKV_ERR_WORKSPACE before anything runs (pkv_last_error_string()
 *    gives the bytes needed); use pkv_decode_attention for it.
 */
int pkv_decode_attention_noalloc(void *out, const void *q, const void *k_cache,
                                 const void *v_cache, const int32_t *block_tables,
                                 const int32_t *seq_lens, float scale, int32_t num_heads,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                 int32_t num_seqs, int32_t max_blocks_per_seq,
                                 int32_t max_seq_len, int64_t num_blocks, pkv_stream_t stream);

/* Zero-fill a workspace on `stream` (cudaMemsetAsync). */
int pkv_decode_workspace_init(void *workspace, size_t workspace_bytes, pkv_stream_t stream);

/*
 * Synchronise `stream`, then read and clear the device-side error record of
 * the current device: *kind receives a pkv_device_error value (0 = none) and
 * *index its index (-1 when none).  Either pointer may be NULL.
 */
int pkv_get_device_error(int32_t *kind, int64_t *index, pkv_stream_t stream);

/* Static text for a pkv_status value. */
const char *pkv_status_string(int status);

/* Text of the last CUDA error a call of this thread returned PKV_ERR_CUDA for. */
const char *pkv_last_error_string(void);

/* ABI version of this header (major*10000 + minor*100 + patch). */
int pkv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_H */
