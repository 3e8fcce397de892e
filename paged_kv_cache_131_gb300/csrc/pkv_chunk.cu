// pkv_chunk.cu -- attention of a chunk of new tokens per sequence: scratch layout,
// routing between the tile kernel (pkv_chunk.cuh) and the balanced decode schedule,
// and the C ABI.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pkv_chunk.cuh"

namespace pkv {
namespace chunk {
namespace {

ChunkFn select(int D, bool scored, const dec::RuleParams &rules) {
    if (scored) return select_chunk_rules(D, rules.cap_log2 > 0.f, rules.slopes != nullptr);
    if (D == 128) return chunk_attention_kernel<128, kPlain>;
    if (D == 64) return chunk_attention_kernel<64, kPlain>;
    return nullptr;
}

struct Sizes {
    int64_t tiles, parts, counters_bytes, ml_bytes, o_bytes, list_bytes;
    int col_tiles;          // balanced schedule's column n-tiles (0: not used)
    dec::BalancedShape bal;  // its shape (workspace first in the scratch)
    int64_t bal_bytes;
};

// scored: under score rules, which need no more of anything than without (so the
// workspace sized without them does), but other shared memory on the balanced schedule,
// whose grid and scratch may be smaller.  The tile kernel's part then lies elsewhere than
// without rules; nothing in it has to hold over from one call to the next.
Sizes sizes(int64_t S, int64_t H, int64_t Hk, int64_t D, int64_t Tq, int64_t max_q,
            int64_t max_len, bool scored) {
    Sizes z{};
    const int64_t G = H / Hk;
    z.tiles = std::max<int64_t>(1, (max_q * G + kRows - 1) / kRows);
    z.parts = std::max<int64_t>(1, (max_len + kPartTokens - 1) / kPartTokens);
    z.counters_bytes = dec::align256(S * Hk * z.tiles * kSoftmaxWarps * 4);  // per softmax warp
    z.list_bytes = dec::align256((2 * S + 4) * 4);  // big_seq, big_cum, n_big, work, split
    z.ml_bytes = z.parts > 1 ? dec::align256(2 * z.parts * Tq * H * 8) : 0;  // per group
    z.o_bytes = z.parts > 1 ? z.parts * Tq * H * D * 4 : 0;
    // the balanced schedule takes the chunks of up to 8 query rows, or of up
    // to 16 when no chunk needs the tile kernel (one column tile is the
    // cheaper policy, so it is used whenever the tile kernel runs anyway)
    z.col_tiles = (max_q * G <= 8 || max_q * G > 16) ? 1 : 2;
    z.bal = dec::balanced_shape(static_cast<int>(S), static_cast<int>(Hk), static_cast<int>(G),
                                static_cast<int>(D), sm_count(), false, 8 * z.col_tiles, scored);
    if (!z.bal.ok) z.col_tiles = 0;
    // (the room for tickets at the start is kept by every call)
    z.bal_bytes = z.bal.ok ? dec::align256(z.bal.workspace) : dec::kTicketBytes;
    return z;
}

}  // namespace
}  // namespace chunk
}  // namespace pkv

extern "C" size_t pkv_chunk_workspace_bytes(int32_t num_seqs, int32_t num_heads,
                                            int32_t num_kv_heads, int32_t head_dim,
                                            int32_t num_query_tokens, int32_t max_query_len,
                                            int32_t max_seq_len) {
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        num_heads % num_kv_heads != 0 || num_query_tokens < 0 || max_query_len <= 0 ||
        max_seq_len <= 0)
        return 0;
    const auto z = pkv::chunk::sizes(num_seqs, num_heads, num_kv_heads, head_dim,
                                     num_query_tokens, max_query_len, max_seq_len, false);
    return static_cast<size_t>(z.bal_bytes + z.list_bytes + z.counters_bytes + z.ml_bytes +
                               z.o_bytes);
}

namespace pkv {
namespace chunk {
namespace {

// Either entry point (rules null: without score rules, scored false).
int chunk_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *block_tables, const int32_t *seq_lens,
                    const int32_t *query_start, float scale, int32_t num_heads,
                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_seqs,
                    int32_t max_blocks_per_seq, int32_t num_query_tokens, int32_t max_query_len,
                    int32_t max_seq_len, int64_t num_blocks, void *workspace,
                    size_t workspace_bytes, bool scored, const pkv_score_rules *rules,
                    pkv_stream_t stream) {
    if (num_seqs < 0 || num_query_tokens < 0) return PKV_ERR_INVALID;
    if (num_seqs == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start)
        return PKV_ERR_NULL;
    if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 || head_dim <= 0 ||
        block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || max_query_len <= 0 ||
        max_seq_len <= 0 || !std::isfinite(scale))
        return PKV_ERR_INVALID;
    const int G = num_heads / num_kv_heads;
    if (!(G == 1 || G == 2 || G == 4 || G == 8)) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (block_size != kBS) return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start, 4) ||
        (workspace != nullptr && !aligned(workspace, 16)))
        return PKV_ERR_ALIGNMENT;
    dec::RuleParams rp{};
    if (scored) {
        const int st = dec::make_rules(rules, scale, &rp);
        if (st != PKV_OK) return st;
    }
    const auto z = sizes(num_seqs, num_heads, num_kv_heads, head_dim, num_query_tokens,
                         max_query_len, max_seq_len, scored);
    // work items (and their prefix sums) are 32-bit: at most
    // (sum of tiles <= Tq*G/64 + S) * partitions * Hk of them
    const int64_t tiles_sum = (static_cast<int64_t>(num_query_tokens) * G + kRows - 1) / kRows +
                              num_seqs;
    if (tiles_sum * z.parts * num_kv_heads > INT32_MAX || z.tiles > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    const int64_t need = z.bal_bytes + z.list_bytes + z.counters_bytes + z.ml_bytes + z.o_bytes;
    if (workspace == nullptr || static_cast<int64_t>(workspace_bytes) < need)
        return PKV_ERR_WORKSPACE;
    ChunkFn fn = select(head_dim, scored, rp);
    if (fn == nullptr) return PKV_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    const int row_bytes = num_kv_heads * head_dim * 2;

    // ---- chunks of up to 8 * col_tiles query rows: the balanced schedule,
    // launched after the tile kernel (below) when there are long chunks too
    int min_rows = 1;
    bool use_bal = false;
    dec::BalancedParams b{};
    // (the balanced schedule indexes the flattened block list in 32 bits)
    if (z.col_tiles > 0 && static_cast<int64_t>(num_seqs) * max_blocks_per_seq <= INT32_MAX) {
        b.out = static_cast<__half *>(out);
        b.q = static_cast<const __half *>(q);
        b.k_cache = static_cast<const __half *>(k_cache);
        b.v_cache = static_cast<const __half *>(v_cache);
        b.block_tables = block_tables;
        b.seq_lens = seq_lens;
        b.scale_log2 = scale_log2;
        b.num_seqs = num_seqs;
        b.num_heads = num_heads;
        b.num_kv_heads = num_kv_heads;
        b.max_blocks_per_seq = max_blocks_per_seq;
        b.num_blocks = num_blocks;
        b.query_start = query_start;
        b.max_cols = 8 * z.col_tiles;
        b.num_query_tokens = num_query_tokens;
        b.rules = rp;
        const int st = dec::setup_balanced(b, z.bal, b.max_cols, ws, k_cache, v_cache);
        if (st != PKV_OK) return st;
        b.err = device_error_record();
        if (b.err == nullptr) return PKV_ERR_CUDA;
        min_rows = b.max_cols + 1;
        if (static_cast<int64_t>(max_query_len) * G < min_rows)  // no long chunks
            return dec::launch_balanced(b, z.bal, head_dim, G, false, false, s, z.col_tiles, scored);
        use_bal = true;
    }

    // ---- the larger chunks: query tiles of 128 rows
    ChunkParams p{};
    p.out = static_cast<__half *>(out);
    p.q = static_cast<const __half *>(q);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.query_start = query_start;
    p.scale_log2 = scale_log2;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_query_len = max_query_len;
    p.max_seq_len = max_seq_len;
    p.num_tiles = static_cast<int>(z.tiles);
    p.num_parts = static_cast<int>(z.parts);
    p.num_query_tokens = num_query_tokens;
    p.min_rows = min_rows;
    p.num_blocks = num_blocks;
    p.rules = rp;
    p.v_cache = static_cast<const __half *>(v_cache);
    uint8_t *cws = ws + z.bal_bytes;
    p.num_seqs = num_seqs;
    p.big_seq = reinterpret_cast<int *>(cws);
    p.big_cum = p.big_seq + num_seqs;
    p.n_big = p.big_cum + num_seqs + 1;
    p.work = p.n_big + 1;
    p.split = p.work + 1;
    p.head_dim = head_dim;
    p.max_cols = use_bal ? b.max_cols : 0;
    cws += z.list_bytes;
    p.counters = reinterpret_cast<int *>(cws);
    p.part_ml = reinterpret_cast<float2 *>(cws + z.counters_bytes);
    p.part_o = reinterpret_cast<float *>(cws + z.counters_bytes + z.ml_bytes);
    {
        // keys: one 128-byte chunk per copy; values: the head's chunks (a
        // head's head_dim * 2 bytes are whole 128-byte chunks); query rows
        const int chunks = head_dim * 2 / 128;
        int st = dec::make_kv_tensor_map(&p.tm_k, k_cache, num_blocks, row_bytes, 1);
        if (st == PKV_OK)
            st = dec::make_kv_tensor_map(&p.tm_v, v_cache, num_blocks, row_bytes, chunks);
        if (st == PKV_OK)
            st = dec::make_q_tensor_map(&p.tm_q, q, num_query_tokens, num_heads, head_dim, G);
        if (st != PKV_OK) return st;
    }
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;

    // the work list (one CTA), then persistent CTAs that pull from it
    const int smem = smem_bytes(head_dim);
    int per_sm = 0;
    {
        const int st = prepare_kernel(reinterpret_cast<const void *>(fn), kThreads, smem, &per_sm);
        if (st != PKV_OK) return st;
    }
    p.num_ctas = std::max(1, sm_count() * std::max(1, per_sm));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t pcfg = {};
    pcfg.gridDim = dim3(1);
    pcfg.blockDim = dim3(1024);
    pcfg.stream = s;
    pcfg.attrs = attr;
    pcfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(
        &pcfg, scored ? chunk_plan_kernel<true> : chunk_plan_kernel<false>, p, G);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failure(e, "chunk plan launch");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fn, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failure(e, "chunk attention launch");
    if (!use_bal) return PKV_OK;
    // the short chunks: their CTAs start as the tile kernel's leave (it
    // allows dependents at its start); the caches were written before the
    // plan kernel completed (it waits for the previous kernel), and the two
    // kernels write disjoint rows and scratch, so this grid waits for the
    // tile kernel only before it exits
    b.defer_wait = 1;
    b.active_ctas = p.split;  // its ranges over the SMs the plan left it
    return dec::launch_balanced(b, z.bal, head_dim, G, false, false, s, z.col_tiles, scored);
}

}  // namespace
}  // namespace chunk
}  // namespace pkv

extern "C" int pkv_chunk_attention(void *out, const void *q, const void *k_cache,
                                   const void *v_cache, const int32_t *block_tables,
                                   const int32_t *seq_lens, const int32_t *query_start,
                                   float scale, int32_t num_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t block_size, int32_t num_seqs,
                                   int32_t max_blocks_per_seq, int32_t num_query_tokens,
                                   int32_t max_query_len, int32_t max_seq_len,
                                   int64_t num_blocks, void *workspace, size_t workspace_bytes,
                                   pkv_stream_t stream) {
    return pkv::chunk::chunk_attention(out, q, k_cache, v_cache, block_tables, seq_lens,
                                       query_start, scale, num_heads, num_kv_heads, head_dim,
                                       block_size, num_seqs, max_blocks_per_seq, num_query_tokens,
                                       max_query_len, max_seq_len, num_blocks, workspace,
                                       workspace_bytes, false, nullptr, stream);
}

extern "C" int pkv_chunk_attention_scored(
    void *out, const void *q, const void *k_cache, const void *v_cache,
    const int32_t *block_tables, const int32_t *seq_lens, const int32_t *query_start, float scale,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int32_t num_seqs, int32_t max_blocks_per_seq, int32_t num_query_tokens, int32_t max_query_len,
    int32_t max_seq_len, int64_t num_blocks, void *workspace, size_t workspace_bytes,
    const pkv_score_rules *rules, pkv_stream_t stream) {
    return pkv::chunk::chunk_attention(out, q, k_cache, v_cache, block_tables, seq_lens,
                                       query_start, scale, num_heads, num_kv_heads, head_dim,
                                       block_size, num_seqs, max_blocks_per_seq, num_query_tokens,
                                       max_query_len, max_seq_len, num_blocks, workspace,
                                       workspace_bytes, true, rules, stream);
}
