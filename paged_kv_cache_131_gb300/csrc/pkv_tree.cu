// pkv_tree.cu -- attention of a tree of drafted tokens per sequence over the
// paged cache (fp16 or FP8).
//
// Sequence i holds L tokens, the last Q of them drafted; query row r sees the
// context 0 .. L-Q-1 and the drafted tokens whose mask bit is set:
//     out = sum_vis 2^(s_j - m) V_j / sum_vis 2^(s_j - m),
//     s_j = scale log2(e) q . K_j,  m the running maximum.
// One warp per (query row, head): lanes hold the head dims, one key at a time.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

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

template <int D, bool FP8>
__device__ __forceinline__ void load_dims(const void *cache, const float *scale, int64_t row,
                                          int lane, float (&x)[D / 32]) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const int64_t at = row * D + lane + 32 * i;
        if constexpr (FP8) {
            __nv_fp8_e4m3 c;
            c.__x = static_cast<const uint8_t *>(cache)[at];
            x[i] = static_cast<float>(c) * scale[row];
        } else {
            x[i] = __half2float(static_cast<const __half *>(cache)[at]);
        }
    }
}

template <int D, bool FP8>
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
        load_dims<D, FP8>(p.k_cache, p.k_scale, row, lane, x);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale_log2;
        if (s == -INFINITY) continue;
        const float mn = fmaxf(m, s), a = exp2f(m - mn), pr = exp2f(s - mn);
        load_dims<D, FP8>(p.v_cache, p.v_scale, row, lane, x);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = fmaf(o[i], a, pr * x[i]);
        l = fmaf(l, a, pr);
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        p.out[w * D + lane + 32 * i] = __float2half_rn(l == 0.f ? 0.f : o[i] / l);
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
    using Fn = void (*)(const TreeParams);
    const Fn fn = head_dim == 128 ? (fp8 ? tree_rows_kernel<128, true> : tree_rows_kernel<128, false>)
                                  : (fp8 ? tree_rows_kernel<64, true> : tree_rows_kernel<64, false>);
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
    return 256;
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
