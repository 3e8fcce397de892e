// pkv_decode_balanced.cu -- the balanced schedule of paged decode attention
// (pkv_decode_balanced.cuh): shapes, scratch layout and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "pkv_decode_balanced.cuh"

namespace pkv {
namespace dec {
namespace {

template <int D, int G>
BalancedFn pick(bool simt, bool fp8, int col_tiles) {
    if (col_tiles == 1) return decode_balanced_kernel<D, G, MmaColsPolicy<D, G, 1>, false>;
    if (col_tiles == 2) return decode_balanced_kernel<D, G, MmaColsPolicy<D, G, 2>, false>;
    if (fp8) return decode_balanced_kernel<D, G, MmaFp8Policy<D, G>, true>;
    if (simt) return decode_balanced_kernel<D, G, SimtPolicy<D, G>, false>;
    return decode_balanced_kernel<D, G, MmaPolicy<D, G>, false>;
}

BalancedFn select(int D, int G, bool simt, bool fp8, int col_tiles) {
#define PKV_CASE(d, g) \
    if (D == d && G == g) return pick<d, g>(simt, fp8, col_tiles);
    PKV_CASE(128, 1) PKV_CASE(128, 2) PKV_CASE(128, 4) PKV_CASE(128, 8)
    PKV_CASE(64, 1) PKV_CASE(64, 2) PKV_CASE(64, 4) PKV_CASE(64, 8)
#undef PKV_CASE
    return nullptr;
}

}  // namespace

BalancedShape balanced_shape(int num_seqs, int num_kv_heads, int G, int D, int num_sms,
                             bool fp8, int rows, bool scored) {
    if (rows <= 0) rows = G;
    BalancedShape r{};
    r.ok = num_kv_heads >= 1 && num_seqs >= 1 && (D == 64 || D == 128) &&
           (G == 1 || G == 2 || G == 4 || G == 8);
    if (!r.ok) return r;
    // heads per CTA: the largest divisor of num_kv_heads up to 8 whose staged
    // row has the swizzle chunk of the whole row (the tensor maps span whole
    // rows; a group's box starts at a chunk boundary)
    const int elem = fp8 ? 1 : 2;
    const int chunk = chunk_bytes_for_row(num_kv_heads * D * elem);
    int hc = 0;
    for (int h = std::min(num_kv_heads, kMaxBalancedKvHeads); h >= 1 && hc == 0; --h)
        if (num_kv_heads % h == 0 && chunk_bytes_for_row(h * D * elem) == chunk) hc = h;
    // (virtual sequence numbers group * S + seq stay 32-bit)
    if (hc == 0 || static_cast<int64_t>(num_seqs) * (num_kv_heads / hc) > INT32_MAX) {
        r.ok = false;
        return r;
    }
    const int row_bytes = hc * D * elem;
    const int stage_bytes = stage_bytes_for(row_bytes, num_kv_heads, fp8);
    int stages = fp8 ? kMaxStagesFp8 : kMaxStages;
    while (stages >= 2 && smem_bytes(stages, stage_bytes, num_seqs, hc, G, scored) > kSmemPerSM) --stages;
    if (stages < 2) {
        r.ok = false;
        return r;
    }
    r.stages = stages;
    r.heads = hc;
    r.groups = num_kv_heads / hc;
    r.row_bytes = row_bytes;
    r.smem = smem_bytes(stages, stage_bytes, num_seqs, hc, G, scored);
    const int threads = (hc + 1) * 32;
    r.ctas_per_sm = std::max(1, std::min({(228 * 1024) / (r.smem + 1024), 2048 / threads, 32}));
    r.grid = std::max(1, num_sms) * r.ctas_per_sm;
    const int64_t slots = 2 * static_cast<int64_t>(r.grid) * hc * rows;
    r.workspace = kTicketBytes + align256(slots * 8) + slots * D * 4;
    if (static_cast<int64_t>(r.grid) * hc * 4 > kTicketBytes) r.ok = false;
    return r;
}

int setup_balanced(BalancedParams &p, const BalancedShape &shape, int rows, void *workspace,
                   const void *k_cache, const void *v_cache) {
    p.num_stages = shape.stages;
    p.row_bytes = shape.row_bytes;
    p.heads_per_cta = shape.heads;
    p.groups = shape.groups;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const int64_t slots = 2 * static_cast<int64_t>(shape.grid) * shape.heads * rows;
    p.counters = reinterpret_cast<int *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + kTicketBytes);
    p.part_o = reinterpret_cast<float *>(ws + kTicketBytes + align256(slots * 8));
    // maps over whole rows (all heads); a box covers one head group
    const int full_row = shape.row_bytes * shape.groups;
    const int box = shape.row_bytes / chunk_bytes_for_row(shape.row_bytes);
    int st = make_kv_tensor_map(&p.tm_k, k_cache, p.num_blocks, full_row, box);
    if (st == PKV_OK) st = make_kv_tensor_map(&p.tm_v, v_cache, p.num_blocks, full_row, box);
    return st;
}

int launch_balanced(const BalancedParams &p, const BalancedShape &shape, int D, int G, bool simt,
                    bool fp8, cudaStream_t stream, int col_tiles, bool scored) {
    BalancedFn fn = scored ? select_balanced_rules(D, G, fp8, col_tiles)
                           : select(D, G, simt, fp8, col_tiles);
    if (fn == nullptr) return PKV_ERR_UNSUPPORTED;
    const int threads = (p.heads_per_cta + 1) * 32;
    int per_sm = 0;
    const int st = prepare_kernel(reinterpret_cast<const void *>(fn), threads, shape.smem, &per_sm);
    if (st != PKV_OK) return st;
    per_sm = std::max(1, std::min(per_sm, shape.ctas_per_sm));
    const int grid = std::min(shape.grid, per_sm * std::max(1, shape.grid / shape.ctas_per_sm));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shape.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failure(e, "decode balanced launch");
}

}  // namespace dec
}  // namespace pkv
