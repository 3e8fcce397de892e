// pkv_tree_accept.cu -- keeping an accepted path of a drafted tree: the cache
// row of drafted token path[d] moves to place d behind the context, in every
// cache and layer.
//
// A path ascends strictly, so path[d] >= d and no later row is read from a
// place that an earlier one was written to: a thread that owns one column
// (a vector of every row) may move its rows in order with no barrier, a batch
// of loads ahead of its stores.  One CTA per (sequence, cache and layer,
// stretch of columns); it checks the path and turns it into byte offsets in
// shared memory first, and writes nothing when an entry is bad.
// Bound: HBM (two row widths per moved row), or latency for small calls: path,
// block id, row and store are dependent.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 8;  // rows of a column in flight
constexpr int kMaxDepth = PKV_MAX_ACCEPT_DEPTH;

struct AcceptDesc {
    uint8_t *base;  // cache + view.offset + view.layer * view.layer_stride
    int64_t layer_stride;
    int64_t block_stride;
    int64_t row_width;
    int32_t vec;  // bytes per vector: 16, 8, 4, 2 or 1
};

struct AcceptParams {
    AcceptDesc d[PKV_MAX_WRITE_DESCS];
    const int32_t *path;
    const int32_t *ctx_lens;
    const int32_t *block_tables;
    int32_t max_depth;
    int32_t max_blocks;
    int32_t block_size;
    int32_t num_layers;
    int64_t num_blocks;
    ErrorRecord *err;
};

template <typename VT>
__device__ __forceinline__ void move_column(uint8_t *col, const int64_t *src, const int64_t *dst,
                                            int n) {
    for (int i = 0; i < n; i += kBatch) {
        VT r[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i + u < n) r[u] = *reinterpret_cast<const VT *>(col + src[i + u]);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i + u < n) *reinterpret_cast<VT *>(col + dst[i + u]) = r[u];
    }
}

__global__ void __launch_bounds__(kThreads)
    tree_accept_kernel(const __grid_constant__ AcceptParams p) {
    __shared__ int64_t src[kMaxDepth], dst[kMaxDepth];
    __shared__ int depth, bad;
    const int seq = blockIdx.x;
    const AcceptDesc &d = p.d[blockIdx.y / p.num_layers];
    const int layer = blockIdx.y % p.num_layers;
    if (threadIdx.x == 0) {
        depth = p.max_depth;
        bad = 0;
    }
    grid_dependency_wait();  // paths and rows may come from the kernel just before
    __syncthreads();
    const int32_t *path = p.path + static_cast<int64_t>(seq) * p.max_depth;
    for (int i = threadIdx.x; i < p.max_depth; i += kThreads)
        if (path[i] < 0) atomicMin(&depth, i);
    __syncthreads();
    const int n = depth;
    const int64_t ctx = p.ctx_lens[seq];
    const int32_t *table = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks;
    // place `pos` of the sequence in this cache, or -1 (kind: the error)
    auto place = [&](int64_t pos, int &kind) -> int64_t {
        const int64_t b = pos / p.block_size;
        if (pos < 0 || b >= p.max_blocks) {
            kind = PKV_DEVERR_PATH;
            return -1;
        }
        const int64_t id = table[b];
        if (id < 0 || id >= p.num_blocks) {
            if (kind == 0) kind = PKV_DEVERR_BLOCK_ID;
            return -1;
        }
        return id * d.block_stride + (pos - b * p.block_size) * d.row_width;
    };
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int node = path[i];
        int kind = i > 0 && path[i - 1] >= node ? PKV_DEVERR_PATH : ctx < 0 ? PKV_DEVERR_PATH : 0;
        if (kind == 0) {
            src[i] = place(ctx + node, kind);
            dst[i] = place(ctx + i, kind);
        }
        if (kind != 0) atomicMax(&bad, kind);
    }
    __syncthreads();
    if (bad != 0) {
        if (threadIdx.x == 0) record_error(p.err, bad, seq);
        return;
    }
    const int64_t at = (static_cast<int64_t>(blockIdx.z) * kThreads + threadIdx.x) * d.vec;
    if (at >= d.row_width) return;
    uint8_t *col = d.base + layer * d.layer_stride + at;
    switch (d.vec) {
        case 16: move_column<uint4>(col, src, dst, n); break;
        case 8: move_column<uint2>(col, src, dst, n); break;
        case 4: move_column<unsigned int>(col, src, dst, n); break;
        case 2: move_column<unsigned short>(col, src, dst, n); break;
        default: move_column<unsigned char>(col, src, dst, n); break;
    }
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_tree_accept(const pkv_cache_desc *descs, int32_t num_descs,
                               int32_t num_layers, const int32_t *path, int32_t max_depth,
                               const int32_t *ctx_lens, const int32_t *block_tables,
                               int32_t num_seqs, int32_t max_blocks_per_seq, int32_t block_size,
                               int64_t num_blocks, pkv_stream_t stream) {
    using namespace pkv;
    if (num_descs < 0 || num_layers < 0 || num_seqs < 0 || max_depth < 0) return PKV_ERR_INVALID;
    if (num_descs > PKV_MAX_WRITE_DESCS || max_depth > kMaxDepth) return PKV_ERR_UNSUPPORTED;
    if (num_descs == 0 || num_layers == 0 || num_seqs == 0 || max_depth == 0) return PKV_OK;
    if (!descs || !path || !ctx_lens || !block_tables) return PKV_ERR_NULL;
    if (block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0) return PKV_ERR_INVALID;
    if (static_cast<int64_t>(num_descs) * num_layers > 65535) return PKV_ERR_UNSUPPORTED;
    if (!aligned(path, 4) || !aligned(ctx_lens, 4) || !aligned(block_tables, 4))
        return PKV_ERR_ALIGNMENT;
    AcceptParams p{};
    int64_t columns = 0;  // vectors of the widest row
    for (int i = 0; i < num_descs; ++i) {
        const pkv_view &v = descs[i].view;
        if (!descs[i].cache) return PKV_ERR_NULL;
        if (v.row_width <= 0 || v.row_width > (int64_t(1) << 30) || v.block_stride <= 0 ||
            v.offset < 0 || v.layer < 0 || v.layer_stride < 0 ||
            (num_layers > 1 && v.layer_stride <= 0))
            return PKV_ERR_INVALID;
        AcceptDesc &d = p.d[i];
        d.base = static_cast<uint8_t *>(descs[i].cache) + v.offset + v.layer * v.layer_stride;
        d.layer_stride = v.layer_stride;
        // rows that two descriptors share would move twice
        const int64_t span = std::max<int64_t>(v.layer_stride, 1) * num_layers;
        for (int j = 0; j < i; ++j) {
            const int64_t apart = d.base - p.d[j].base;
            if (apart == 0 || (p.d[j].layer_stride == v.layer_stride && v.layer_stride > 0 &&
                               apart < span && -apart < span && apart % v.layer_stride == 0))
                return PKV_ERR_INVALID;
        }
        d.block_stride = v.block_stride;
        d.row_width = v.row_width;
        const uintptr_t bits = reinterpret_cast<uintptr_t>(d.base) |
                               (num_layers > 1 ? static_cast<uintptr_t>(v.layer_stride) : 0) |
                               static_cast<uintptr_t>(v.block_stride) |
                               static_cast<uintptr_t>(v.row_width);
        d.vec = (bits & 15) == 0 ? 16 : (bits & 7) == 0 ? 8 : (bits & 3) == 0 ? 4
              : (bits & 1) == 0 ? 2 : 1;
        columns = std::max(columns, v.row_width / d.vec);
    }
    const int64_t stretches = (columns + kThreads - 1) / kThreads;
    if (stretches > 65535) return PKV_ERR_UNSUPPORTED;
    p.path = path;
    p.ctx_lens = ctx_lens;
    p.block_tables = block_tables;
    p.max_depth = max_depth;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    p.num_layers = num_layers;
    p.num_blocks = num_blocks;
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_seqs),
                       static_cast<unsigned>(num_descs * num_layers),
                       static_cast<unsigned>(stretches));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, tree_accept_kernel, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failure(e, "tree_accept_kernel launch");
}
