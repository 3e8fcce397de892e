// pkv_resize.cu -- block tables, slot maps and the free list of a step, from the
// lengths that the sequences have and are to have (pkv_resize_sequences).
//
// Everything follows from three exclusive prefix sums over the sequences in
// order: blocks given back, blocks needed and new tokens.  With them every output
// element is computed by itself: row t finds its sequence in the token sums, its
// block is the table's or, past the blocks that the sequence has, new block
// number r of the step, which is block number r given back while those last and
// then the list's entry r - R from the top (R: blocks given back).  So no element
// waits for another: released entries are read from the table, where only other
// sequences' entries are written, and the list is read below its old top and
// written above it.
//
// One cluster of up to 8 CTAs.  Each sums over all sequences by itself (a thread
// takes a stretch of them) and keeps the sums in shared memory, which costs less
// than an exchange; the rows are spread over the cluster.  The one barrier of the
// cluster stands between the reads of the lengths and count and the writes of
// those that may be the same buffers.
// Bound: latency -- lengths, then table or list entry, then store are dependent: 3.5 us
// for 64 sequences that get a token each.  1000 sequences with 16384 new rows and some
// 20000 blocks given back: 9.0 us, half of it the searches (ten steps in shared memory
// for each row and block).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxCluster = 8;  // the portable cluster size
constexpr int kBatch = 2;       // rows or blocks that a thread has in flight
constexpr int kMaxSeqs = PKV_MAX_RESIZE_SEQS;
constexpr unsigned kFull = 1u << 30;  // the sums saturate here (two fit 32 bits)

struct ResizeParams {
    int32_t *tables;
    const int32_t *seq_lens;
    const int32_t *new_lens;
    int32_t *out_lens;
    int32_t *free_blocks;
    const int32_t *free_count;
    int32_t *out_free_count;
    int32_t *query_start;
    int64_t *slots;
    int64_t *positions;
    int num_seqs;
    int max_blocks;
    int max_tokens;
    int capacity;
    int block_size;
    int shift;  // block_size is 2^shift; -1: not a power of two
    int64_t num_blocks;
    ErrorRecord *err;
};

__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kFull); }

struct Sums {
    unsigned back, need, rows;
};

__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) {
    return {sat_add(a.back, b.back), sat_add(a.need, b.need), sat_add(a.rows, b.rows)};
}

__device__ __forceinline__ Sums shfl_up(const Sums &a, int d) {
    return {__shfl_up_sync(0xffffffffu, a.back, d), __shfl_up_sync(0xffffffffu, a.need, d),
            __shfl_up_sync(0xffffffffu, a.rows, d)};
}

// Largest i in [0, n) with sums[i] <= x (non-decreasing, sums[0] = 0 <= x).
__device__ __forceinline__ int find(const unsigned *sums, int n, unsigned x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads)
    resize_kernel(const __grid_constant__ ResizeParams p) {
    extern __shared__ unsigned smem[];
    const int S = p.num_seqs, bs = p.block_size;
    unsigned *back = smem;           // [S + 1] blocks given back before a sequence
    unsigned *rows = back + S + 1;   // [S + 1] rows before it
    unsigned *need = rows + S + 1;   // [S] new blocks before it, kFull: not granted
    int *old = reinterpret_cast<int *>(need + S);  // [S] its length
    int *size = old + S;                           // [S] the length it is to have (L: bad data)
    __shared__ Sums warp_sums[kThreads / 32 + 1];
    __shared__ unsigned taken;  // new blocks granted
    auto cluster = cooperative_groups::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cta = static_cast<int>(cluster.block_rank());
    const int ctas = static_cast<int>(cluster.num_blocks());
    const int64_t room = static_cast<int64_t>(p.max_blocks) * bs;

    grid_dependency_wait();  // lengths, tables and the list come from earlier kernels
    int count = __ldcg(p.free_count);
    if (threadIdx.x == 0) taken = 0;

    // ---- the sums
    const int per = (S + kThreads - 1) / kThreads;
    const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
    // (block sizes are powers of two where it counts: three 64-bit divisions a row were
    // half of this kernel's instructions)
    auto quotient = [&](unsigned x) {
        return p.shift >= 0 ? x >> p.shift : x / static_cast<unsigned>(bs);
    };
    auto blocks = [&](int len) {
        return static_cast<int>(quotient(static_cast<unsigned>(len) + static_cast<unsigned>(bs) - 1u));
    };
    auto delta = [&](int L, int N) -> Sums {
        const int more = blocks(N) - blocks(L);
        return {static_cast<unsigned>(max(-more, 0)), static_cast<unsigned>(max(more, 0)),
                static_cast<unsigned>(max(N - L, 0))};
    };
    Sums mine{0, 0, 0};
    for (int s = s0; s < s1; ++s) {
        const int L = __ldcg(p.seq_lens + s);
        int N = __ldcg(p.new_lens + s);
        if (L < 0 || L > room || N < 0 || N > room) {
            if (cta == 0) record_error(p.err, PKV_DEVERR_SEQ_LEN, s);
            N = L;
        }
        old[s] = L;
        size[s] = N;
        if (N != L) {
            const Sums d = delta(L, N);
            mine = mine + Sums{min(d.back, kFull), min(d.need, kFull), min(d.rows, kFull)};
        }
    }
    Sums incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums y = shfl_up(incl, o);
        if (lane >= o) incl = incl + y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        Sums v = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums y = shfl_up(v, o);
            if (lane >= o) v = v + y;
        }
        __syncwarp();
        warp_sums[lane + 1] = v;
        if (lane == 0) warp_sums[0] = Sums{0, 0, 0};
    }
    __syncthreads();
    const Sums total = warp_sums[kThreads / 32];
    if (count < 0 || count > p.capacity) {
        if (cta == 0 && threadIdx.x == 0) record_error(p.err, PKV_DEVERR_FREE_LIST, count);
        count = count < 0 ? 0 : p.capacity;
    }
    // blocks given back that the list has room for
    const unsigned R = min(total.back, static_cast<unsigned>(p.capacity - count));
    if (R < total.back && cta == 0 && threadIdx.x == 0)
        record_error(p.err, PKV_DEVERR_FREE_LIST, count);
    const unsigned top = static_cast<unsigned>(count) + R;  // the list before blocks are taken
    const unsigned T = static_cast<unsigned>(p.max_tokens);
    {
        // before this thread's stretch: its warp's offset and the lanes below
        Sums run = shfl_up(incl, 1);
        if (lane == 0) run = Sums{0, 0, 0};
        run = warp_sums[warp] + run;
        unsigned most = 0;
        for (int s = s0; s < s1; ++s) {
            back[s] = run.back;
            rows[s] = min(run.rows, T);
            const int L = old[s], N = size[s];
            unsigned at = kFull;
            if (N != L) {
                const Sums d = delta(L, N);
                const unsigned before = run.need;
                run = run + Sums{min(d.back, kFull), min(d.need, kFull), min(d.rows, kFull)};
                if (N > L && run.rows <= T && (d.need == 0 || run.need <= top)) {
                    at = before;
                    if (d.need != 0) most = run.need;
                }
            }
            need[s] = at;
        }
        if (most != 0) atomicMax(&taken, most);
        if (threadIdx.x == kThreads - 1) {
            back[S] = total.back;
            rows[S] = min(total.rows, T);
        }
    }
    __syncthreads();

    // ---- what may be the same buffers: written once every CTA has read them
    cluster.sync();
    const int threads = ctas * kThreads;
    const int me = cta * kThreads + static_cast<int>(threadIdx.x);
    for (int s = me; s < S; s += threads) {
        const int L = old[s], N = size[s];
        p.out_lens[s] = N > L && need[s] == kFull ? L : N;
    }
    for (int s = me; s <= S; s += threads) p.query_start[s] = static_cast<int>(rows[s]);
    if (me == 0) *p.out_free_count = static_cast<int>(top - taken);

    // block number r given back: its entry in the table
    auto released = [&](unsigned r) -> const int32_t * {
        const int s = find(back, S + 1, r);
        return p.tables + static_cast<int64_t>(s) * p.max_blocks + blocks(size[s]) + (r - back[s]);
    };

    // ---- rows, kBatch of them in flight for each thread
    const unsigned used = rows[S];
    for (unsigned t0 = me; t0 < T; t0 += kBatch * threads) {
        const int32_t *from[kBatch];  // where the row's block id is, or null
        int32_t *entry[kBatch];       // its table entry
        unsigned off[kBatch];
        int64_t pos[kBatch];
        bool fresh[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const unsigned t = t0 + u * threads;
            from[u] = nullptr;
            pos[u] = 0;
            if (t >= used) continue;
            const int s = find(rows, S + 1, t);
            const int L = old[s];
            pos[u] = static_cast<int64_t>(L) + (t - rows[s]);
            if (need[s] == kFull) continue;
            const unsigned blk = quotient(static_cast<unsigned>(pos[u]));
            const unsigned have = static_cast<unsigned>(blocks(L));
            off[u] = static_cast<unsigned>(pos[u]) - blk * bs;
            entry[u] = p.tables + static_cast<int64_t>(s) * p.max_blocks + blk;
            fresh[u] = blk >= have;
            if (!fresh[u]) {
                from[u] = entry[u];
            } else {
                const unsigned r = need[s] + (blk - have);
                from[u] = r < R ? released(r) : p.free_blocks + (count - 1 - static_cast<int>(r - R));
            }
        }
        int id[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) id[u] = from[u] != nullptr ? *from[u] : -1;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const unsigned t = t0 + u * threads;
            if (t >= T) break;
            int64_t slot = -1;
            if (from[u] != nullptr) {
                // (a new block's first row is a new token's)
                if (fresh[u] && off[u] == 0) *entry[u] = id[u];
                if (id[u] < 0 || id[u] >= p.num_blocks)
                    record_error(p.err, PKV_DEVERR_BLOCK_ID, entry[u] - p.tables);
                else
                    slot = static_cast<int64_t>(id[u]) * bs + off[u];
            }
            p.slots[t] = slot;
            if (p.positions != nullptr) p.positions[t] = pos[u];
        }
    }
    // ---- blocks given back, the first on top
    for (unsigned r0 = me; r0 < R; r0 += kBatch * threads) {
        int id[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (r0 + u * threads < R) id[u] = *released(r0 + u * threads);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (r0 + u * threads < R) p.free_blocks[top - 1 - (r0 + u * threads)] = id[u];
    }
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_resize_sequences(int32_t *block_tables, const int32_t *seq_lens,
                                    const int32_t *new_lens, int32_t *out_lens,
                                    int32_t *free_blocks, const int32_t *free_count,
                                    int32_t *out_free_count, int32_t *query_start,
                                    int64_t *slot_mapping, int64_t *positions, int32_t num_seqs,
                                    int32_t max_blocks_per_seq, int32_t max_tokens,
                                    int32_t free_capacity, int32_t block_size,
                                    int64_t num_blocks, pkv_stream_t stream) {
    using namespace pkv;
    if (num_seqs < 0 || max_tokens < 0 || free_capacity < 0) return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !seq_lens || !new_lens || !out_lens || !free_count || !out_free_count ||
        !query_start || (max_tokens > 0 && !slot_mapping) || (free_capacity > 0 && !free_blocks))
        return PKV_ERR_NULL;
    if (max_blocks_per_seq <= 0 || block_size <= 0 || num_blocks <= 0) return PKV_ERR_INVALID;
    if (num_seqs > kMaxSeqs || max_tokens >= static_cast<int>(kFull) ||
        free_capacity >= static_cast<int>(kFull))
        return PKV_ERR_UNSUPPORTED;
    if (!aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(new_lens, 4) ||
        !aligned(out_lens, 4) || !aligned(free_blocks, 4) || !aligned(free_count, 4) ||
        !aligned(out_free_count, 4) || !aligned(query_start, 4) || !aligned(slot_mapping, 8) ||
        !aligned(positions, 8))
        return PKV_ERR_ALIGNMENT;
    ResizeParams p{};
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.out_lens = out_lens;
    p.free_blocks = free_blocks;
    p.free_count = free_count;
    p.out_free_count = out_free_count;
    p.query_start = query_start;
    p.slots = slot_mapping;
    p.positions = positions;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.max_tokens = max_tokens;
    p.capacity = free_capacity;
    p.block_size = block_size;
    p.shift = (block_size & (block_size - 1)) == 0 ? __builtin_ctz(block_size) : -1;
    p.num_blocks = num_blocks;
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;
    const int smem = (5 * num_seqs + 2) * 4;
    const int st = prepare_kernel(reinterpret_cast<const void *>(resize_kernel), kThreads,
                                  (5 * kMaxSeqs + 2) * 4, nullptr);
    if (st != PKV_OK) return st;
    // a CTA per 1024 rows, up to a cluster
    const int ctas = std::max(1, std::min(kMaxCluster, (max_tokens + kThreads - 1) / kThreads));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, resize_kernel, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failure(e, "resize_kernel launch");
}
