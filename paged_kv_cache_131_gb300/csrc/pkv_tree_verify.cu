// pkv_tree_verify.cu -- verification of drafted trees against the target's
// probabilities from given random numbers (pkv_tree_verify).
//
// At a node with target p and drafts q, child after child is accepted with
// probability min(1, r/q), r being the normalised rest of the target that the
// rejections so far have left: r_0 = p, r_{j+1} = norm(max(r_j - q, 0)).  Without
// the norm, R_{j+1} = max(R_j - W_j q, 0) with W_j = sum R_j, and since
// max(max(a, 0) - b, 0) = max(a - b, 0) for b >= 0, R_j = max(p - C_j q, 0) with
// C_j = W_0 + .. + W_{j-1}: a rejection is one number and one sum over the row,
// whatever came before it, and nothing of the row is kept or written.
//
// One cluster of CTAs per sequence; every warp of it walks the tree alike (the
// nodes' probabilities are gathered into shared memory once), and all of them sum
// a row when a child is rejected or the next token is drawn: each warp a stretch
// of its CTA's share, the CTAs' sums exchanged through distributed shared memory.
// The draw finds the CTA and the warp from those sums, and that CTA goes through
// the warp's stretch again (out of L2), a few elements a thread.
//
// Arithmetic: an element of R is two fused multiply-adds of the row's fp32 values (C as
// a pair of fp32; 2^-24 of it each), four neighbours are added in fp32 (two more such
// roundings: 2^-22 of a sum in all), and from there sums, masses and tests are carried as pairs of
// fp32 whose errors are kept (47 bits).  fp64 would hold as much, but its
// rate here is 2 a cycle and SM, and every warp walks: the first kernel, in fp64,
// took 22.6, 129 and 44 us for a chain of 5 nodes, 64 trees of 16 (V 128256) and
// 32 of 63 without drafts, with pairs 9.3, 41 and 13.5.
// Bound: latency.  64 trees of 16 nodes (V 128256) take 35 us with inputs from HBM, 30
// from the L2, where their rows are 70 MB (10.4 us): the chain of the slowest sequence,
// up to six passes of 3 to 6 us; one chain of 5 takes 7.7: starts, nodes,
// probabilities, a row and the draw, each behind the one before.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;  // vectors of either row that a thread has in flight
constexpr int kMaxCluster = 8;
constexpr int kMaxNodes = PKV_MAX_TREE_NODES;
constexpr unsigned kAll = 0xffffffffu;

struct VerifyParams {
    int32_t *path;
    int32_t *path_lens;
    int32_t *next_tokens;
    const int32_t *tokens;
    const int32_t *parents;
    const int32_t *query_start;
    const float *target;
    const float *draft;
    int64_t target_stride;
    int64_t draft_stride;
    const float *accept_u;
    const float *sample_u;
    int max_depth;
    int num_nodes;
    int vocab;
    ErrorRecord *err;
};

// A uniform number as the nearest of [0, 1).
__device__ __forceinline__ float unit(float u) {
    return fminf(fmaxf(u, 0.f), 0.99999994f);  // 1 - 2^-24
}

// The rest of the target at a node.
struct Rest {
    const float *p;       // target row
    const float *q;       // drafts' row, or null
    float c_hi, c_lo;     // C
    const int *gone;      // without drafts' rows: rejected tokens
    int num_gone;
};

// Its element at index i.
__device__ __forceinline__ float rest_of(const Rest &r, float p, float q) {
    q = fmaxf(q, 0.f);  // (the maximum of a NaN and 0 is 0)
    return fmaxf(fmaf(-r.c_lo, q, fmaf(-r.c_hi, q, p)), 0.f);
}

// Elements i .. i + 3 (0 outside [0, vocab)), by 16-byte loads where `vec`
// (both rows have element i at a 16-byte boundary).
__device__ __forceinline__ void load_rest(const Rest &r, int i, int vocab, bool vec,
                                          float (&x)[4]) {
    float p[4], q[4];
    if (vec && i >= 0 && i + 4 <= vocab) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(r.p + i));
        p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
        if (r.q != nullptr) {
            const float4 b = __ldg(reinterpret_cast<const float4 *>(r.q + i));
            q[0] = b.x; q[1] = b.y; q[2] = b.z; q[3] = b.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool in = i + k >= 0 && i + k < vocab;
            p[k] = in ? __ldg(r.p + i + k) : 0.f;
            q[k] = in && r.q != nullptr ? __ldg(r.q + i + k) : 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = r.q != nullptr ? rest_of(r, p[k], q[k]) : fmaxf(p[k], 0.f);
    if (r.num_gone != 0)
        for (int g = 0; g < r.num_gone; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r.gone[g] == i + k) x[k] = 0.f;
}

// A number as the sum of two fp32, the second below half a step of the first.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair renorm(float s, float e) {
    const float h = __fadd_rn(s, e);
    return {h, __fsub_rn(e, __fsub_rn(h, s))};
}

// The rounding error of s = a + b.
__device__ __forceinline__ float sum_error(float a, float b, float s) {
    const float t = __fsub_rn(s, a);
    return __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

__device__ __forceinline__ Pair operator+(const Pair &a, const Pair &b) {
    const float s = __fadd_rn(a.hi, b.hi);
    return renorm(s, __fadd_rn(sum_error(a.hi, b.hi, s), __fadd_rn(a.lo, b.lo)));
}

__device__ __forceinline__ Pair operator-(const Pair &a, const Pair &b) {
    return a + Pair{-b.hi, -b.lo};
}

__device__ __forceinline__ Pair operator*(const Pair &a, float b) {
    const float p = __fmul_rn(a.hi, b);
    return renorm(p, __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -p)));
}

__device__ __forceinline__ bool operator<(const Pair &a, const Pair &b) {
    return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo);
}

__device__ __forceinline__ bool positive(const Pair &a) { return a.hi > 0.f; }

// s += x, the rounding error kept in e.
__device__ __forceinline__ void add_to(float &s, float &e, float x) {
    const float t = __fadd_rn(s, x);
    e = __fadd_rn(e, sum_error(s, x, t));
    s = t;
}

__device__ __forceinline__ Pair shfl_xor(const Pair &v, int o) {
    return {__shfl_xor_sync(kAll, v.hi, o), __shfl_xor_sync(kAll, v.lo, o)};
}

__device__ __forceinline__ Pair shfl(const Pair &v, int lane) {
    return {__shfl_sync(kAll, v.hi, lane), __shfl_sync(kAll, v.lo, lane)};
}

__device__ __forceinline__ Pair lanes_sum(Pair v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = v + shfl_xor(v, o);
    return v;
}

// The sum of the lanes below this one and (incl) of this one too.
__device__ __forceinline__ Pair lanes_below(const Pair &v, int lane, Pair *incl) {
    Pair run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y = {__shfl_up_sync(kAll, run.hi, o), __shfl_up_sync(kAll, run.lo, o)};
        if (lane >= o) run = run + y;
    }
    *incl = run;
    const Pair below = {__shfl_up_sync(kAll, run.hi, 1), __shfl_up_sync(kAll, run.lo, 1)};
    return lane == 0 ? Pair{0.f, 0.f} : below;
}

// Lane of the share in which the running sum passes `goal`: the last one with
// anything in it whose sum before it is not above the goal; -1 if all are empty.
__device__ __forceinline__ int lane_of(const Pair &share, const Pair &before, const Pair &goal) {
    const unsigned any = __ballot_sync(kAll, positive(share));
    const unsigned fit = __ballot_sync(kAll, positive(share) && !(goal < before));
    return fit != 0 ? 31 - __clz(fit) : __ffs(any) - 1;
}

__global__ void __launch_bounds__(kThreads, 3)
    tree_verify_kernel(const __grid_constant__ VerifyParams p) {
    // per node: its token's probability under its parent's target and drafts
    __shared__ float node_p[kMaxNodes], node_q[kMaxNodes], node_u[kMaxNodes];
    __shared__ int node_token[kMaxNodes];
    __shared__ int node_up[kMaxNodes];      // its parent; -1: never a child
    __shared__ int gone[kWarps][kMaxNodes];  // fixed guesses rejected at this node, by warp
    __shared__ Pair warp_part[2][kWarps];       // this CTA's warps, by parity of the pass
    __shared__ Pair cta_part[2][kMaxCluster];   // every CTA's sum, written by it
    __shared__ Pair draw_part[kWarps];
    __shared__ int draw_first, draw_last;
    __shared__ Pair draw_before;
    auto cluster = cooperative_groups::this_cluster();
    const int cta = static_cast<int>(cluster.block_rank());
    const int ctas = static_cast<int>(cluster.num_blocks());
    const int seq = static_cast<int>(blockIdx.x) / ctas;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int V = p.vocab;
    const bool drafted = p.draft != nullptr;

    cluster.barrier_arrive();
    grid_dependency_wait();
    const int row0 = __ldg(p.query_start + seq), row1 = __ldg(p.query_start + seq + 1);
    const bool in = row0 >= 0 && row1 >= row0 && row1 <= p.num_nodes;  // (so row1 - row0 fits)
    int Q = in ? row1 - row0 : 0;
    if (!in || Q > kMaxNodes) {
        if (cta == 0 && threadIdx.x == 0) record_error(p.err, PKV_DEVERR_SEQ_LEN, seq);
        Q = 0;
    }
    int32_t *path = p.path + static_cast<int64_t>(seq) * p.max_depth;
    if (Q == 0) {  // (the whole cluster)
        cluster.barrier_wait();
        if (cta == 0) {
            for (int d = threadIdx.x; d < p.max_depth; d += kThreads) path[d] = -1;
            if (threadIdx.x == 0) {
                p.path_lens[seq] = 0;
                p.next_tokens[seq] = -1;
            }
        }
        return;
    }
    for (int k = threadIdx.x; k < Q; k += kThreads) {
        const int64_t row = row0 + k;
        const int parent = __ldg(p.parents + row), token = __ldg(p.tokens + row);
        float a = 0.f, b = 0.f;
        int up = -1;
        if (k > 0 && parent >= 0) {
            if (parent >= k || token < 0 || token >= V) {
                if (cta == 0) record_error(p.err, PKV_DEVERR_TREE, row);
            } else {
                up = parent;
                a = __ldg(p.target + (row0 + parent) * p.target_stride + token);
                if (drafted) b = __ldg(p.draft + (row0 + parent) * p.draft_stride + token);
            }
        }
        node_p[k] = a;
        node_q[k] = b;
        node_u[k] = unit(__ldg(p.accept_u + row));
        node_token[k] = token;
        node_up[k] = up;
    }
    const float draw_u = unit(__ldg(p.sample_u + seq));
    __syncthreads();
    // (the first exchange writes other CTAs' shared memory: all have started by then)
    cluster.barrier_wait();

    int pass = 0;
    bool vec = false;
    int first = 0, last = 0;  // this warp's stretch of the row
    Rest r{};
    // Points r at node `at`'s rows with nothing rejected.
    auto open = [&](int at) {
        r.p = p.target + (row0 + at) * p.target_stride;
        r.q = nullptr;
        r.c_hi = r.c_lo = 0.f;
        r.gone = gone[warp];
        r.num_gone = 0;
        const uintptr_t pa = reinterpret_cast<uintptr_t>(r.p) & 15;
        const float *q = drafted ? p.draft + (row0 + at) * p.draft_stride : r.p;
        vec = pa == (reinterpret_cast<uintptr_t>(q) & 15);
        // stretches of 128 elements from the 16-byte boundary at or before the row
        const int skew = static_cast<int>(pa >> 2);
        const int units = (V + skew + 127) / 128, parts = ctas * kWarps;
        const int part = cta * kWarps + warp;
        first = static_cast<int>(static_cast<int64_t>(units) * part / parts) * 128 - skew;
        last = static_cast<int>(static_cast<int64_t>(units) * (part + 1) / parts) * 128 - skew;
    };
    // The sum of the rest over the whole row, the same in every thread of the
    // cluster; its parts stay in warp_part / cta_part until the pass after next.
    auto sum_rest = [&]() -> Pair {
        float s = 0.f, e = 0.f;
        int i = first + 4 * lane;
        // whole batches of 16-byte vectors, every load before the first use
        if (vec && r.num_gone == 0) {
            for (; i < min(last, 0); i += 128) {
                float x[4];
                load_rest(r, i, V, vec, x);
                add_to(s, e, (x[0] + x[1]) + (x[2] + x[3]));
            }
            const int whole = min(last, V) - (kBatch - 1) * 128 - 4;
            if (r.q == nullptr) {
                for (; i <= whole; i += kBatch * 128) {
                    float4 a[kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j)
                        a[j] = __ldg(reinterpret_cast<const float4 *>(r.p + i + j * 128));
#pragma unroll
                    for (int j = 0; j < kBatch; ++j)
                        add_to(s, e, (fmaxf(a[j].x, 0.f) + fmaxf(a[j].y, 0.f)) +
                                         (fmaxf(a[j].z, 0.f) + fmaxf(a[j].w, 0.f)));
                }
            } else {
                for (; i <= whole; i += kBatch * 128) {
                    float4 a[kBatch], b[kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        a[j] = __ldg(reinterpret_cast<const float4 *>(r.p + i + j * 128));
                        b[j] = __ldg(reinterpret_cast<const float4 *>(r.q + i + j * 128));
                    }
#pragma unroll
                    for (int j = 0; j < kBatch; ++j)
                        add_to(s, e, (rest_of(r, a[j].x, b[j].x) + rest_of(r, a[j].y, b[j].y)) +
                                         (rest_of(r, a[j].z, b[j].z) + rest_of(r, a[j].w, b[j].w)));
                }
            }
        }
        for (; i < last; i += 128) {
            float x[4];
            load_rest(r, i, V, vec, x);
            add_to(s, e, (x[0] + x[1]) + (x[2] + x[3]));
        }
        const Pair w = lanes_sum(renorm(s, e));
        const int half = pass & 1;
        ++pass;
        if (lane == 0) warp_part[half][warp] = w;
        __syncthreads();
        if (warp == 0) {
            const Pair c = lanes_sum(lane < kWarps ? warp_part[half][lane] : Pair{0.f, 0.f});
            if (lane < ctas) *cluster.map_shared_rank(&cta_part[half][cta], lane) = c;
        }
        cluster.sync();
        return lanes_sum(lane < ctas ? cta_part[half][lane] : Pair{0.f, 0.f});
    };

    // ---- the walk (every warp of the cluster alike)
    int at = 0, depth = 1;
    int seen = 0;  // fixed guesses rejected at this node (r.num_gone once they are all)
    bool summed = false;  // the last pass summed r as it stands
    Pair total{0.f, 0.f};
    if (cta == 0 && threadIdx.x == 0) path[0] = 0;
    for (;;) {
        open(at);
        summed = false;
        int step = -1;
        seen = 0;
        if (depth < p.max_depth) {
            Pair W{1.f, 0.f}, C{0.f, 0.f};
            bool empty = false;
            for (int j = (at + 1) >> 5; j < (Q + 31) >> 5 && step < 0 && !empty; ++j) {
                const int node = 32 * j + lane;
                unsigned kids = __ballot_sync(kAll, node < Q && node_up[node] == at);
                while (kids != 0 && step < 0 && !empty) {
                    const int k = 32 * j + __ffs(kids) - 1;
                    kids &= kids - 1;
                    const float u = node_u[k], pt = fmaxf(node_p[k], 0.f);
                    const float qt = fmaxf(node_q[k], 0.f);
                    if (drafted) {
                        const Pair have = Pair{pt, 0.f} - C * qt;
                        if (positive(have) && (W * u) * qt < have) {
                            step = k;
                            break;
                        }
                        // rejected: the rest without what the drafts cover
                        const Rest before = r;
                        C = C + W;
                        r.q = p.draft + (row0 + at) * p.draft_stride;
                        r.c_hi = C.hi;
                        r.c_lo = C.lo;
                        const Pair w = sum_rest();
                        if (positive(w)) {
                            W = total = w;
                            summed = true;
                        } else {
                            r = before;
                            summed = false;
                            empty = true;
                        }
                    } else {
                        // (a guess that was rejected before has nothing left)
                        const int token = node_token[k];
                        bool again = false;
                        for (int g = lane; g < seen; g += 32) again = again || gone[warp][g] == token;
                        again = __any_sync(kAll, again);
                        const Pair have{again ? 0.f : pt, 0.f};
                        if (W * u < have) {
                            step = k;
                            break;
                        }
                        const Pair less = W - have;
                        if (!positive(less)) {
                            empty = true;
                        } else {
                            W = less;
                            if (!again) {
                                if (lane == 0) gone[warp][seen] = token;
                                __syncwarp();
                                ++seen;
                            }
                        }
                    }
                }
            }
        }
        if (step < 0) break;
        if (cta == 0 && threadIdx.x == 0) path[depth] = step;
        ++depth;
        at = step;
    }

    // ---- the next token
    r.num_gone = seen;
    if (!summed) total = sum_rest();
    const int half = (pass - 1) & 1;
    if (cta == 0) {
        for (int d = depth + threadIdx.x; d < p.max_depth; d += kThreads) path[d] = -1;
        if (threadIdx.x == 0) p.path_lens[seq] = depth;
    }
    if (!positive(total)) {
        if (cta == 0 && threadIdx.x == 0) p.next_tokens[seq] = -1;
        return;
    }
    const Pair goal = total * draw_u;
    Pair incl;
    {
        // the CTA, then its warp, in whose share the running sum passes the goal
        const Pair share = lane < ctas ? cta_part[half][lane] : Pair{0.f, 0.f};
        const Pair before = lanes_below(share, lane, &incl);
        const int c = lane_of(share, before, goal);
        if (c != cta) return;
        const Pair base = shfl(before, c);
        const Pair part = lane < kWarps ? warp_part[half][lane] : Pair{0.f, 0.f};
        const Pair start = base + lanes_below(part, lane, &incl);
        const int w = lane_of(part, start, goal);
        if (warp == w && lane == w) {
            draw_first = first;
            draw_last = last;
            draw_before = start;
        }
    }
    __syncthreads();
    // its stretch again, the same number of neighbouring elements for each thread
    const int each = ((draw_last - draw_first + kThreads - 1) / kThreads + 3) & ~3;
    const int from = draw_first + static_cast<int>(threadIdx.x) * each;
    const int to = min(from + each, draw_last);
    float s = 0.f, e = 0.f;
    for (int i = from; i < to; i += 4) {
        float x[4];
        load_rest(r, i, V, vec, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) add_to(s, e, x[k]);
    }
    const Pair mine = renorm(s, e);
    Pair before = lanes_below(mine, lane, &incl);
    if (lane == 31) draw_part[warp] = incl;
    __syncthreads();
    {
        const Pair part = lane < kWarps ? draw_part[lane] : Pair{0.f, 0.f};
        const Pair start = draw_before + lanes_below(part, lane, &incl);
        if (lane_of(part, start, goal) != warp) return;
        before = shfl(start, warp) + before;
    }
    if (lane_of(mine, before, goal) != lane) return;
    // this thread's elements one by one; the last one with anything in it where
    // rounding leaves the sum at or below the goal
    int token = -1;
    Pair run = before;
    for (int i = from; i < to; i += 4) {
        float x[4];
        load_rest(r, i, V, vec, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (x[k] > 0.f && (token < 0 || !(goal < run))) token = i + k;
            run = run + Pair{x[k], 0.f};
        }
    }
    p.next_tokens[seq] = token;
}

// CTAs of a sequence's cluster: as many (up to 8, and a vector of 16 bytes for each
// thread) as let all sequences' clusters run at once, since a sequence that starts when
// another ends adds its whole chain to the call -- 64 sequences of V 128256: 33.6 us
// with 6 CTAs, all at once; 37.7 with 7 and 40.2 with 8, which do not all fit; 43.7
// with 4.  Returns a negative number on a CUDA error.
int cluster_size(int num_seqs, int vocab) {
    constexpr int kDevices = 256;
    static std::atomic<int> fits[kDevices][kMaxCluster];  // 1 + clusters at once; 0: not asked
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_failure(e, "cudaGetDevice");
    const int most = std::max(1, std::min(kMaxCluster, (vocab + 4 * kThreads - 1) / (4 * kThreads)));
    for (int c = most; c > 1; --c) {
        int n = dev < kDevices ? fits[dev][c - 1].load(std::memory_order_relaxed) - 1 : -1;
        if (n < 0) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = c;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(c));
            cfg.blockDim = dim3(kThreads);
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, tree_verify_kernel, &cfg);
            if (e != cudaSuccess) return cuda_failure(e, "cudaOccupancyMaxActiveClusters");
            if (dev < kDevices) fits[dev][c - 1].store(n + 1, std::memory_order_relaxed);
        }
        if (n >= num_seqs) return c;
    }
    return 1;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_tree_verify(int32_t *path, int32_t max_depth, int32_t *path_lens,
                               int32_t *next_tokens, const int32_t *draft_tokens,
                               const int32_t *parents, const int32_t *query_start,
                               const float *target_probs, int64_t target_stride,
                               const float *draft_probs, int64_t draft_stride,
                               const float *accept_uniforms, const float *sample_uniforms,
                               int32_t num_seqs, int32_t num_nodes, int32_t vocab_size,
                               pkv_stream_t stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_nodes < 0) return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    if (!path || !path_lens || !next_tokens || !query_start || !sample_uniforms ||
        (num_nodes > 0 && (!draft_tokens || !parents || !target_probs || !accept_uniforms)))
        return PKV_ERR_NULL;
    if (max_depth <= 0 || vocab_size <= 0 || target_stride < vocab_size ||
        (draft_probs != nullptr && draft_stride < vocab_size))
        return PKV_ERR_INVALID;
    if (max_depth > PKV_MAX_ACCEPT_DEPTH || vocab_size > (1 << 30) ||
        num_seqs > INT32_MAX / kMaxCluster)
        return PKV_ERR_UNSUPPORTED;
    if (!aligned(path, 4) || !aligned(path_lens, 4) || !aligned(next_tokens, 4) ||
        !aligned(draft_tokens, 4) || !aligned(parents, 4) || !aligned(query_start, 4) ||
        !aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(accept_uniforms, 4) ||
        !aligned(sample_uniforms, 4))
        return PKV_ERR_ALIGNMENT;
    VerifyParams p{};
    p.path = path;
    p.path_lens = path_lens;
    p.next_tokens = next_tokens;
    p.tokens = draft_tokens;
    p.parents = parents;
    p.query_start = query_start;
    p.target = target_probs;
    p.draft = draft_probs;
    p.target_stride = target_stride;
    p.draft_stride = draft_stride;
    p.accept_u = accept_uniforms;
    p.sample_u = sample_uniforms;
    p.max_depth = max_depth;
    p.num_nodes = num_nodes;
    p.vocab = vocab_size;
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;
    const int ctas = cluster_size(num_seqs, vocab_size);
    if (ctas < 0) return PKV_ERR_CUDA;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_seqs) * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, tree_verify_kernel, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failure(e, "tree_verify_kernel launch");
}
