// pkv_norm_rope.cu -- per-head norm of queries and keys, rotation by position
// and the paged cache write, in one pass over the rows of the QKV product.
//
// For a head row x of a token at position p (fp32 throughout):
//     n_d = x_d w_d rsqrt(mean_d x_d^2 + eps),
//     a' = a cos_i - b sin_i,  b' = b cos_i + a sin_i   for pair i = (a, b) of n,
// rounded once: to fp16 for q_out and fp16 caches; for FP8 caches to
// s = amax/448 and the E4M3 codes nearest y / s, from the fp32 values (no fp16
// rounding in between).
//
// A row of D fp16 is held by D/8 lanes, 8 dims (one 16-byte load) each, so the
// sum over a row, and the other halves of its pairs, are shuffles inside 8 or
// 16 lanes.  A token's rows are cut into chunks of kRows rows per row group,
// all of one kind (query, key or value); a warp's job is a run of chunks of
// one token, the next chunk's rows loaded while this one's are worked on (the
// first ones before it is known whether the token is padding).  Weights and
// rotation are two factors per dim, A = w cos and B = -+ w' sin, made once per
// job and kind: y = rsqrt(..) (x A + x' B).  Large calls get long jobs (fewer
// factors made), small ones a chunk per warp.
//
// Bound: HBM -- every row read and written once; the table's rows come from L2.
// 32 query and 8 KV heads of 128 dims: 16384 tokens 74.4 us into fp16 caches
// (5.5 TB/s), 82 us into FP8 ones (4.5 TB/s).  Chunks of 4 rows: 77 and 90 us;
// a third more resident warps: 86 and 100 (spills); a chunk per warp: 139 and
// 154 (the factors are then made per chunk).
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
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 2;       // rows per row group and chunk
constexpr int kMinBlocks = 6;  // resident blocks per SM
// A job's start-up (factors, first loads) as the choice of job length counts it, in
// chunks.  1, 2, 4, 8: 16384 tokens 78.3, 75.1, 75.1, 75.1 us, into FP8 caches 88.0,
// 82.4, 82.4, 82.4; 4000 tokens 23.2, 21.8, 21.7, 23.8; 2001 tokens of 64 query heads
// into FP8 caches 18.9, 18.9, 17.4, 20.8 (in a graph; the last two sizes out of
// the L2); up to 1000 tokens all the same.
constexpr int kJobStart = 4;

struct NormRopeParams {
    const __half *src[3];  // q, k, v
    int64_t stride[3];     // elements between tokens
    __half *q_out;         // [T, H, D]
    void *cache[2];        // [NB, bs, Hk, D] fp16 or codes
    float *scale[2];       // [NB, bs, Hk] (FP8)
    const __half *weight[2];
    float eps;
    const float *table;  // [max_position][rot]: rot/2 cosines, rot/2 sines
    int64_t max_position;
    int32_t rot;
    int32_t interleaved;
    const int64_t *positions;
    const int64_t *slot_mapping;
    int64_t num_slots;
    uint32_t num_jobs;
    uint32_t jobs_per_token;
    int32_t job_chunks;    // chunks of a job
    int32_t token_chunks;  // of a token: the queries', the keys', the values'
    int32_t query_chunks;
    int32_t row_chunks;    // of the keys, and of the values
    int32_t num_heads;
    int32_t num_kv_heads;
    ErrorRecord *err;
};

__device__ __forceinline__ void unpack8(const uint4 &r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_half2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Packed fp32 pairs: one instruction for two dims.
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
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void unpack_pairs(const uint4 &r, uint64_t (&x)[4]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_half2(w[i]);
        x[i] = f32x2(f.x, f.y);
    }
}
__device__ __forceinline__ uint4 pack_pairs(const uint64_t (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = f32x2_split(x[i]);
        w[i] = pack_half2(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return static_cast<uint32_t>(
        __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}

// The factors of a lane's dims d0 .. d0 + 7 (their other halves': dp on) at
// position pos, with this weight (or none).
__device__ __forceinline__ void make_factors(const NormRopeParams &p, const __half *weight,
                                             int64_t pos, int d0, int dp, bool rotates,
                                             bool second, uint64_t (&A)[4], uint64_t (&B)[4]) {
    const int half = p.rot >> 1;
    float w[8], wp[8], a[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
    if (weight != nullptr) {
        unpack8(__ldg(reinterpret_cast<const uint4 *>(weight + d0)), w);
        if (rotates && !p.interleaved)
            unpack8(__ldg(reinterpret_cast<const uint4 *>(weight + dp)), wp);
    }
    if (!rotates) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] = w[e];
            b[e] = 0.f;
        }
    } else {
        const float4 *cs = reinterpret_cast<const float4 *>(p.table + pos * p.rot);
        if (p.interleaved) {  // pairs d0/2 .. d0/2 + 3
            const float4 c = __ldg(cs + d0 / 8), s = __ldg(cs + half / 4 + d0 / 8);
            const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[2 * e] = w[2 * e] * cv[e];
                b[2 * e] = -w[2 * e + 1] * sv[e];
                a[2 * e + 1] = w[2 * e + 1] * cv[e];
                b[2 * e + 1] = w[2 * e] * sv[e];
            }
        } else {  // pairs d0 .. d0 + 7, or those of the other half
            const int i0 = (second ? dp : d0) / 4;
            const float4 c0 = __ldg(cs + i0), c1 = __ldg(cs + i0 + 1);
            const float4 s0 = __ldg(cs + half / 4 + i0), s1 = __ldg(cs + half / 4 + i0 + 1);
            const float cv[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[e] = w[e] * cv[e];
                b[e] = (second ? wp[e] : -wp[e]) * sv[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        A[e] = f32x2(a[2 * e], a[2 * e + 1]);
        B[e] = f32x2(b[2 * e], b[2 * e + 1]);
    }
}

// A token's chunk: kind, first row of the warp's first row group.
struct Chunk {
    int kind;  // query, key, value; or none
    int h0;
};

template <int D>
__device__ __forceinline__ Chunk chunk_of(const NormRopeParams &p, int c) {
    constexpr int kChunk = 256 / D * kRows;
    if (c < p.query_chunks) return Chunk{0, c * kChunk};
    c -= p.query_chunks;
    if (c < p.row_chunks) return Chunk{1, c * kChunk};
    return Chunk{2, (c - p.row_chunks) * kChunk};
}

// D: head_dim; FP8: quantised caches.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, kMinBlocks)
    norm_rope_write_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LPR = D / 8;    // lanes per row
    constexpr int RG = 32 / LPR;  // row groups of a warp
    const uint32_t job = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (job >= p.num_jobs) return;
    const int lane = threadIdx.x & 31;
    const int d0 = 8 * (lane % LPR), rg = lane / LPR;
    const uint32_t token = job / p.jobs_per_token;
    const int64_t t = token;
    int c = static_cast<int>(job - token * p.jobs_per_token) * p.job_chunks;
    const int c1 = min(c + p.job_chunks, p.token_chunks);
    const int half = p.rot >> 1;
    const bool rotates = d0 < p.rot;
    const bool second = d0 >= half;  // the b half of its pairs
    const int dp = second ? d0 - half : d0 + half;  // the other halves' dims
    const int partner = rotates && !p.interleaved ? lane + (dp - d0) / 8 : lane;
    auto load = [&](const Chunk &ch, uint4 (&r)[kRows]) {
        const int heads = ch.kind == 0 ? p.num_heads : p.num_kv_heads;
        const __half *src =
            (ch.kind == 0 ? p.src[0] : ch.kind == 1 ? p.src[1] : p.src[2]) +
            t * (ch.kind == 0 ? p.stride[0] : ch.kind == 1 ? p.stride[1] : p.stride[2]) +
            (ch.h0 + rg) * D + d0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            r[i] = make_uint4(0u, 0u, 0u, 0u);
            if (ch.h0 + rg + i * RG < heads)
                r[i] = *reinterpret_cast<const uint4 *>(src + i * RG * D);
        }
    };
    grid_dependency_wait();  // the rows may come from the kernel just before
    const int64_t slot = p.slot_mapping[t];
    const int64_t pos = p.rot ? p.positions[t] : 0;
    Chunk ch = chunk_of<D>(p, c);
    uint4 next[kRows];
    load(ch, next);
    if (slot < 0) return;  // padding
    const bool bad_slot = slot >= p.num_slots;
    if (bad_slot || (p.rot && (pos < 0 || pos >= p.max_position))) {
        if (lane == 0) record_error(p.err, bad_slot ? PKV_DEVERR_SLOT : PKV_DEVERR_POSITION, t);
        return;
    }
    uint64_t A[4], B[4];  // the factors of dims 2i, 2i + 1
    int made = -1;        // the kind they are for
    const __half *weight = nullptr;
    while (true) {
        uint4 raw[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) raw[i] = next[i];
        const int kind = ch.kind, h0 = ch.h0 + rg;
        const int heads = kind == 0 ? p.num_heads : p.num_kv_heads;
        const bool more = ++c < c1;
        if (more) {
            ch = chunk_of<D>(p, c);
            load(ch, next);
        }
        if (kind < 2 && kind != made) {
            made = kind;
            weight = kind == 0 ? p.weight[0] : p.weight[1];
            make_factors(p, weight, pos, d0, dp, rotates, second, A, B);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int h = h0 + i * RG;
            const bool live = h < heads;
            if (!FP8 && kind == 2) {  // values move as they are
                if (live)
                    *reinterpret_cast<uint4 *>(static_cast<__half *>(p.cache[1]) +
                                               (slot * heads + h) * D + d0) = raw[i];
                continue;
            }
            uint64_t x[4];
            unpack_pairs(raw[i], x);
            if (kind < 2) {
                uint64_t r2 = f32x2(1.f, 1.f);
                if (weight != nullptr) {
                    uint64_t q2 = mul_f32x2(x[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) q2 = fma_f32x2(x[e], x[e], q2);
                    const float2 q = f32x2_split(q2);
                    float ss = q.x + q.y;
#pragma unroll
                    for (int o = LPR / 2; o >= 1; o >>= 1)
                        ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float r = rsqrtf(ss * (1.f / D) + p.eps);
                    r2 = f32x2(r, r);
                }
                uint64_t y[4];
                if (p.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 v = f32x2_split(x[e]);
                        y[e] = f32x2(v.y, v.x);
                    }
                } else {
                    uint4 o;
                    o.x = __shfl_sync(0xffffffffu, raw[i].x, partner);
                    o.y = __shfl_sync(0xffffffffu, raw[i].y, partner);
                    o.z = __shfl_sync(0xffffffffu, raw[i].z, partner);
                    o.w = __shfl_sync(0xffffffffu, raw[i].w, partner);
                    unpack_pairs(o, y);
                }
                // (a dim that is not rotated meets no other)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t z = mul_f32x2(x[e], A[e]);
                    x[e] = mul_f32x2(rotates ? fma_f32x2(y[e], B[e], z) : z, r2);
                }
            }
            if constexpr (FP8) {
                if (kind > 0) {
                    float v[8], amax = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = f32x2_split(x[e]);
                        v[2 * e] = f.x;
                        v[2 * e + 1] = f.y;
                        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
#pragma unroll
                    for (int o = LPR / 2; o >= 1; o >>= 1)
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    if (!live) continue;
                    const float sc = amax / 448.f;  // 448: E4M3's largest finite value
                    if (sc > 0x1p-100f && sc < 0x1p100f) {
                        // x / sc rounded to nearest from the rounded reciprocal
                        // r and one correction, q + r (x - q sc) with q = x r
                        // (Markstein 1990): three operations instead of a
                        // division's.  (Where x - q sc underflows, the code is 0.)
                        const float r = 1.f / sc;
                        const uint64_t r2 = f32x2(r, r), ns2 = f32x2(-sc, -sc);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint64_t q = mul_f32x2(x[e], r2);
                            const float2 f = f32x2_split(fma_f32x2(fma_f32x2(q, ns2, x[e]), r2, q));
                            v[2 * e] = copysignf(f.x, v[2 * e]);  // (the correction of -0 is +0)
                            v[2 * e + 1] = copysignf(f.y, v[2 * e + 1]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = sc == 0.f ? 0.f : v[e] / sc;
                    }
                    const int64_t at = slot * heads + h;
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.cache[kind - 1]) +
                                               at * D + d0) =
                        make_uint2(e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16),
                                   e4m3x2(v[4], v[5]) | (e4m3x2(v[6], v[7]) << 16));
                    if (d0 == 0) p.scale[kind - 1][at] = sc;
                    continue;
                }
            }
            if (!live) continue;
            __half *dst = kind == 0 ? p.q_out + (t * heads + h) * D
                                    : static_cast<__half *>(p.cache[0]) + (slot * heads + h) * D;
            *reinterpret_cast<uint4 *>(dst + d0) = pack_pairs(x);
        }
        if (!more) break;
    }
}

int norm_rope_write(void *q_out, const void *q, const void *k, const void *v, int64_t q_stride,
                    int64_t k_stride, int64_t v_stride, const pkv_norm_rope *nr,
                    const int64_t *positions, const int64_t *slot_mapping, int64_t num_tokens,
                    void *k_cache, void *v_cache, float *k_scale, float *v_scale, bool fp8,
                    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                    int32_t block_size, int64_t num_blocks, pkv_stream_t stream) {
    if (num_tokens < 0) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!q_out || !q || !k || !v || !nr || !slot_mapping || !k_cache || !v_cache ||
        (fp8 && (!k_scale || !v_scale)))
        return PKV_ERR_NULL;
    if (nr->rot_dim != 0 && (!nr->cos_sin || !positions)) return PKV_ERR_NULL;
    if (num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || num_blocks > INT64_MAX / block_size || q_stride < 0 || k_stride < 0 ||
        v_stride < 0 || nr->rot_dim < 0 || nr->rot_dim > head_dim ||
        (nr->rot_dim != 0 && nr->max_position <= 0) || !std::isfinite(nr->eps) || nr->eps < 0.f)
        return PKV_ERR_INVALID;
    if (q_out == q && q_stride != static_cast<int64_t>(num_heads) * head_dim && num_tokens > 1)
        return PKV_ERR_INVALID;
    if ((head_dim != 64 && head_dim != 128) || nr->rot_dim % 16 != 0 || num_heads > 4096 ||
        num_kv_heads > 4096)
        return PKV_ERR_UNSUPPORTED;
    if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(nr->q_weight, 16) || !aligned(nr->k_weight, 16) ||
        !aligned(nr->cos_sin, 16) || !aligned(positions, 8) || !aligned(slot_mapping, 8) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return PKV_ERR_ALIGNMENT;
    NormRopeParams p{};
    p.src[0] = static_cast<const __half *>(q);
    p.src[1] = static_cast<const __half *>(k);
    p.src[2] = static_cast<const __half *>(v);
    p.stride[0] = q_stride;
    p.stride[1] = k_stride;
    p.stride[2] = v_stride;
    p.q_out = static_cast<__half *>(q_out);
    p.cache[0] = k_cache;
    p.cache[1] = v_cache;
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.weight[0] = static_cast<const __half *>(nr->q_weight);
    p.weight[1] = static_cast<const __half *>(nr->k_weight);
    p.eps = nr->eps;
    p.table = nr->cos_sin;
    p.max_position = nr->max_position;
    p.rot = nr->rot_dim;
    p.interleaved = nr->interleaved != 0;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.num_slots = num_blocks * block_size;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    const int chunk_rows = 32 / (head_dim / 8) * kRows;
    p.query_chunks = (num_heads + chunk_rows - 1) / chunk_rows;
    p.row_chunks = (num_kv_heads + chunk_rows - 1) / chunk_rows;
    p.token_chunks = p.query_chunks + 2 * p.row_chunks;
    if (num_tokens > INT32_MAX / static_cast<int64_t>(p.token_chunks)) return PKV_ERR_UNSUPPORTED;
    // the job length with the shortest estimated time: rounds of the resident
    // warps, times a job's chunks and its start-up (kJobStart chunks)
    const int64_t warps = static_cast<int64_t>(sm_count()) * kMinBlocks * (kThreads / 32);
    int64_t best = INT64_MAX;
    for (int c = 1; c <= p.token_chunks; ++c) {
        const int64_t jobs = num_tokens * ((p.token_chunks + c - 1) / c);
        const int64_t cost = (jobs + warps - 1) / warps * (c + kJobStart);
        if (cost < best) {
            best = cost;
            p.job_chunks = c;
        }
    }
    p.jobs_per_token = static_cast<uint32_t>((p.token_chunks + p.job_chunks - 1) / p.job_chunks);
    p.num_jobs = static_cast<uint32_t>(num_tokens) * p.jobs_per_token;
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;
    using Fn = void (*)(const NormRopeParams);
    const Fn fn = head_dim == 128 ? (fp8 ? norm_rope_write_kernel<128, true>
                                         : norm_rope_write_kernel<128, false>)
                                  : (fp8 ? norm_rope_write_kernel<64, true>
                                         : norm_rope_write_kernel<64, false>);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.num_jobs + kThreads / 32 - 1) / (kThreads / 32));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failure(e, "norm_rope_write_kernel launch");
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_norm_rope_write(void *q_out, const void *q, const void *k, const void *v,
                                   int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                   const pkv_norm_rope *norm_rope, const int64_t *positions,
                                   const int64_t *slot_mapping, int64_t num_tokens,
                                   void *k_cache, void *v_cache, int32_t num_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                   int64_t num_blocks, pkv_stream_t stream) {
    return pkv::norm_rope_write(q_out, q, k, v, q_stride, k_stride, v_stride, norm_rope,
                                positions, slot_mapping, num_tokens, k_cache, v_cache, nullptr,
                                nullptr, false, num_heads, num_kv_heads, head_dim, block_size,
                                num_blocks, stream);
}

extern "C" int pkv_norm_rope_write_fp8(void *q_out, const void *q, const void *k, const void *v,
                                       int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                       const pkv_norm_rope *norm_rope, const int64_t *positions,
                                       const int64_t *slot_mapping, int64_t num_tokens,
                                       void *k_cache, void *v_cache, float *k_scale,
                                       float *v_scale, int32_t num_heads, int32_t num_kv_heads,
                                       int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                       pkv_stream_t stream) {
    return pkv::norm_rope_write(q_out, q, k, v, q_stride, k_stride, v_stride, norm_rope,
                                positions, slot_mapping, num_tokens, k_cache, v_cache, k_scale,
                                v_scale, true, num_heads, num_kv_heads, head_dim, block_size,
                                num_blocks, stream);
}
