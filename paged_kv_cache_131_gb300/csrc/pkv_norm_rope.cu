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
// sum over a row is shuffles inside 8 or 16 lanes.  A warp's job is kRows rows
// for each of its row groups, all of one token and one kind (query, key or
// value).  Every load of the job is issued before the first is used, the other
// halves of the pairs among them (a second load of the same line instead of
// shuffles), and before it is known whether the token is padding.  Weights
// and rotation are two factors per dim, A = w cos and B = -+ w' sin, shared by
// the job's rows: y = rsqrt(..) (x A + x' B).
//
// Bound: HBM -- every row read and written once; the table's rows come from L2
// or, for a token's later jobs, L1.
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

constexpr int kThreads = 256;
constexpr int kRows = 4;  // rows per row group and job

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
    int32_t query_jobs;  // the first of a token's jobs; then the keys', the values'
    int32_t row_jobs;    // of the keys, and of the values
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

// D: head_dim; FP8: quantised caches.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads)
    norm_rope_write_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LPR = D / 8;    // lanes per row
    constexpr int RG = 32 / LPR;  // row groups of a warp
    const uint32_t job = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (job >= p.num_jobs) return;
    const int lane = threadIdx.x & 31;
    const int d0 = 8 * (lane % LPR), rg = lane / LPR;
    const uint32_t token = job / p.jobs_per_token;
    const int64_t t = token;
    int j = static_cast<int>(job - token * p.jobs_per_token);
    int kind = 0;  // query, key, value
    if (j >= p.query_jobs) {
        j -= p.query_jobs;
        kind = 1;
        if (j >= p.row_jobs) {
            j -= p.row_jobs;
            kind = 2;
        }
    }
    const int heads = kind == 0 ? p.num_heads : p.num_kv_heads;
    const int h0 = j * (RG * kRows) + rg;
    const __half *src = (kind == 0 ? p.src[0] : kind == 1 ? p.src[1] : p.src[2]) +
                        t * (kind == 0 ? p.stride[0] : kind == 1 ? p.stride[1] : p.stride[2]);
    const int half = p.rot >> 1;
    const bool rotates = kind < 2 && d0 < p.rot;
    const bool halves = rotates && !p.interleaved;
    const bool second = d0 >= half;  // the b half of its pairs
    const int dp = second ? d0 - half : d0 + half;  // the other halves' dims
    grid_dependency_wait();  // the rows may come from the kernel just before
    const int64_t slot = p.slot_mapping[t];
    const int64_t pos = p.rot ? p.positions[t] : 0;
    uint4 raw[kRows], other[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const __half *row = src + (h0 + i * RG) * D;
        raw[i] = other[i] = make_uint4(0u, 0u, 0u, 0u);
        if (h0 + i * RG < heads) {
            raw[i] = *reinterpret_cast<const uint4 *>(row + d0);
            if (halves) other[i] = *reinterpret_cast<const uint4 *>(row + dp);
        }
    }
    if (slot < 0) return;  // padding
    const bool bad_slot = slot >= p.num_slots;
    if (bad_slot || (p.rot && (pos < 0 || pos >= p.max_position))) {
        if (lane == 0) record_error(p.err, bad_slot ? PKV_DEVERR_SLOT : PKV_DEVERR_POSITION, t);
        return;
    }
    uint64_t A[4], B[4];  // the factors of dims 2i, 2i + 1
    const __half *weight = kind == 0 ? p.weight[0] : p.weight[1];
    if (kind < 2) {
        float w[8], wp[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
        if (weight != nullptr) {
            unpack8(__ldg(reinterpret_cast<const uint4 *>(weight + d0)), w);
            if (halves) unpack8(__ldg(reinterpret_cast<const uint4 *>(weight + dp)), wp);
        }
        float a[8], b[8];
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
    __syncwarp();  // (the queries may be rewritten in place)
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
                for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
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
                unpack_pairs(other[i], y);
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
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = sc == 0.f ? 0.f : v[e] / sc;
                const int64_t at = slot * heads + h;
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.cache[kind - 1]) + at * D +
                                           d0) =
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
    const int job_rows = 32 / (head_dim / 8) * kRows;
    p.query_jobs = (num_heads + job_rows - 1) / job_rows;
    p.row_jobs = (num_kv_heads + job_rows - 1) / job_rows;
    p.jobs_per_token = static_cast<uint32_t>(p.query_jobs + 2 * p.row_jobs);
    if (num_tokens > INT32_MAX / static_cast<int64_t>(p.jobs_per_token)) return PKV_ERR_UNSUPPORTED;
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
