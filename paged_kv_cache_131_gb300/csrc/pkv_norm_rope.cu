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
// sums over a row are shuffles inside 8 or 16 lanes and a pair's other half is
// at most one shuffle away.  A warp's job is kRows rows for each of its row
// groups, all of one token: every load of the job is issued before the first
// is used, and the token's cosines and sines are read once for all its rows.
//
// Bound: HBM -- every row read and written once.  The table's rows come from
// L2 or, for a token's later jobs, L1.
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
    int64_t num_jobs;
    int32_t jobs_per_token;
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

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]),
                      pack_half2(x[6], x[7]));
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return static_cast<uint32_t>(
        __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}

// D: head_dim; FP8: quantised caches.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads)
    norm_rope_write_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LPR = D / 8;     // lanes per row
    constexpr int RG = 32 / LPR;   // row groups of a warp
    constexpr int kJobRows = RG * kRows;
    const int lane = threadIdx.x & 31;
    const int sl = lane % LPR, rg = lane / LPR;
    const int d0 = 8 * sl;
    const int H = p.num_heads, Hk = p.num_kv_heads;
    const int rows = H + 2 * Hk;
    const int half = p.rot >> 1;
    const bool rotates = d0 < p.rot;
    const bool second = !p.interleaved && d0 >= half;  // the b half of its pairs
    const int partner = p.interleaved || !rotates ? lane : second ? lane - half / 8 : lane + half / 8;
    grid_dependency_wait();  // the rows may come from the kernel just before
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * kThreads) >> 5;
    for (int64_t job = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
         job < p.num_jobs; job += nwarps) {
        const int64_t t = job / p.jobs_per_token;
        const int row0 = static_cast<int>(job - t * p.jobs_per_token) * kJobRows + rg;
        const int64_t slot = p.slot_mapping[t];
        const int64_t pos = p.rot ? p.positions[t] : 0;
        if (slot < 0) continue;  // padding
        const bool bad_slot = slot >= p.num_slots;
        if (bad_slot || (p.rot && (pos < 0 || pos >= p.max_position))) {
            if (lane == 0)
                record_error(p.err, bad_slot ? PKV_DEVERR_SLOT : PKV_DEVERR_POSITION, t);
            continue;
        }
        uint4 raw[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int row = row0 + i * RG;
            const int kind = row < H ? 0 : row < H + Hk ? 1 : 2;
            const int h = row - (kind == 0 ? 0 : kind == 1 ? H : H + Hk);
            if (row < rows)
                raw[i] = *reinterpret_cast<const uint4 *>(p.src[kind] + t * p.stride[kind] +
                                                          h * D + d0);
        }
        // this lane's cosines and sines: pairs d0 .. d0+7 (halves) or
        // d0/2 .. d0/2 + 3 (interleaved)
        float c[8], s[8];
        if (rotates) {
            const float *row = p.table + pos * p.rot;
            const int i0 = p.interleaved ? d0 / 2 : second ? d0 - half : d0;
            *reinterpret_cast<float4 *>(c) = __ldg(reinterpret_cast<const float4 *>(row + i0));
            *reinterpret_cast<float4 *>(s) =
                __ldg(reinterpret_cast<const float4 *>(row + half + i0));
            if (!p.interleaved) {
                *reinterpret_cast<float4 *>(c + 4) =
                    __ldg(reinterpret_cast<const float4 *>(row + i0 + 4));
                *reinterpret_cast<float4 *>(s + 4) =
                    __ldg(reinterpret_cast<const float4 *>(row + half + i0 + 4));
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int row = row0 + i * RG;
            const bool live = row < rows;
            const int kind = row < H ? 0 : row < H + Hk ? 1 : 2;
            const int h = row - (kind == 0 ? 0 : kind == 1 ? H : H + Hk);
            float x[8];
            if (live) {
                unpack8(raw[i], x);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
            }
            const __half *w = kind < 2 ? p.weight[kind] : nullptr;
            // (the shuffles run in every lane; rows of other kinds drop the sum)
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (w != nullptr) {
                const float r = rsqrtf(ss * (1.f / D) + p.eps);
                float wf[8];
                unpack8(__ldg(reinterpret_cast<const uint4 *>(w + d0)), wf);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * r * wf[e];
            }
            if (p.interleaved) {
                if (rotates && kind < 2) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = x[2 * e], b = x[2 * e + 1];
                        x[2 * e] = a * c[e] - b * s[e];
                        x[2 * e + 1] = b * c[e] + a * s[e];
                    }
                }
            } else if (p.rot) {
                const float sign = second ? 1.f : -1.f;
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
                if (rotates && kind < 2) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = x[e] * c[e] + sign * y[e] * s[e];
                }
            }
            if constexpr (FP8) {
                float amax = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
                for (int o = LPR / 2; o >= 1; o >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                if (live && kind > 0) {
                    const float sc = amax / 448.f;  // 448: E4M3's largest finite value
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = sc == 0.f ? 0.f : x[e] / sc;
                    const int64_t at = slot * Hk + h;
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.cache[kind - 1]) + at * D +
                                               d0) =
                        make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16),
                                   e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
                    if (sl == 0) p.scale[kind - 1][at] = sc;
                    continue;
                }
            }
            if (!live) continue;
            __half *dst = kind == 0 ? p.q_out + (t * H + h) * D
                                    : static_cast<__half *>(p.cache[kind - 1]) +
                                          (slot * Hk + h) * D;
            // values move as they are (their bits, not a round trip through fp32)
            *reinterpret_cast<uint4 *>(dst + d0) = kind == 2 ? raw[i] : pack8(x);
        }
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
    p.jobs_per_token = (num_heads + 2 * num_kv_heads + job_rows - 1) / job_rows;
    if (num_tokens > INT64_MAX / p.jobs_per_token) return PKV_ERR_INVALID;
    p.num_jobs = num_tokens * p.jobs_per_token;
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;
    using Fn = void (*)(const NormRopeParams);
    const Fn fn = head_dim == 128 ? (fp8 ? norm_rope_write_kernel<128, true>
                                         : norm_rope_write_kernel<128, false>)
                                  : (fp8 ? norm_rope_write_kernel<64, true>
                                         : norm_rope_write_kernel<64, false>);
    const int64_t want = (p.num_jobs + kThreads / 32 - 1) / (kThreads / 32);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(want, 1 << 20)));
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
