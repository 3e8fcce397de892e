// pkv_read_fp8.cu -- rows of an FP8 (E4M3) cache read back in 16 bits: the
// inverse of the quantising write.  Row (t, h) = value(code) * scale of slot
// slot_mapping[t], the product in fp32, rounded to fp16 once (the code's value
// is exact in fp16 and in fp32).
//
// A token's Hk*D codes are contiguous in the cache and its outputs contiguous
// in the rows, so a thread's unit is 16 codes: one 16-byte load, one scale
// (head_dim is a multiple of 16), one 32-byte store.  Each thread has
// kUnits units in flight, one block of threads apart, so loads and stores of a
// warp cover consecutive bytes.  A unit's token is a division, 32-bit wherever
// the call has fewer than 2^31 units.
// Bound: HBM -- 1 + 4/D bytes read and 2 written per value: 131072 tokens of 8
// heads of 128 dims (815 MB) 121 us, 6.7 TB/s (4 units per thread: 127 us, 1:
// 139); 953 tokens of 4 heads of 64 dims 2 us.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;

struct ReadParams {
    __half *dst[2];
    const uint8_t *cache[2];
    const float *scale[2];
    const int64_t *slot_mapping;
    int64_t num_slots;
    int64_t num_units;  // 16-code units of one cache
    uint32_t units_per_token;
    uint32_t units_per_head;
    int32_t num_kv_heads;
    ErrorRecord *err;
};

// Two E4M3 codes (low byte first) times s, as an fp16 pair.
__device__ __forceinline__ uint32_t dequant2(uint32_t codes, float s) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return pack_half2(f.x * s, f.y * s);
}

// Unit: the type that holds the call's unit indexes.
template <typename Unit>
__global__ void __launch_bounds__(kThreads)
    cache_read_fp8_kernel(const __grid_constant__ ReadParams p) {
    const int c = blockIdx.y;
    const Unit u0 = static_cast<Unit>(blockIdx.x) * (kThreads * kUnits) + threadIdx.x;
    grid_dependency_wait();  // the cache may be written by the kernel just before
    int64_t slot[kUnits];
    uint32_t w[kUnits];  // unit inside the token's row
    uint4 codes[kUnits];
    float scale[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = u0 + i * kThreads;
        slot[i] = -1;
        if (u < static_cast<Unit>(p.num_units)) {
            const Unit t = u / p.units_per_token;
            w[i] = static_cast<uint32_t>(u - t * p.units_per_token);
            slot[i] = __ldg(p.slot_mapping + t);
            if (slot[i] >= p.num_slots) {
                record_error(p.err, PKV_DEVERR_SLOT, static_cast<long long>(t));
                slot[i] = -1;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (slot[i] < 0) continue;
        codes[i] = __ldg(reinterpret_cast<const uint4 *>(p.cache[c]) +
                         slot[i] * p.units_per_token + w[i]);
        scale[i] = __ldg(p.scale[c] + slot[i] * p.num_kv_heads + w[i] / p.units_per_head);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (slot[i] < 0) continue;
        const uint32_t in[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
        uint32_t r[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[2 * e] = dequant2(in[e], scale[i]);
            r[2 * e + 1] = dequant2(in[e] >> 16, scale[i]);
        }
        __half *dst = p.dst[c] + static_cast<int64_t>(u0 + i * kThreads) * 16;
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                     "r"(r[7])
                     : "memory");
    }
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_cache_read_fp8(void *k, void *v, const int64_t *slot_mapping,
                                  int64_t num_tokens, const void *k_cache, const void *v_cache,
                                  const float *k_scale, const float *v_scale,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                  int64_t num_blocks, pkv_stream_t stream) {
    using namespace pkv;
    if (num_tokens < 0) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !k_cache || !k_scale || !slot_mapping) return PKV_ERR_NULL;
    if ((v == nullptr) != (v_cache == nullptr) || (v == nullptr) != (v_scale == nullptr))
        return PKV_ERR_NULL;
    if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        num_blocks > INT64_MAX / block_size)
        return PKV_ERR_INVALID;
    if ((head_dim != 64 && head_dim != 128) || num_kv_heads > 65536) return PKV_ERR_UNSUPPORTED;
    if (!aligned(k, 32) || !aligned(v, 32) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(slot_mapping, 8))
        return PKV_ERR_ALIGNMENT;
    ReadParams p{};
    p.dst[0] = static_cast<__half *>(k);
    p.dst[1] = static_cast<__half *>(v);
    p.cache[0] = static_cast<const uint8_t *>(k_cache);
    p.cache[1] = static_cast<const uint8_t *>(v_cache);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.slot_mapping = slot_mapping;
    p.num_slots = num_blocks * block_size;
    p.num_kv_heads = num_kv_heads;
    p.units_per_head = static_cast<uint32_t>(head_dim / 16);
    p.units_per_token = static_cast<uint32_t>(num_kv_heads) * p.units_per_head;
    if (num_tokens > INT64_MAX / static_cast<int64_t>(p.units_per_token)) return PKV_ERR_INVALID;
    p.num_units = num_tokens * static_cast<int64_t>(p.units_per_token);
    const int64_t grid = (p.num_units + kThreads * kUnits - 1) / (kThreads * kUnits);
    if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    p.err = device_error_record();
    if (p.err == nullptr) return PKV_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), v ? 2 : 1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // (the last block's indexes too)
    cudaError_t e = p.num_units < INT32_MAX - kThreads * kUnits
                        ? cudaLaunchKernelEx(&cfg, cache_read_fp8_kernel<uint32_t>, p)
                        : cudaLaunchKernelEx(&cfg, cache_read_fp8_kernel<uint64_t>, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failure(e, "cache_read_fp8_kernel launch");
}
