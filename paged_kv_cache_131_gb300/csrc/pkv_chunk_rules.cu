// pkv_chunk_rules.cu -- the chunk tile kernels under score rules, in a translation
// unit of their own so that they compile beside the plain ones.
#include "pkv_chunk.cuh"

namespace pkv {
namespace chunk {
namespace {

template <int D>
ChunkFn pick(bool capped, bool biased) {
    if (capped)
        return biased ? chunk_attention_kernel<D, kRuled | kCapped | kBiased>
                      : chunk_attention_kernel<D, kRuled | kCapped>;
    return biased ? chunk_attention_kernel<D, kRuled | kBiased> : chunk_attention_kernel<D, kRuled>;
}

}  // namespace

ChunkFn select_chunk_rules(int D, bool capped, bool biased) {
    if (D == 128) return pick<128>(capped, biased);
    if (D == 64) return pick<64>(capped, biased);
    return nullptr;
}

}  // namespace chunk
}  // namespace pkv
