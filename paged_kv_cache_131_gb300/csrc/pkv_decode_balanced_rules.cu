// pkv_decode_balanced_rules.cu -- the balanced schedule's kernels under score
// rules (capped scores, bias by distance, windows, prefixes): the same body with
// the policies' rule forms, in a translation unit of their own so that they
// compile beside the others.
//
// Blocks that no rule lets a sequence's tokens see are left out of the work list, so
// a window's call reads what it sees: 64 sequences of up to 32768 tokens (H 32, Hk 8, D
// 128), window 4096 and a prefix of 4: 155 us, 6.56 TB/s of 1.02 GB (605 us without
// the rules).  Bound by HBM in fp16 (8 x 32768 tokens with a bias: 162 us, 6.6 TB/s);
// by the consumers' instructions for drafted tokens (64 x 4: 124 us where the calls
// without rules take 114) and in FP8 (16 sequences of 8000 to 32768, capped: 131 us
// where those take 115 and the bytes 103): about 850 a head and two blocks there, issue
// slots 44% busy with two warps a scheduler, and a chain of conversion, scores, cap,
// maximum, weights and P V behind each step.
#include "pkv_decode_balanced.cuh"

namespace pkv {
namespace dec {
namespace {

template <int D, int G>
BalancedFn pick(bool fp8, int col_tiles) {
    if (col_tiles == 1) return decode_balanced_kernel<D, G, MmaColsPolicy<D, G, 1, true>, false>;
    if (col_tiles == 2) return decode_balanced_kernel<D, G, MmaColsPolicy<D, G, 2, true>, false>;
    if (fp8) return decode_balanced_kernel<D, G, MmaFp8Policy<D, G, true>, true>;
    return decode_balanced_kernel<D, G, MmaPolicy<D, G, true>, false>;
}

}  // namespace

BalancedFn select_balanced_rules(int D, int G, bool fp8, int col_tiles) {
#define PKV_CASE(d, g) \
    if (D == d && G == g) return pick<d, g>(fp8, col_tiles);
    PKV_CASE(128, 1) PKV_CASE(128, 2) PKV_CASE(128, 4) PKV_CASE(128, 8)
    PKV_CASE(64, 1) PKV_CASE(64, 2) PKV_CASE(64, 4) PKV_CASE(64, 8)
#undef PKV_CASE
    return nullptr;
}

}  // namespace dec
}  // namespace pkv
