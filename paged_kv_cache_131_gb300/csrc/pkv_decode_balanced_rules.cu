// pkv_decode_balanced_rules.cu -- the balanced schedule's kernels under score
// rules (capped scores, bias by distance, windows, prefixes): the same body with
// the policies' rule forms, in a translation unit of their own so that they
// compile beside the others.
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
