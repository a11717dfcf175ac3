// gemm_grouped_wgrad_4x4.hip -- FP8 products over groups of K values on tiles of 256 x 256, 16-bit outputs.
#include "gemm_block128_tile.h"

namespace bsfp8 {
hipError_t launch_gemm_wgrad_4x4(const GroupedKArgs& t) {
    return by_type(t, [](auto AF, auto BF, auto OUT, const GroupedKArgs& g) {
        if constexpr (OUT == BSFP8_OUT_F32) return hipErrorInvalidValue;
        else return g.fast_ok() ? launch_columns<AF, BF, OUT, 4, 4, true>(g) : hipErrorInvalidValue;
    });
}
}  // namespace bsfp8
