// gemm_grouped_wgrad_2x2.hip -- FP8 products over groups of K values on tiles of 128 x 128.
#include "gemm_block128_tile.h"

namespace bsfp8 {
hipError_t launch_gemm_wgrad_2x2(const GroupedKArgs& t) {
    return by_type(t, [](auto AF, auto BF, auto OUT, const GroupedKArgs& g) {
        return g.fast_ok() ? launch_columns<AF, BF, OUT, 2, 2, true>(g) : launch_columns<AF, BF, OUT, 2, 2, false>(g);
    });
}
}  // namespace bsfp8
