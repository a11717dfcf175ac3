// gemm_grouped_2x2.hip -- FP8 products grouped by expert on tiles of 128 x 128.
#include "gemm_block128_tile.h"

namespace bsfp8 {
hipError_t launch_gemm_grouped_2x2(const GroupedArgs& t) { return launch_grouped_tile<2, 2, true>(t); }
}  // namespace bsfp8
