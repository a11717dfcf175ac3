// gemm_grouped_4x4.hip -- FP8 products grouped by expert on tiles of 256 x 256.
#include "gemm_block128_tile.h"

namespace bsfp8 {
hipError_t launch_gemm_grouped_4x4(const GroupedArgs& t) { return launch_grouped_tile<4, 4, false>(t); }
}  // namespace bsfp8
