// gemm_block128_3x2.hip -- the block-of-128 FP8 GEMM on tiles of 192 x 128.
#include "gemm_block128_tile.h"

namespace bsfp8 {
hipError_t launch_gemm_block128_3x2(const TileArgs& t) { return launch_tile<3, 2>(t); }
}  // namespace bsfp8
