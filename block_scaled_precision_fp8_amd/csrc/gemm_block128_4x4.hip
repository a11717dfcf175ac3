// gemm_block128_4x4.hip -- the block-of-128 FP8 GEMM on tiles of 256 x 256.
#include "gemm_block128_tile.h"

namespace bsfp8 {
hipError_t launch_gemm_block128_4x4(const TileArgs& t) { return launch_tile<4, 4>(t); }
}  // namespace bsfp8
