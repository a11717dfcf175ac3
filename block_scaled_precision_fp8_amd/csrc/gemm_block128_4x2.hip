// gemm_block128_4x2.hip -- the block-of-128 FP8 GEMM on tiles of 256 x 128
// (16-bit outputs: for FP32 two tiles of 128 x 128 always took no longer).
#include "gemm_block128_tile.h"

namespace bsfp8 {
hipError_t launch_gemm_block128_4x2(const TileArgs& t) { return launch_tile<4, 2, false>(t); }
}  // namespace bsfp8
