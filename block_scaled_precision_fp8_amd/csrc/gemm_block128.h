// gemm_block128.h -- shared by the forms of the block-of-128 FP8 GEMM.
#pragma once

#include "big_tile.h"

namespace bsfp8 {

// One operand's scales: byte j of word (g, r) is the scale of K block 4 g + j
// of scale row r; shift is 0 (a scale row per row) or 7 (one per 128 rows).
struct ScaleRows {
    const uint32_t* words;
    int64_t rows;
    int shift;
};

template <int FMT>
constexpr int mfma_fmt() { return FMT == BSFP8_E4M3 ? 0 : 1; }

// One product, for the tiled forms (one source file per tile size: A rows x B
// rows in units of 64).
struct TileArgs {
    int64_t M, N, K;
    int a_fmt;
    const uint8_t* a;
    ScaleRows sa;
    int b_fmt;
    const uint8_t* b;
    ScaleRows sb;
    int out;
    void* d;
    int64_t ldd;
    Epilogue ep;
    hipStream_t stream;
};
hipError_t launch_gemm_block128_4x4(const TileArgs& t);
hipError_t launch_gemm_block128_4x2(const TileArgs& t);
hipError_t launch_gemm_block128_3x2(const TileArgs& t);
hipError_t launch_gemm_block128_2x2(const TileArgs& t);

}  // namespace bsfp8
