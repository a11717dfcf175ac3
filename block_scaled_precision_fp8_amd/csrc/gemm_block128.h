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

// 256 x 256 tiles.
hipError_t launch_gemm_block128_big(int64_t M, int64_t N, int64_t K, int a_fmt, const uint8_t* a, const ScaleRows& sa,
                                    int b_fmt, const uint8_t* b, const ScaleRows& sb, int out, void* d, int64_t ldd,
                                    const Epilogue& ep, hipStream_t stream);

}  // namespace bsfp8
