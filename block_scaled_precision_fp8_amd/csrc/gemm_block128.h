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

// Eight FP8 codes (two dwords) times the scale -> eight bf16 (four dwords),
// exactly as long as the products are normal bf16.
template <int FMT>
__device__ __forceinline__ big_tile::u32x4 widen8(uint32_t w0, uint32_t w1, float s) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    bf2 a, b, c, d;
    if constexpr (FMT == BSFP8_E4M3) {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true);
    } else {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w0, s, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w0, s, true);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w1, s, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w1, s, true);
    }
    return big_tile::u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                 __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}

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
// Up to 16 rows of A and a few thousand columns.
constexpr int64_t kRowsMaxM = 16;
constexpr int64_t kRowsMaxN = 5120;
hipError_t launch_gemm_block128_rows(const TileArgs& t);
hipError_t launch_gemm_block128_4x4(const TileArgs& t);
hipError_t launch_gemm_block128_4x2(const TileArgs& t);
hipError_t launch_gemm_block128_3x2(const TileArgs& t);
hipError_t launch_gemm_block128_2x2(const TileArgs& t);

}  // namespace bsfp8
