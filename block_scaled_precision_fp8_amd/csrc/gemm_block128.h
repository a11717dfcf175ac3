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

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
using big_tile::u32x4;
using big_tile::v16f;

// acc += x^T y over 64 K values of one scale block; x: row operand (B, scale
// byte sb), y: column operand (A, scale byte sa), each lane's 32 codes in two
// quarters.  All 64 K values share the scales, so the order of K within the
// step is free as long as both operands use the same one.
template <int AF, int BF, int OUT>
__device__ __forceinline__ v16f step64(const u32x4& x0, const u32x4& x1, const u32x4& y0, const u32x4& y1,
                                       uint32_t sb, uint32_t sa, v16f acc) {
    if constexpr (OUT != BSFP8_OUT_F32) {
        const v8i x = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
        const v8i y = {(int)y0[0], (int)y0[1], (int)y0[2], (int)y0[3], (int)y1[0], (int)y1[1], (int)y1[2], (int)y1[3]};
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, mfma_fmt<BF>(), mfma_fmt<AF>(), 0,
                                                               static_cast<int>(sb), 0, static_cast<int>(sa));
    } else {
        const float fb = __uint_as_float(sb << 23), fa = __uint_as_float(sa << 23);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const u32x4& xs = q < 2 ? x0 : x1;
            const u32x4& ys = q < 2 ? y0 : y1;
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8<BF>(xs[2 * (q & 1)], xs[2 * (q & 1) + 1], fb),
                                                          widen8<AF>(ys[2 * (q & 1)], ys[2 * (q & 1) + 1], fa), acc, 0, 0, 0);
        }
        return acc;
    }
}

// acc += x^T y over one K block, byte J of the scale words; x: rows of B.
template <int AF, int BF, int OUT, int J>
__device__ __forceinline__ v4f block_product(const u32x4& x0, const u32x4& x1, const u32x4& y0, const u32x4& y1,
                                             uint32_t sb, uint32_t sa, v4f acc) {
    if constexpr (OUT != BSFP8_OUT_F32) {
        const v8i x = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
        const v8i y = {(int)y0[0], (int)y0[1], (int)y0[2], (int)y0[3], (int)y1[0], (int)y1[1], (int)y1[2], (int)y1[3]};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, mfma_fmt<BF>(), mfma_fmt<AF>(), J,
                                                                static_cast<int>(sb), J, static_cast<int>(sa));
    } else {
        const float fb = __uint_as_float(((sb >> (8 * J)) & 255u) << 23), fa = __uint_as_float(((sa >> (8 * J)) & 255u) << 23);
        typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const u32x4& xs = q < 2 ? x0 : x1;
            const u32x4& ys = q < 2 ? y0 : y1;
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf8v, widen8<BF>(xs[2 * (q & 1)], xs[2 * (q & 1) + 1], fb)),
                __builtin_bit_cast(bf8v, widen8<AF>(ys[2 * (q & 1)], ys[2 * (q & 1) + 1], fa)), acc, 0, 0, 0);
        }
        return acc;
    }
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
