// gemm_grouped.h -- shared by the forms of the grouped block-of-128 FP8 products.
//
// Products are summed as in the ungrouped product: for 16-bit outputs by the FP8 matrix instruction, twice as fast as
// bf16's, which keeps 13 fraction bits within a group of products (up to 7 2^-13 of sum |a b|, about 2% of bf16 outputs
// one step from those of FP32 sums); for FP32 output in bf16, which is exact for the codes.
#pragma once

#include "gemm_block128.h"
#include "groups.h"

namespace bsfp8 {

// What the tiled forms' epilogue by buffer stores takes: 32-bit offsets within a tile's rows, and C for
// FP32 output only.  Rows of D and C may start at any element (the hardware takes 16 bytes at any address).
inline bool fast_epilogue(int out, int64_t ldd, const Epilogue& ep) {
    constexpr int64_t most = int64_t(1) << 21;
    return ldd < most && ep.ldc < most && (out == BSFP8_OUT_F32 || ep.beta == 0.0f);
}

// D[i] = alpha A[i] B[e(i)]^T (+ beta C[i]): b and its scales are `groups`
// matrices one after another; sb.words points to the first one's.
struct GroupedArgs {
    int64_t M, N, K;
    int groups;
    const int32_t* offsets;
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
    bool fast_ok() const { return fast_epilogue(out, ldd, ep); }
};
hipError_t launch_gemm_grouped(const GroupedArgs& t);
hipError_t launch_gemm_grouped_rows(const GroupedArgs& t);
hipError_t launch_gemm_grouped_4x4(const GroupedArgs& t);
hipError_t launch_gemm_grouped_2x2(const GroupedArgs& t);
hipError_t launch_gemm_grouped_1x2(const GroupedArgs& t);

// D[e] = alpha sum over group e's columns i of A[:, i] B[:, i]^T (+ beta C[e]):
// K values `columns` to a row, each group's from a multiple of 128 on and its scales from a word on.
struct GroupedKArgs {
    int64_t M, N, columns, words;
    int groups;
    const int32_t* offsets;
    int a_fmt;
    const uint8_t* a;
    const uint32_t* sa;
    int b_fmt;
    const uint8_t* b;
    const uint32_t* sb;
    int out;
    void* d;
    int64_t ldd, d_group, c_group;
    Epilogue ep;
    hipStream_t stream;
    bool fast_ok() const { return fast_epilogue(out, ldd, ep); }
};
hipError_t launch_gemm_grouped_wgrad(const GroupedKArgs& t);
hipError_t launch_gemm_wgrad_narrow(const GroupedKArgs& t);
hipError_t launch_gemm_wgrad_4x4(const GroupedKArgs& t);           // 16-bit outputs
hipError_t launch_gemm_wgrad_4x4_f32(const GroupedKArgs& t);
hipError_t launch_gemm_wgrad_2x2(const GroupedKArgs& t);

// Which form a call runs on (0 few rows or 32 x 32 tiles, 1 64 x 128, 2 128 x 128, 3 256 x 256), for the tests.
int gemm_grouped_form(int64_t M, int64_t N, int64_t K, int groups, int out, int64_t ldd, int64_t ldc, float beta);
int gemm_wgrad_form(int64_t M, int64_t N, int64_t columns, int groups, int out, int64_t ldd, int64_t ldc, float beta);

// finish_row_chunk for four columns at any alignment: a whole chunk moves in one access (the hardware
// takes any element's address).  With D of 2001 columns 32 products 1000 x 2001 x 69 took
// 106 us element by element, 81 so.
template <int OUT>
__device__ __forceinline__ void finish_chunk(void* D, int64_t ldd, const Epilogue& ep, int m, int n, int M, int N, float4 acc) {
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t h4 __attribute__((ext_vector_type(2), aligned(2)));
    if (m >= M || n >= N) return;
    const bool whole = n + 4 <= N;
    float v[4] = {ep.alpha * acc.x, ep.alpha * acc.y, ep.alpha * acc.z, ep.alpha * acc.w};
    if (ep.beta != 0.0f) {
        const int64_t at = static_cast<int64_t>(m) * ep.ldc + n;
        float c[4] = {};
        if constexpr (OUT == BSFP8_OUT_F32) {
            const float* p = static_cast<const float*>(ep.c) + at;
            if (whole) {
                const f4 w = *reinterpret_cast<const f4*>(p);
#pragma unroll
                for (int j = 0; j < 4; ++j) c[j] = w[j];
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (n + j < N) c[j] = p[j];
            }
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(ep.c) + at;
            if (whole) {
                const h4 w = *reinterpret_cast<const h4*>(p);
#pragma unroll
                for (int j = 0; j < 4; ++j) c[j] = from_half_bits<OUT>(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (n + j < N) c[j] = from_half_bits<OUT>(p[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(ep.beta, c[j], v[j]);
    }
    const int64_t at = static_cast<int64_t>(m) * ldd + n;
    if constexpr (OUT == BSFP8_OUT_F32) {
        float* p = static_cast<float*>(D) + at;
        if (whole) {
            *reinterpret_cast<f4*>(p) = f4{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (n + j < N) p[j] = v[j];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(D) + at;
        uint16_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = to_half_bits<OUT>(v[j]);
        if (whole) {
            *reinterpret_cast<h4*>(p) = h4{h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16)};
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (n + j < N) p[j] = h[j];
        }
    }
}

// launch(A's format, B's format, output type, args) with the three as constants.
template <class T, class F>
hipError_t by_type(const T& t, F&& launch) {
    auto outs = [&](auto AF, auto BF) {
        if (t.out == BSFP8_OUT_F32) return launch(AF, BF, std::integral_constant<int, BSFP8_OUT_F32>{}, t);
        if (t.out == BSFP8_OUT_BF16) return launch(AF, BF, std::integral_constant<int, BSFP8_OUT_BF16>{}, t);
        return launch(AF, BF, std::integral_constant<int, BSFP8_OUT_F16>{}, t);
    };
    constexpr std::integral_constant<int, BSFP8_E4M3> e4m3{};
    constexpr std::integral_constant<int, BSFP8_E5M2> e5m2{};
    if (t.a_fmt == BSFP8_E4M3) return t.b_fmt == BSFP8_E4M3 ? outs(e4m3, e4m3) : outs(e4m3, e5m2);
    return t.b_fmt == BSFP8_E4M3 ? outs(e5m2, e4m3) : outs(e5m2, e5m2);
}

}  // namespace bsfp8
