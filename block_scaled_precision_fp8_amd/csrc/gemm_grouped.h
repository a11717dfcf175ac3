// gemm_grouped.h -- shared by the forms of the grouped block-of-128 FP8 products.
#pragma once

#include "gemm_block128.h"
#include "groups.h"

namespace bsfp8 {

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
};
hipError_t launch_gemm_grouped(const GroupedArgs& t);

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
};

hipError_t launch_gemm_grouped_wgrad(const GroupedKArgs& t);

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
