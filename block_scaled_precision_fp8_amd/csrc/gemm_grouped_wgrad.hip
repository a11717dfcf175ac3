// gemm_grouped_wgrad.hip -- FP8 products over the rows of each group, one power-of-two
// scale per 128 of them (gfx950):
//
//   D[e][m][n] = alpha sum_{i in group e} A[m][i] B[n][i] (+ beta C[e][m][n]),
//
// the weight gradients of experts.  A and B are transposes that
// quantize_grouped.hip wrote: a group's columns start at a multiple of 128 and end in
// zeros, its scale bytes start at a word.  A group without rows gives beta C.
//
// One workgroup per 32 x 32 tile of a group's D, its four waves taking contiguous
// ranges of the group's K blocks, as the narrow form of gemm_block128.hip.
#include "gemm_grouped.h"

namespace bsfp8 {

namespace {

using namespace big_tile;

constexpr int kDepth = 2;
constexpr int kWaves = 4;

template <int AF, int BF, int OUT>
__global__ __launch_bounds__(64 * kWaves, 2) void gemm_grouped_wgrad_kernel(
    int M, int N, int64_t columns, int64_t words, int count, const int32_t* __restrict__ offsets,
    const uint8_t* __restrict__ A, const uint32_t* __restrict__ sA, const uint8_t* __restrict__ B,
    const uint32_t* __restrict__ sB, void* __restrict__ D, int64_t ldd, int64_t d_group, int64_t c_group, Epilogue ep,
    int tiles_m, int tiles_n) {
    __shared__ v16f part[kWaves - 1][64];
    __shared__ __attribute__((aligned(16))) uint8_t stage[kWaves][2][32 * 128];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = tiles_m * tiles_n;
    const int e = blockIdx.x / tiles, t = blockIdx.x - e * tiles;
    const int m0 = t / tiles_n * 32, n0 = t % tiles_n * 32;
    const groups::Lane own = groups::at<128>(offsets, count, static_cast<int>(min(columns, int64_t(1) << 30)), e);
    // what the buffers hold, whatever the offsets are
    const int nkb = static_cast<int>(max(int64_t(0), min(min(static_cast<int64_t>(own.tiles), (columns >> 7) - own.tile),
                                                         4 * (words - own.word))));
    const int per = (nkb + kWaves - 1) / kWaves;
    const int c0 = min(wave * per, nkb), c1 = min(c0 + per, nkb);

    const int ld = static_cast<int>(columns);
    const int rows_a = min(32, M - m0), rows_b = min(32, N - n0);
    const int64_t k0 = static_cast<int64_t>(own.tile) * 128;
    const int span = nkb * 128;
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(A) + static_cast<int64_t>(m0) * columns + k0, 0, nkb ? (rows_a - 1) * ld + span : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(B) + static_cast<int64_t>(n0) * columns + k0, 0, nkb ? (rows_b - 1) * ld + span : 0, 0x00020000);
    const int r = lane & 31, h = lane >> 5;
    const uint32_t* words_a = sA + static_cast<int64_t>(own.word) * M + min(m0 + r, M - 1);
    const uint32_t* words_b = sB + static_cast<int64_t>(own.word) * N + min(n0 + r, N - 1);
    const int lr = lane >> 3, lg = lane & 7;
    uint8_t* st_a = stage[wave][0];
    uint8_t* st_b = stage[wave][1];
    u32x4 ga[kDepth][4], gb[kDepth][4];
    uint32_t wa[kDepth], wb[kDepth];
    auto fetch = [&](auto SLOT, int c) {
        constexpr int j = SLOT;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = c < c1 ? static_cast<uint32_t>((lr + 8 * i) * ld + 128 * c + 16 * lg) : 0x80000000u;
            const auto a = __builtin_amdgcn_raw_buffer_load_b128(rs_a, static_cast<int>(o), 0, 0);
            const auto b = __builtin_amdgcn_raw_buffer_load_b128(rs_b, static_cast<int>(o), 0, 0);
            ga[j][i] = u32x4{a[0], a[1], a[2], a[3]};
            gb[j][i] = u32x4{b[0], b[1], b[2], b[3]};
        }
        // past the range: no word (its codes are zero)
        wa[j] = c < c1 ? words_a[static_cast<int64_t>(c >> 2) * M] : 0x7F7F7F7Fu;
        wb[j] = c < c1 ? words_b[static_cast<int64_t>(c >> 2) * N] : 0x7F7F7F7Fu;
    };
    v16f acc = v16f{};
    static_for<kDepth>([&](auto J) { fetch(J, c0 + J); });
    for (int c = c0; c < c1; c += kDepth) {
        static_for<kDepth>([&](auto J) {
            constexpr int j = J;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = lr + 8 * i;
                const int pos = row * 128 + 16 * (lg ^ (row & 7));
                *reinterpret_cast<u32x4*>(st_a + pos) = ga[j][i];
                *reinterpret_cast<u32x4*>(st_b + pos) = gb[j][i];
            }
            const int sh = ((c + j) & 3) * 8;
            const uint32_t sa = (wa[j] >> sh) & 255u, sb = (wb[j] >> sh) & 255u;
            fetch(J, c + j + kDepth);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u32x4 xa[2], xb[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int pos = r * 128 + 16 * ((4 * s + 2 * q + h) ^ (r & 7));
                    xa[q] = *reinterpret_cast<const u32x4*>(st_a + pos);
                    xb[q] = *reinterpret_cast<const u32x4*>(st_b + pos);
                }
                acc = step64<AF, BF, OUT>(xb[0], xb[1], xa[0], xa[1], sb, sa, acc);
            }
        });
    }
    if (wave > 0) part[wave - 1][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) {
        const v16f q = part[w][lane];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] += q[i];
    }
    constexpr int es = OUT == BSFP8_OUT_F32 ? 4 : 2;
    ep.c = ep.c ? static_cast<const uint8_t*>(ep.c) + e * c_group * es : nullptr;
    void* d = static_cast<uint8_t*>(D) + e * d_group * es;
    // lane (r, h) holds row m0 + r, columns n0 + 8 q + 4 h + i in acc[4 q + i]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        finish_chunk<OUT>(d, ldd, ep, m0 + r, n0 + 8 * q + 4 * h, M, N,
                          make_float4(acc[4 * q + 0], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]));
    }
}

template <int AF, int BF, int OUT>
hipError_t launch_out(const GroupedKArgs& t) {
    const int tm = static_cast<int>((t.M + 31) / 32), tn = static_cast<int>((t.N + 31) / 32);
    hipLaunchKernelGGL((gemm_grouped_wgrad_kernel<AF, BF, OUT>),
                       dim3(static_cast<uint32_t>(static_cast<int64_t>(tm) * tn * t.groups)), dim3(64 * kWaves), 0,
                       t.stream, static_cast<int>(t.M), static_cast<int>(t.N), t.columns, t.words, t.groups, t.offsets,
                       t.a, t.sa, t.b, t.sb, t.d, t.ldd, t.d_group, t.c_group, t.ep, tm, tn);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_wgrad_narrow(const GroupedKArgs& t) {
    return by_type(t, [](auto AF, auto BF, auto OUT, const GroupedKArgs& g) { return launch_out<AF, BF, OUT>(g); });
}

}  // namespace bsfp8
