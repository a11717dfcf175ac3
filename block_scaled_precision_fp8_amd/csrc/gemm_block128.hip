// gemm_block128.hip -- FP8 GEMM with one power-of-two (E8M0) scale per 128
// consecutive K values (gfx950).
//
//   D[m][n] = alpha sum_kb 2^(ea(m, kb) + eb(n, kb)) sum_{k in kb} qa[m][k] qb[n][k]  (+ beta C[m][n]),
//
// ea per row (1 x 128 blocks) or per 128 rows (128 x 128 blocks) of A, eb
// likewise of B.  For 16-bit outputs the scales go to the matrix core with the
// codes: v_mfma_scale_f32_32x32x64_f8f6f4 multiplies each lane's 32 K values by
// its row's E8M0 byte, so the sum over all of K stays in the accumulators and
// no VALU work is done per block.  FP32 output needs more than that
// instruction's 13 fraction bits per group of 8 products: there the codes are
// widened to bf16 with their scale (exact in bf16's normal range) and multiplied by
// v_mfma_f32_32x32x16_bf16, which keeps 24.
//
// Scale bytes lie in words of four K blocks, [ceil(K / 512)][scale rows][4]: a
// lane reads one word per 512 K, and the 32 rows of a tile lie side by side.
#include "gemm_block128.h"

namespace bsfp8 {

namespace {

using namespace big_tile;
typedef int v8i __attribute__((ext_vector_type(8)));

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

// Narrow form: one workgroup per 32 x 32 output tile, its four waves taking
// contiguous ranges of the K blocks.  Each load instruction reads whole
// 128-byte row segments (8 rows x 128 bytes), which pass through the wave's
// own LDS area into the MFMA layout; kDepth K blocks are in flight.  Range-
// checked buffer loads: rows past M or N and chunks past K read as zero.  The
// four partial sums are added in a fixed order.
constexpr int kNarrowDepth = 2;
constexpr int kNarrowWaves = 4;

template <int AF, int BF, int OUT>
__global__ __launch_bounds__(64 * kNarrowWaves, 2) void gemm_block128_narrow_kernel(
    int M, int N, int K, const uint8_t* __restrict__ A, ScaleRows sA, const uint8_t* __restrict__ B, ScaleRows sB,
    void* __restrict__ D, int64_t ldd, Epilogue ep, int tiles_m, int tiles_n, int vec_ok) {
    __shared__ v16f part[kNarrowWaves - 1][64];
    __shared__ __attribute__((aligned(16))) uint8_t stage[kNarrowWaves][2][32 * 128];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The row tiles of one column tile are launched 8 apart: the same XCD, so
    // that tile's B rows pass through one L2.  Padding workgroups exit.
    const int grp = static_cast<int>(blockIdx.x) / (8 * tiles_m);
    const int rem = static_cast<int>(blockIdx.x) - grp * 8 * tiles_m;
    const int tm = rem >> 3, tn = grp * 8 + (rem & 7);
    if (tn >= tiles_n) return;
    const int m0 = tm * 32, n0 = tn * 32;
    const int nkb = (K + 127) >> 7;
    const int per = (nkb + kNarrowWaves - 1) / kNarrowWaves;
    const int c0 = min(wave * per, nkb), c1 = min(c0 + per, nkb);

    const int rows_a = min(32, M - m0), rows_b = min(32, N - n0);
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(A) + static_cast<int64_t>(m0) * K, 0, rows_a * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(B) + static_cast<int64_t>(n0) * K, 0, rows_b * K, 0x00020000);
    const int r = lane & 31, h = lane >> 5;
    const int64_t ra = min(m0 + r, M - 1) >> sA.shift, rb = min(n0 + r, N - 1) >> sB.shift;
    const int lr = lane >> 3, lg = lane & 7;
    uint8_t* st_a = stage[wave][0];
    uint8_t* st_b = stage[wave][1];
    u32x4 ga[kNarrowDepth][4], gb[kNarrowDepth][4];
    uint32_t wa[kNarrowDepth], wb[kNarrowDepth];
    auto fetch = [&](auto SLOT, int c) {
        constexpr int j = SLOT;
        const bool ok = c < c1 && 128 * c + 16 * lg < K;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = ok ? static_cast<uint32_t>((lr + 8 * i) * K + 128 * c + 16 * lg) : 0x80000000u;
            const auto a = __builtin_amdgcn_raw_buffer_load_b128(rs_a, static_cast<int>(o), 0, 0);
            const auto b = __builtin_amdgcn_raw_buffer_load_b128(rs_b, static_cast<int>(o), 0, 0);
            ga[j][i] = u32x4{a[0], a[1], a[2], a[3]};
            gb[j][i] = u32x4{b[0], b[1], b[2], b[3]};
        }
        // past the range: the word of a block that exists (its codes are zero)
        const int64_t g = min(c, nkb - 1) >> 2;
        wa[j] = sA.words[g * sA.rows + ra];
        wb[j] = sB.words[g * sB.rows + rb];
    };
    v16f acc = v16f{};
    static_for<kNarrowDepth>([&](auto J) { fetch(J, c0 + J); });
    for (int c = c0; c < c1; c += kNarrowDepth) {
        static_for<kNarrowDepth>([&](auto J) {
            constexpr int j = J;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = lr + 8 * i;
                const int pos = row * 128 + 16 * (lg ^ (row & 7));
                *reinterpret_cast<u32x4*>(st_a + pos) = ga[j][i];
                *reinterpret_cast<u32x4*>(st_b + pos) = gb[j][i];
            }
            // a block past the range holds zero codes; a unit scale keeps them
            // zero whatever the byte is
            const bool in = c + j < c1;
            const int sh = ((c + j) & 3) * 8;
            const uint32_t sa = in ? (wa[j] >> sh) & 255u : 127u, sb = in ? (wb[j] >> sh) & 255u : 127u;
            fetch(J, c + j + kNarrowDepth);
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
    for (int w = 0; w < kNarrowWaves - 1; ++w) {
        const v16f q = part[w][lane];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] += q[e];
    }
    // lane (r, h) holds row m0 + r, columns n0 + 8 q + 4 h + e in acc[4 q + e]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float a4[4] = {acc[4 * q + 0], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
        finish_row_chunk<OUT, 4>(D, ldd, ep, m0 + r, n0 + 8 * q + 4 * h, M, N, vec_ok, a4);
    }
}

template <int AF, int BF, int OUT>
hipError_t launch_out(int64_t M, int64_t N, int64_t K, const uint8_t* a, const ScaleRows& sa, const uint8_t* b,
                      const ScaleRows& sb, void* d, int64_t ldd, const Epilogue& ep, hipStream_t stream) {
    const int vec = vec16_ok(OUT, d, ldd, ep);
    const int Mi = static_cast<int>(M), Ni = static_cast<int>(N), Ki = static_cast<int>(K);
    const int tm = static_cast<int>((M + 31) / 32), tn = static_cast<int>((N + 31) / 32);
    const uint32_t wgs = static_cast<uint32_t>((tn + 7) / 8) * 8u * static_cast<uint32_t>(tm);
    hipLaunchKernelGGL((gemm_block128_narrow_kernel<AF, BF, OUT>), dim3(wgs), dim3(64 * kNarrowWaves), 0, stream, Mi,
                       Ni, Ki, a, sa, b, sb, d, ldd, ep, tm, tn, vec);
    return hipGetLastError();
}

template <int AF, int BF>
hipError_t launch_typed(int64_t M, int64_t N, int64_t K, const uint8_t* a, const ScaleRows& sa, const uint8_t* b,
                        const ScaleRows& sb, int out, void* d, int64_t ldd, const Epilogue& ep, hipStream_t stream) {
    if (out == BSFP8_OUT_F32) return launch_out<AF, BF, BSFP8_OUT_F32>(M, N, K, a, sa, b, sb, d, ldd, ep, stream);
    if (out == BSFP8_OUT_BF16) return launch_out<AF, BF, BSFP8_OUT_BF16>(M, N, K, a, sa, b, sb, d, ldd, ep, stream);
    return launch_out<AF, BF, BSFP8_OUT_F16>(M, N, K, a, sa, b, sb, d, ldd, ep, stream);
}

// Which form is the quickest, from what each one's parts were measured to take
// (microseconds on MI355X): a tiled form runs ceil(tiles / 256) tiles one after
// another on the fullest CU, each `stage` per 128 K and `tile` besides; large tiles
// move fewer bytes per product, small ones fill the chip.  The narrow form splits
// K over a workgroup's waves and moves 64 bytes per K and 32 x 32 tile at up to
// 19 TB/s.  Examples (16-bit / FP32 output, us; narrow, 128 x 128, 192 x 128,
// 256 x 128, 256 x 256): 256 x 4096 x 4096: 16.5, 17.3, 20.4, 23.3, 37.5;
// 1111 x 4000 x 4064: 95, 39, 28.3, 32.4, 43.8; 2048 x 4096 x 4096: 147, 33.7,
// 44.6, 32.9, 43.5; 1024 x 14336 x 4096: 187, 60, 65, 55.7, 48.6; FP32
// 1024 x 1024 x 16384: 75, 101, 131, 163, 282.  `stage` and `tile` come from one
// round; over several they are low: 1700 x 14336 x 4096 (four of 192 x 128) is put
// at 87 and takes 109, 4608 x 12288 x 4096 (seven of 256 x 128) 186 and 205.
int choose_form(int64_t M, int64_t N, int64_t K, int out) {
    struct Cost { int rows_a, rows_b; double stage, stage_f32, tile; };
    static constexpr Cost kCost[4] = {
        {256, 256, 1.35, 3.05, 8.0}, {256, 128, 0.72, 1e9, 3.0}, {192, 128, 0.60, 1.55, 1.5}, {128, 128, 0.515, 1.0, 0.0}};
    const double stages = static_cast<double>((K + 127) / 128);
    // one workgroup per tile: only as many as a launch takes (2^32 threads)
    constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;
    const int64_t narrow_tiles = ((M + 31) / 32) * (((N + 31) / 32 + 7) / 8 * 8);
    double best = 4.0 + static_cast<double>(narrow_tiles) * static_cast<double>(K) * 64.0 / (out == BSFP8_OUT_F32 ? 14.0e6 : 19.0e6);
    if (narrow_tiles > kMaxGroups) best = 1e300;
    int form = 4;
    for (int i = 0; i < 4; ++i) {
        const int64_t tiles = ((M + kCost[i].rows_a - 1) / kCost[i].rows_a) * ((N + kCost[i].rows_b - 1) / kCost[i].rows_b);
        if (i == 3 && tiles > kMaxGroups) continue;
        const double rounds = static_cast<double>((tiles + 255) / 256);
        const double t = 4.0 + rounds * (stages * (out == BSFP8_OUT_F32 ? kCost[i].stage_f32 : kCost[i].stage) + kCost[i].tile);
        if (t < best) {
            best = t;
            form = i;
        }
    }
    return form;
}

ScaleRows scale_rows(const uint8_t* s, int64_t rows, int block_rows) {
    return {reinterpret_cast<const uint32_t*>(s), block_rows == 128 ? (rows + 127) / 128 : rows,
            block_rows == 128 ? 7 : 0};
}

}  // namespace

hipError_t launch_gemm_block128(int64_t M, int64_t N, int64_t K, int a_fmt, const uint8_t* a, const uint8_t* a_scales,
                                int a_block_rows, int b_fmt, const uint8_t* b, const uint8_t* b_scales,
                                int b_block_rows, int out, void* d, int64_t ldd, const Epilogue& ep,
                                hipStream_t stream) {
    const ScaleRows sa = scale_rows(a_scales, M, a_block_rows), sb = scale_rows(b_scales, N, b_block_rows);
    const TileArgs t{M, N, K, a_fmt, a, sa, b_fmt, b, sb, out, d, ldd, ep, stream};
    if (M <= kRowsMaxM && N <= kRowsMaxN) return launch_gemm_block128_rows(t);
    switch (choose_form(M, N, K, out)) {
    case 0: return launch_gemm_block128_4x4(t);
    case 1: return launch_gemm_block128_4x2(t);
    case 2: return launch_gemm_block128_3x2(t);
    case 3: return launch_gemm_block128_2x2(t);
    default: break;
    }
    if (a_fmt == BSFP8_E4M3 && b_fmt == BSFP8_E4M3)
        return launch_typed<BSFP8_E4M3, BSFP8_E4M3>(M, N, K, a, sa, b, sb, out, d, ldd, ep, stream);
    if (a_fmt == BSFP8_E4M3)
        return launch_typed<BSFP8_E4M3, BSFP8_E5M2>(M, N, K, a, sa, b, sb, out, d, ldd, ep, stream);
    if (b_fmt == BSFP8_E4M3)
        return launch_typed<BSFP8_E5M2, BSFP8_E4M3>(M, N, K, a, sa, b, sb, out, d, ldd, ep, stream);
    return launch_typed<BSFP8_E5M2, BSFP8_E5M2>(M, N, K, a, sa, b, sb, out, d, ldd, ep, stream);
}

}  // namespace bsfp8
