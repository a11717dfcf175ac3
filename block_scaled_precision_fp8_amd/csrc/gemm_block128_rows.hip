// gemm_block128_rows.hip -- the block-of-128 FP8 GEMM for up to 16 rows of A
// (decoded tokens) and few columns: bound by streaming B once.
//
// A workgroup computes 16 columns of D.  Its waves take groups of four K blocks
// (512 K, one scale word per row) in turn, load them straight into the MFMA
// layout, all of a group's loads in flight at once, and add their partial sums
// in LDS in the order of the waves.  With K spread over up to 16 waves and 16
// columns per workgroup, few columns still occupy many CUs: with weights from
// HBM 1 x 1024 x 4096 takes 4.9 us against 6.8 by the narrow form (32 columns
// per workgroup, 4 waves), 16 x 2048 x 8192 10.6 against 13.0,
// 16 x 4096 x 14336 19.3 against 23.2.  From about 5000 columns on the narrow
// form fills the chip too and its whole-line loads win: 16 x 6144 x 4096 11.5
// against 10.3, 16 x 8192 x 8192 21.5 against 17.1.  Several 16-row tiles of A
// per workgroup were slower than the narrow form at every size tried.
// v_mfma_scale_f32_16x16x128_f8f6f4 covers one K block; lane (r = l % 16,
// q = l / 16) of an operand supplies 32 of row r's 128 codes, and since they
// share their scale any split of them works that is the same on both sides:
// bytes 16 q .. and 64 + 16 q .., so that a load instruction reads 64
// consecutive bytes of each of 16 rows and its twin the rest of the lines.
#include "gemm_block128.h"

namespace bsfp8 {

namespace {

using namespace big_tile;
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kMaxWaves = 16;

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

template <int AF, int BF, int OUT>
__global__ __launch_bounds__(64 * kMaxWaves) void gemm_block128_rows_kernel(
    int M, int N, int K, const uint8_t* __restrict__ A, ScaleRows sA, const uint8_t* __restrict__ B, ScaleRows sB,
    void* __restrict__ D, int64_t ldd, Epilogue ep, int vec_ok) {
    __shared__ v4f part[kMaxWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * 16;
    const int r = lane & 15, q = lane >> 4;
    const int nkb = (K + 127) >> 7, ngr = (nkb + 3) >> 2;

    // rows of B from n0 on, all of A: range-checked loads, zeros past the edge
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(B) + static_cast<int64_t>(n0) * K, 0, min(16, N - n0) * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(A), 0, M * K, 0x00020000);
    const int64_t sra = min(r, M - 1) >> sA.shift, srb = min(n0 + r, N - 1) >> sB.shift;
    const uint32_t used = (nkb & 3) ? (1u << (8 * (nkb & 3))) - 1u : 0xFFFFFFFFu;

    // piece p (0..7) of a group: half p & 1 of K block p / 2 of row r
    auto piece = [&](const __amdgpu_buffer_rsrc_t& rs, int g, int p) {
        const int k = g * 512 + (p >> 1) * 128 + (p & 1) * 64 + q * 16;
        const auto w = __builtin_amdgcn_raw_buffer_load_b128(rs, k < K ? r * K + k : static_cast<int>(0x80000000u), 0, 0);
        return u32x4{w[0], w[1], w[2], w[3]};
    };
    v4f acc = v4f{};
    for (int g = wave; g < ngr; g += waves) {
        u32x4 a[8], b[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            b[p] = piece(rs_b, g, p);
            a[p] = piece(rs_a, g, p);
        }
        // unused bytes of the last word: their codes are zero, a unit scale keeps them so
        const uint32_t keep = g == ngr - 1 ? used : 0xFFFFFFFFu;
        const uint32_t wa = (sA.words[g * sA.rows + sra] & keep) | (0x7F7F7F7Fu & ~keep);
        const uint32_t wb = (sB.words[g * sB.rows + srb] & keep) | (0x7F7F7F7Fu & ~keep);
        // every load is issued before the first product waits for one
        __builtin_amdgcn_sched_barrier(0);
        static_for<4>([&](auto J) {
            constexpr int j = J;
            acc = block_product<AF, BF, OUT, j>(b[2 * j], b[2 * j + 1], a[2 * j], a[2 * j + 1], wb, wa, acc);
        });
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    for (int w = 1; w < waves; ++w) acc += part[w][lane];
    // lane (r, q) holds row r, columns n0 + 4 q ..
    const float a4[4] = {acc[0], acc[1], acc[2], acc[3]};
    finish_row_chunk<OUT, 4>(D, ldd, ep, r, n0 + 4 * q, M, N, vec_ok, a4);
}

template <int AF, int BF, int OUT>
hipError_t launch_out(const TileArgs& t) {
    const int ngr = static_cast<int>((t.K + 511) / 512);
    const int rounds = (ngr + kMaxWaves - 1) / kMaxWaves, waves = (ngr + rounds - 1) / rounds;
    hipLaunchKernelGGL((gemm_block128_rows_kernel<AF, BF, OUT>), dim3(static_cast<uint32_t>((t.N + 15) / 16)),
                       dim3(64 * waves), 0, t.stream, static_cast<int>(t.M), static_cast<int>(t.N),
                       static_cast<int>(t.K), t.a, t.sa, t.b, t.sb, t.d, t.ldd, t.ep, vec16_ok(OUT, t.d, t.ldd, t.ep));
    return hipGetLastError();
}

template <int AF, int BF>
hipError_t launch_typed(const TileArgs& t) {
    if (t.out == BSFP8_OUT_F32) return launch_out<AF, BF, BSFP8_OUT_F32>(t);
    if (t.out == BSFP8_OUT_BF16) return launch_out<AF, BF, BSFP8_OUT_BF16>(t);
    return launch_out<AF, BF, BSFP8_OUT_F16>(t);
}

}  // namespace

hipError_t launch_gemm_block128_rows(const TileArgs& t) {
    if (t.a_fmt == BSFP8_E4M3)
        return t.b_fmt == BSFP8_E4M3 ? launch_typed<BSFP8_E4M3, BSFP8_E4M3>(t) : launch_typed<BSFP8_E4M3, BSFP8_E5M2>(t);
    return t.b_fmt == BSFP8_E4M3 ? launch_typed<BSFP8_E5M2, BSFP8_E4M3>(t) : launch_typed<BSFP8_E5M2, BSFP8_E5M2>(t);
}

}  // namespace bsfp8
