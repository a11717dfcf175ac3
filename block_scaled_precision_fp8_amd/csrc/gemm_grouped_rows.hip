// gemm_grouped_rows.hip -- FP8 products grouped by expert, one power-of-two scale per 128
// K values (gfx950), for few rows per group:
//
//   D[i][n] = alpha sum_k A[i][k] B[e(i)][n][k] (+ beta C[i][n]),   i in group e(i).
//
// A workgroup computes 16 columns of one group's D, as gemm_block128_rows.hip does
// of a whole product: its waves take groups of four K blocks in turn, load them
// straight into the MFMA layout and add their partial sums in LDS in the order of the
// waves.  It needs no more of the offsets than its group's two, and a group without
// rows costs a load of them.
#include "gemm_grouped.h"

namespace bsfp8 {

namespace {

using namespace big_tile;

constexpr int kMaxWaves = 16;
// A launch's threads are counted in 32 bits: workgroups of 1024.  (Only products without K values, which the
// choice of forms does not see, have more tiles: up to 2^27.)
constexpr int64_t kMostGroups = (int64_t(1) << 22) - 1;

template <int AF, int BF, int OUT>
__global__ __launch_bounds__(64 * kMaxWaves) void gemm_grouped_rows_kernel(
    int M, int N, int K, const int32_t* __restrict__ offsets, const uint8_t* __restrict__ A, ScaleRows sA,
    const uint8_t* __restrict__ B, ScaleRows sB, void* __restrict__ D, int64_t ldd, Epilogue ep, int tiles_n, int tiles) {
    __shared__ v4f part[kMaxWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const int nkb = (K + 127) >> 7, ngr = (nkb + 3) >> 2;
    const uint32_t used = (nkb & 3) ? (1u << (8 * (nkb & 3))) - 1u : 0xFFFFFFFFu;

    // (more than one only where there are more than a launch can count)
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int e = tile / tiles_n, n0 = (tile - e * tiles_n) * 16;
        const int first = min(max(offsets[e], 0), M), end = min(max(offsets[e + 1], first), M);
        // rows of B from n0 on: range-checked loads, zeros past the edge
        const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(B) + (static_cast<int64_t>(e) * N + n0) * K, 0, min(16, N - n0) * K, 0x00020000);
        const uint32_t* words_b = sB.words + static_cast<int64_t>(e) * ngr * sB.rows + (min(n0 + r, N - 1) >> sB.shift);
        // piece p (0..7) of a group of K blocks: half p & 1 of K block p / 2 of row r
        auto piece = [&](const __amdgpu_buffer_rsrc_t& rs, int g, int p) {
            const int k = g * 512 + (p >> 1) * 128 + (p & 1) * 64 + q * 16;
            const auto w = __builtin_amdgcn_raw_buffer_load_b128(rs, k < K ? r * K + k : static_cast<int>(0x80000000u), 0, 0);
            return u32x4{w[0], w[1], w[2], w[3]};
        };
        for (int m0 = first; m0 < end; m0 += 16) {
            const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t*>(A) + static_cast<int64_t>(m0) * K, 0, min(16, end - m0) * K, 0x00020000);
            const int64_t sra = min(m0 + r, end - 1);
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
                const uint32_t wb = (words_b[g * sB.rows] & keep) | (0x7F7F7F7Fu & ~keep);
                // every load is issued before the first product waits for one
                __builtin_amdgcn_sched_barrier(0);
                static_for<4>([&](auto J) {
                    constexpr int j = J;
                    acc = block_product<AF, BF, OUT, j>(b[2 * j], b[2 * j + 1], a[2 * j], a[2 * j + 1], wb, wa, acc);
                });
            }
            // A matrix instruction's result may be read some cycles after its issue only.  This compiler leaves those
            // out behind a loop that may be skipped: the first of each four columns came out wrong.
            asm volatile("s_nop 15" : "+v"(acc));
            part[wave][lane] = acc;
            __syncthreads();
            if (wave == 0) {
                for (int w = 1; w < waves; ++w) acc += part[w][lane];
                // lane (r, q) holds row r, columns n0 + 4 q ..
                finish_chunk<OUT>(D, ldd, ep, m0 + r, n0 + 4 * q, end, N, make_float4(acc[0], acc[1], acc[2], acc[3]));
            }
            __syncthreads();
        }
    }
}

template <int AF, int BF, int OUT>
hipError_t launch_out(const GroupedArgs& t) {
    const int ngr = static_cast<int>((t.K + 511) / 512);
    const int rounds = (ngr + kMaxWaves - 1) / kMaxWaves, waves = rounds ? (ngr + rounds - 1) / rounds : 1;
    const int64_t tn = (t.N + 15) / 16, tiles = tn * t.groups;
    hipLaunchKernelGGL((gemm_grouped_rows_kernel<AF, BF, OUT>), dim3(static_cast<uint32_t>(tiles < kMostGroups ? tiles : kMostGroups)),
                       dim3(64 * waves), 0, t.stream, static_cast<int>(t.M), static_cast<int>(t.N),
                       static_cast<int>(t.K), t.offsets, t.a, t.sa, t.b, t.sb, t.d, t.ldd, t.ep,
                       static_cast<int>(tn), static_cast<int>(tiles));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_grouped_rows(const GroupedArgs& t) {
    return by_type(t, [](auto AF, auto BF, auto OUT, const GroupedArgs& g) { return launch_out<AF, BF, OUT>(g); });
}

}  // namespace bsfp8
