// gemm_block128_big.hip -- the 256 x 256-tile form of the block-of-128 FP8 GEMM (gfx950).
//
// One workgroup per CU, four waves of 128 x 128 (4 x 4 MFMA tiles of 32 x 32,
// 256 FP32 accumulators per lane in the accumulation registers).  K advances in
// stages of 128, one scale block: 256 rows x 128 bytes of A and of B (64 KB) by
// direct global-to-LDS loads of whole 128-byte lines, in two buffers.  The
// scale words of four stages (512 rows x 4 bytes) come the same way, a group
// ahead.  The main loop is volatile inline assembly, so that loads, fragment
// reads and MFMAs interleave in program order; the waits are explicit.
//
// 16-bit outputs: v_mfma_scale_f32_32x32x64_f8f6f4 with the rows' E8M0 bytes,
// two steps of 64 K per stage.  FP32 output: the codes, times their scale, are
// widened to bf16 (exact) a quarter step ahead of their MFMAs
// (v_mfma_f32_32x32x16_bf16, 24 fraction bits instead of 13), between the MFMAs
// of the quarter before.
#include "gemm_block128.h"

namespace bsfp8 {

namespace {

using namespace big_tile;
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kThreads = 256;
constexpr int kRowBytes = 128;
constexpr int kOperandBytes = 256 * kRowBytes;        // 32 KB
constexpr int kStageBytes = 2 * kOperandBytes;        // 64 KB
constexpr int kScaleLds = 2 * kStageBytes;            // two groups of 512 words after the stages
constexpr int kScaleGroupBytes = 512 * 4;
constexpr int kLdsBytes = kScaleLds + 2 * kScaleGroupBytes;

template <int OFF>
__device__ __forceinline__ void lds_read4(uint32_t& v, uint32_t addr) {
    asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
}

// acc += x^T y over 64 K values, byte SEL of each scale word.
template <int SEL, int CB, int BG>
__device__ __forceinline__ void mfma_scaled(v16f& acc, const u32x8& x, const u32x8& y, uint32_t sx, uint32_t sy) {
    asm volatile(
        "v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%5,0] op_sel_hi:[%6,%6,0] cbsz:%7 blgp:%8"
        : "+a"(acc)
        : "v"(x), "v"(y), "v"(sx), "v"(sy), "i"(SEL & 1), "i"(SEL >> 1), "i"(CB), "i"(BG));
}
__device__ __forceinline__ void mfma_bf16_k16(v16f& acc, const u32x4& x, const u32x4& y) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(x), "v"(y));
}
// Two codes (half HI of w) times the scale s -> two bf16, in place in the stream.
template <int FMT, int HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w, float s) {
    uint32_t d;
    if constexpr (FMT == BSFP8_E4M3) {
        if constexpr (HI) asm volatile("v_cvt_scalef32_pk_bf16_fp8 %0, %1, %2 op_sel:[1,0,0]" : "=v"(d) : "v"(w), "v"(s));
        else asm volatile("v_cvt_scalef32_pk_bf16_fp8 %0, %1, %2" : "=v"(d) : "v"(w), "v"(s));
    } else {
        if constexpr (HI) asm volatile("v_cvt_scalef32_pk_bf16_bf8 %0, %1, %2 op_sel:[1,0,0]" : "=v"(d) : "v"(w), "v"(s));
        else asm volatile("v_cvt_scalef32_pk_bf16_bf8 %0, %1, %2" : "=v"(d) : "v"(w), "v"(s));
    }
    return d;
}

template <int AF, int BF, int OUT, bool STAGE16>
__global__ __launch_bounds__(kThreads, 1) void gemm_block128_big_kernel(
    int M, int N, int K, const uint8_t* __restrict__ A, ScaleRows sA, const uint8_t* __restrict__ B, ScaleRows sB,
    void* __restrict__ D, int64_t ldd, Epilogue ep, int tiles_m, int tiles_n, int vec_ok) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLdsBytes];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1;
    const int wn = wave >> 1;
    int tm, tn;
    map_tile(blockIdx.x, tiles_m, tiles_n, 8, &tm, &tn);
    const int m0 = tm * 256;
    const int n0 = tn * 256;
    const int nst = (K + 127) >> 7;
    const int ngr = (nst + 3) >> 2;

    // The resources start at the tile's first row and end after its last row
    // inside the matrix: rows past the edge read as zero, offsets stay below
    // 256 K < 2^31.
    const int rows_a = min(256, M - m0);
    const int rows_b = min(256, N - n0);
    const __amdgpu_buffer_rsrc_t rs_a = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(A) + static_cast<int64_t>(m0) * K, 0, rows_a * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs_b = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(B) + static_cast<int64_t>(n0) * K, 0, rows_b * K, 0x00020000);

    // Direct loads: load j (0..15) of wave w fills rows 8 g .. 8 g + 7 of operand
    // j & 1 (A, B), g = 4 (j >> 1) + w.  Lane l brings row 8 g + l / 8 and the
    // chunk that belongs at position l % 8: chunk c of row R sits at
    // c ^ ((R >> 1) & 7).  Chunks and stages past K are given an out-of-range
    // offset and read as zero.
    const int drow = lane >> 3;
    const int dchunk = (lane & 7) ^ (((8 * wave + drow) >> 1) & 7);
    const uint32_t dma_row = static_cast<uint32_t>((8 * wave + drow) * K + dchunk * 16);
    const uint32_t dma_grp = static_cast<uint32_t>(32 * K);
    auto dma_one = [&](auto J, int stage, auto BUF) {
        constexpr int j = J;
        constexpr int buf = BUF;
        constexpr int gi = j >> 1;
        const uint32_t vo = stage * 128 + dchunk * 16 < K ? dma_row + gi * dma_grp : 0x80000000u;
        lds_void* dst = (lds_void*)(lds + buf * kStageBytes + (j & 1) * kOperandBytes + (4 * gi + wave) * 1024);
        if constexpr ((j & 1) == 0)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, dst, 16, vo, stage * 128, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, dst, 16, vo, stage * 128, 0, 0);
    };
    // Scale words of a group: this wave's 64 rows of A (q = 0) or B (q = 1);
    // rows past the edge and groups past the end take one that exists.
    const int64_t sra = min(m0 + 64 * wave + lane, M - 1) >> sA.shift;
    const int64_t srb = min(n0 + 64 * wave + lane, N - 1) >> sB.shift;
    auto scale_dma = [&](int group, int q) {
        const int g = min(group, ngr - 1);
        const uint32_t* src = q == 0 ? sA.words + g * sA.rows + sra : sB.words + g * sB.rows + srb;
        lds_void* dst = (lds_void*)(lds + kScaleLds + (group & 1) * kScaleGroupBytes + q * 1024 + wave * 256);
        __builtin_amdgcn_global_load_lds(src, dst, 4, 0, 0);
    };

    // Fragment reads of step ks: lane (frag_row r, half h) reads chunks 4 ks + h
    // and 4 ks + 2 + h of rows wm 128 + 32 t + r (A), wn 128 + 32 t + r (B).
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_byte*)lds));
    const int frag_row = lane & 31;
    const int half = lane >> 5;
    const int sw = (frag_row >> 1) & 7;
    uint32_t rd_a[2][2][2], rd_b[2][2][2];       // [buffer][ks][low, high chunk]
#pragma unroll
    for (int bf = 0; bf < 2; ++bf)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t pos = static_cast<uint32_t>(((4 * ks + 2 * q + half) ^ sw) * 16);
                rd_a[bf][ks][q] = lds0 + bf * kStageBytes + (wm * 128 + frag_row) * kRowBytes + pos;
                rd_b[bf][ks][q] = lds0 + bf * kStageBytes + kOperandBytes + (wn * 128 + frag_row) * kRowBytes + pos;
            }

    v16f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v16f{};

    struct Frag { u32x4 xl[4], xh[4], yl[4], yh[4]; };
    Frag fr[2];
    // read piece R (0..15) of step KS of the stage in buffer BUF
    auto read_one = [&](auto R, Frag& dst, auto BUF, auto KS) {
        constexpr int r = R;
        constexpr int t = r >> 2;
        constexpr int which = r & 3;
        constexpr int off = t * 32 * kRowBytes;
        if constexpr (which == 0) lds_read16<off>(dst.xl[t], rd_b[BUF][KS][0]);
        if constexpr (which == 1) lds_read16<off>(dst.xh[t], rd_b[BUF][KS][1]);
        if constexpr (which == 2) lds_read16<off>(dst.yl[t], rd_a[BUF][KS][0]);
        if constexpr (which == 3) lds_read16<off>(dst.yh[t], rd_a[BUF][KS][1]);
    };
    // the scale words of this lane's rows: nxt as read from LDS, cur in use
    uint32_t nxt[8], cur[8];
    const uint32_t srd_a = lds0 + kScaleLds + (wm * 128 + frag_row) * 4;
    const uint32_t srd_b = lds0 + kScaleLds + 1024 + (wn * 128 + frag_row) * 4;
    auto read_scale = [&](auto T, int group) {
        constexpr int t = T;
        const uint32_t o = (group & 1) * kScaleGroupBytes;
        if constexpr (t < 4) lds_read4<t * 128>(nxt[t], srd_a + o);
        else lds_read4<(t - 4) * 128>(nxt[t], srd_b + o);
    };
    // bytes past the last K block (their codes are zero) become a unit scale
    const uint32_t used = (nst & 3) ? (1u << (8 * (nst & 3))) - 1u : 0xFFFFFFFFu;
    auto take_scales = [&](int group) {
        const uint32_t keep = group == ngr - 1 ? used : 0xFFFFFFFFu;
#pragma unroll
        for (int t = 0; t < 8; ++t) cur[t] = (nxt[t] & keep) | (0x7F7F7F7Fu & ~keep);
        // VALU writes settle before an MFMA of the assembly reads them
        asm volatile("s_nop 4" : "+v"(cur[0]), "+v"(cur[1]), "+v"(cur[2]), "+v"(cur[3]), "+v"(cur[4]), "+v"(cur[5]),
                                 "+v"(cur[6]), "+v"(cur[7]));
    };

    constexpr auto C0 = std::integral_constant<int, 0>{};
    constexpr auto C1 = std::integral_constant<int, 1>{};

    // Prologue: stage 0, the first two scale groups and stage 1 on their way.
    static_for<16>([&](auto J) { dma_one(J, 0, C0); });
    scale_dma(0, 0);
    scale_dma(0, 1);
    static_for<16>([&](auto J) { dma_one(J, 1, C1); });
    asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
    lds_wait_barrier();
    static_for<16>([&](auto R) { read_one(R, fr[0], C0, C0); });
    static_for<8>([&](auto T) { read_scale(T, 0); });
    lds_wait();
    take_scales(0);

    // One K step on fragment set KS: MFMAs, with the next step's fragment reads
    // in their shadows.  Step 1 follows the barrier that publishes stage s + 1
    // and frees this stage's buffer: it reads stage s + 1's first fragments and
    // issues the direct loads of stage s + 2, one per MFMA.
    auto kstep = [&](int s, auto CB_, auto KS, auto U) {
        constexpr int cb = CB_;
        constexpr int ks = KS;
        constexpr int u = U;                  // stage within its scale group
        const Frag& f = fr[ks];
        Frag& g = fr[ks ^ 1];
        constexpr auto rbuf = std::integral_constant<int, ks == 1 ? (cb ^ 1) : cb>{};
        constexpr auto rks = std::integral_constant<int, ks ^ 1>{};
        static_for<16>([&](auto J) {
            constexpr int j = J;
            constexpr int ti = j >> 2, tj = j & 3;
            const u32x8 x = __builtin_shufflevector(f.xl[ti], f.xh[ti], 0, 1, 2, 3, 4, 5, 6, 7);
            const u32x8 y = __builtin_shufflevector(f.yl[tj], f.yh[tj], 0, 1, 2, 3, 4, 5, 6, 7);
            mfma_scaled<u, mfma_fmt<BF>(), mfma_fmt<AF>()>(acc[ti][tj], x, y, cur[4 + ti], cur[tj]);
            read_one(J, g, rbuf, rks);
            if constexpr (ks == 1) {
                dma_one(J, s + 2, CB_);
                if constexpr (u == 3 && j < 8) read_scale(J, (s >> 2) + 1);
                if constexpr (u == 0 && j == 8) scale_dma((s >> 2) + 1, 0);
                if constexpr (u == 0 && j == 9) scale_dma((s >> 2) + 1, 1);
            }
        });
    };
    auto run_stage = [&](int s, auto U) {
        constexpr auto cb = std::integral_constant<int, U & 1>{};
        lds_wait();
        if constexpr (U == 0) {
            if (s > 0) take_scales(s >> 2);
        }
        kstep(s, cb, C0, U);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_wait_barrier();
        kstep(s, cb, C1, U);
    };
    for (int s = 0; s < nst; s += 4) {
        run_stage(s, C0);
        if (s + 1 < nst) run_stage(s + 1, C1);
        if (s + 2 < nst) run_stage(s + 2, std::integral_constant<int, 2>{});
        if (s + 3 < nst) run_stage(s + 3, std::integral_constant<int, 3>{});
    }
    // no direct load may still be writing LDS when the epilogue reuses it, and
    // the last step's reads, which have no consumer, are named after the wait
    // so that their registers are not reused while in flight
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        asm volatile("" :: "v"(fr[q].xl[0]), "v"(fr[q].xl[1]), "v"(fr[q].xl[2]), "v"(fr[q].xl[3]),
                           "v"(fr[q].xh[0]), "v"(fr[q].xh[1]), "v"(fr[q].xh[2]), "v"(fr[q].xh[3]));
        asm volatile("" :: "v"(fr[q].yl[0]), "v"(fr[q].yl[1]), "v"(fr[q].yl[2]), "v"(fr[q].yl[3]),
                           "v"(fr[q].yh[0]), "v"(fr[q].yh[1]), "v"(fr[q].yh[2]), "v"(fr[q].yh[3]));
    }
    asm volatile("" :: "v"(nxt[0]), "v"(nxt[1]), "v"(nxt[2]), "v"(nxt[3]), "v"(nxt[4]), "v"(nxt[5]), "v"(nxt[6]),
                       "v"(nxt[7]));
    // MFMA results must settle before the accumulation registers are read
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7"
                 : "+a"(acc[0][0]), "+a"(acc[0][1]), "+a"(acc[0][2]), "+a"(acc[0][3]),
                   "+a"(acc[1][0]), "+a"(acc[1][1]), "+a"(acc[1][2]), "+a"(acc[1][3]),
                   "+a"(acc[2][0]), "+a"(acc[2][1]), "+a"(acc[2][2]), "+a"(acc[2][3]),
                   "+a"(acc[3][0]), "+a"(acc[3][1]), "+a"(acc[3][2]), "+a"(acc[3][3]));
    NoScale none;
    epilogue<OUT, STAGE16>(acc, lds, wave, lane, m0, n0, M, N, D, ldd, ep, vec_ok, none);
}

template <int AF, int BF, int OUT, bool STAGE16>
hipError_t launch(int64_t M, int64_t N, int64_t K, const uint8_t* a, const ScaleRows& sa, const uint8_t* b,
                  const ScaleRows& sb, void* d, int64_t ldd, const Epilogue& ep, hipStream_t stream) {
    const int tm = static_cast<int>((M + 255) / 256), tn = static_cast<int>((N + 255) / 256);
    hipLaunchKernelGGL((gemm_block128_big_kernel<AF, BF, OUT, STAGE16>),
                       dim3(static_cast<uint32_t>(tm) * static_cast<uint32_t>(tn)), dim3(kThreads), 0, stream,
                       static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), a, sa, b, sb, d, ldd, ep, tm, tn,
                       vec16_ok(OUT, d, ldd, ep));
    return hipGetLastError();
}

template <int AF, int BF>
hipError_t launch_typed(int64_t M, int64_t N, int64_t K, const uint8_t* a, const ScaleRows& sa, const uint8_t* b,
                        const ScaleRows& sb, int out, void* d, int64_t ldd, const Epilogue& ep, hipStream_t stream) {
    if (out == BSFP8_OUT_BF16)
        return ep.beta == 0.0f
                   ? launch<AF, BF, BSFP8_OUT_BF16, true>(M, N, K, a, sa, b, sb, d, ldd, ep, stream)
                   : launch<AF, BF, BSFP8_OUT_BF16, false>(M, N, K, a, sa, b, sb, d, ldd, ep, stream);
    return ep.beta == 0.0f ? launch<AF, BF, BSFP8_OUT_F16, true>(M, N, K, a, sa, b, sb, d, ldd, ep, stream)
                           : launch<AF, BF, BSFP8_OUT_F16, false>(M, N, K, a, sa, b, sb, d, ldd, ep, stream);
}

}  // namespace

hipError_t launch_gemm_block128_big(int64_t M, int64_t N, int64_t K, int a_fmt, const uint8_t* a, const ScaleRows& sa,
                                    int b_fmt, const uint8_t* b, const ScaleRows& sb, int out, void* d, int64_t ldd,
                                    const Epilogue& ep, hipStream_t stream) {
    if (a_fmt == BSFP8_E4M3 && b_fmt == BSFP8_E4M3)
        return launch_typed<BSFP8_E4M3, BSFP8_E4M3>(M, N, K, a, sa, b, sb, out, d, ldd, ep, stream);
    if (a_fmt == BSFP8_E4M3)
        return launch_typed<BSFP8_E4M3, BSFP8_E5M2>(M, N, K, a, sa, b, sb, out, d, ldd, ep, stream);
    if (b_fmt == BSFP8_E4M3)
        return launch_typed<BSFP8_E5M2, BSFP8_E4M3>(M, N, K, a, sa, b, sb, out, d, ldd, ep, stream);
    return launch_typed<BSFP8_E5M2, BSFP8_E5M2>(M, N, K, a, sa, b, sb, out, d, ldd, ep, stream);
}

}  // namespace bsfp8
