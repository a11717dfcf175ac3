// gemm_block128_tile.h -- the tiled forms of the block-of-128 FP8 GEMM (gfx950).
//
// A workgroup of four waves (2 x 2) computes tiles of 64 TA x 64 TB outputs,
// each wave TA x TB MFMA tiles of 32 x 32.  K advances in stages of 128, one
// scale block: the tile's rows x 128 bytes of A and of B come by direct
// global-to-LDS loads of whole 128-byte lines into one of two buffers; the scale
// words of four stages come the same way, a group ahead.  The main loop is
// volatile inline assembly, so that loads, fragment reads and MFMAs interleave
// in program order; the waits are explicit.
//
// The schedule of a stage (2 TA TB MFMA slots) is what carries the kernel: the
// fragments of its second step are read in its first slots, so that a first
// barrier can free its buffer a quarter of the way through and the loads of
// stage s + 2 can start there, spread over the rest of the stage; they have the
// whole next stage but its tail to land, until that stage's second barrier
// publishes them.  One barrier for both, with the loads behind it, measured
// 2380 (FFN 16384 x 14336 x 4096) and 2550 TFLOP/s (8192^3) against 2540 and
// 2780; finer variations of the slots changed nothing.  Buffers and scale bytes
// are compile-time (the loop body is four stages): a loop of one stage with
// addresses moved on at run time took 4% longer (FFN 696 -> 726 us), and with
// the three buffers that it allows the 192 x 128 tile got no faster (28.3, then
// 29.2 us for 1111 x 4000 x 4064).
//
// What holds the smaller tiles is their loads: 1111 x 4000 x 4096, one tile of
// 192 x 128 on each of 192 CUs, takes 25 to 27 us, 23 with the MFMAs left out and
// 17 to 20 with the direct loads left out.  A stage's 40 KB then take 0.57 us, 30
// bytes per cycle and CU at 2.4 GHz, half of what a CU can take from L2.  Code rows whose
// length is no multiple of 128 start within a line, so that a load of 128 bytes
// touches two: K = 4064 takes 31 us, 29 of them without MFMAs (36 and 36, against
// 28 and 27 for K = 4096, with operands from HBM).
//
// With more tiles than workgroups the grid is persistent: the loads run on into
// the next tile's first stages while the last ones of this tile are computed
// and written, so only the first tile of a workgroup waits for memory.
#pragma once

#include "gemm_grouped.h"

namespace bsfp8 {

namespace {

using namespace big_tile;
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kThreads = 256;
constexpr int kRowBytes = 128;
constexpr int kStripBytes = 4096;     // epilogue staging per wave

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
// Two codes (half HI of w) times the scale s -> two bf16, in program order.
template <int FMT, int HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w, float s) {
    uint32_t d;
    if constexpr (FMT == BSFP8_E4M3)
        asm volatile("v_cvt_scalef32_pk_bf16_fp8 %0, %1, %2 op_sel:[%3,0,0]" : "=v"(d) : "v"(w), "v"(s), "i"(HI));
    else
        asm volatile("v_cvt_scalef32_pk_bf16_bf8 %0, %1, %2 op_sel:[%3,0,0]" : "=v"(d) : "v"(w), "v"(s), "i"(HI));
    return d;
}

// Two FP32 values -> two bf16, round to nearest even, in one instruction.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

template <int OUT>
__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    if constexpr (OUT == BSFP8_OUT_BF16) return bf16_pair(a, b);
    else return to_half_bits<OUT>(a) | (static_cast<uint32_t>(to_half_bits<OUT>(b)) << 16);
}

template <int TA, int TB>
struct Tile {
    static constexpr int ROWS_A = 64 * TA, ROWS_B = 64 * TB;
    static constexpr int A_BYTES = ROWS_A * kRowBytes, STAGE_BYTES = A_BYTES + ROWS_B * kRowBytes;
    static constexpr int SCALE_GROUP = (ROWS_A + ROWS_B) * 4;       // words of four K blocks
    static constexpr int SCALES = 2 * STAGE_BYTES;                  // LDS offsets
    // Persistent tiles need the epilogue's strips beside the stages.  The
    // smallest tile runs two workgroups per CU instead, whose loops and
    // epilogues overlap by themselves: its strips reuse the stages.
    static constexpr bool PERSISTENT = TA * TB > 4;
    static constexpr int STRIPS = PERSISTENT ? SCALES + 2 * SCALE_GROUP : 0;
    static constexpr int LDS_BYTES = SCALES + 2 * SCALE_GROUP + (PERSISTENT ? 4 * kStripBytes : 0);
    // slots of a stage: MFMAs per step, fragment reads per step, direct loads per stage and wave
    static constexpr int NM = TA * TB, NR = 2 * (TA + TB), NL = 2 * (TA + TB);
    static constexpr int RPS = (NR + NM / 2 - 1) / (NM / 2);        // reads per slot
    static constexpr int FREE = NM / 2 - 1;                         // first barrier: after this slot
    static constexpr int READY = NM + NM / 4;                       // second barrier
    static constexpr int load_slot(int k) {
        return k < NL / 2 ? NM / 2 + k * (NM / 2) / (NL / 2) : NM + (k - NL / 2) * NM / (NL / 2);
    }
    static constexpr int newer() {                                  // loads issued before READY's wait
        int c = 0;
        for (int k = 0; k < NL; ++k) c += load_slot(k) <= READY ? 1 : 0;
        return c;
    }
    static constexpr int STORES = TA * TB * 2;                      // of the constant-count epilogue
};

// What a kernel's tiles are tiles of: one product; one product per group of rows
// (D[i] = A[i] B[e]^T); or one per group of K values (D[e] = A[:, i] B[:, i]^T over group e's i).
enum Kind { ONE, ROWS, COLUMNS };
// Where the groups' kernels keep what they read off the offsets: for ROWS a group's first row
// and first tile, for COLUMNS its first K block and first scale word, and their ends.  (Static, of
// the most groups: sized at the launch, it made the 256 x 256 tiles take half an hour to compile.)
struct Tables { int32_t at[groups::kMaxGroups + 1], of[groups::kMaxGroups + 1]; };
struct GroupsArg {
    const int32_t* offsets;
    int count;
    int64_t words, d_group, c_group;
};

// FAST: bf16 output, alpha = 1, without C, every chunk of 8 outputs whole and aligned: the
// epilogue is then a fixed number of range-checked buffer stores, so the loop
// can leave them in flight.
// (Groups' products: any alpha, 16-bit outputs without C or FP32 ones with or without, at
// any address, any N: the columns past the last whole chunk are stored beside them.)
//
// Groups' tiles are counted on the device, from the offsets, so a workgroup first
// reads those (one wave, 64 groups at a time) into a table in LDS and looks its tiles up there.
// ROWS: every tile costs the same, so each XCD takes an eighth of them in a row
// (one group's weights stay in one L2), a group's tiles in the order of map_tile.
// COLUMNS: a group's tiles cost what its rows are, so each group's are dealt over all
// XCDs, neighbours to one, and the next group's follow.  K is then the row stride of A and B;
// the K loop runs over the group's blocks, of which there may be none.
template <int AF, int BF, int OUT, int TA, int TB, bool FAST, Kind KIND = ONE>
__global__ __launch_bounds__(kThreads, (Tile<TA, TB>::PERSISTENT ? 1 : 2)) void gemm_block128_tile_kernel(
    int M, int N, int K, const uint8_t* __restrict__ A, ScaleRows sA, const uint8_t* __restrict__ B, ScaleRows sB,
    void* __restrict__ D, int64_t ldd, Epilogue ep, int tiles_m, int tiles_n, int vec_ok, GroupsArg grp) {
    using T = Tile<TA, TB>;
    constexpr bool WIDE = OUT == BSFP8_OUT_F32;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS_BYTES];
    // (not there for ONE, which has no use of it)
    __shared__ Tables tables;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1;
    const int wn = wave >> 1;
    const int tiles = tiles_m * tiles_n;

    // A tile: its first row and column, the end of the rows that are its own, its
    // group, the K blocks that hold values, and for COLUMNS the first block and scale word.
    struct Place { int m0, n0, end, e, real, block, word; };
    // its stages: pairs, so that a stage's buffer is compile-time
    auto stages = [](const Place& p) { return KIND == COLUMNS && p.real == 0 ? 2 : (p.real + 1) & ~1; };
    int share = 0, last = tiles;                     // ROWS: tiles per XCD; the tile numbers that count end here
    if constexpr (KIND != ONE) {
        if (wave == 0) {
            const int limit = KIND == ROWS ? M : static_cast<int>(min(static_cast<int64_t>(K), int64_t(1) << 30));
            groups::for_each<KIND == ROWS ? T::ROWS_A : 128>(grp.offsets, grp.count, limit, [&](const groups::Lane& g, bool in) {
                if (in) {
                    tables.at[g.e] = KIND == ROWS ? g.start : g.tile;
                    tables.of[g.e] = KIND == ROWS ? g.tile : g.word;
                    if (g.e == grp.count - 1) {
                        tables.at[grp.count] = KIND == ROWS ? g.start + g.rows : g.tile + g.tiles;
                        tables.of[grp.count] = KIND == ROWS ? g.tile + g.tiles : g.word + ((g.tiles + 3) >> 2);
                    }
                }
                return false;
            });
        }
        __syncthreads();
        if constexpr (KIND == ROWS) {
            const int total = __builtin_amdgcn_readfirstlane(tables.of[grp.count]) * tiles_n;
            share = (total + 7) >> 3;
            // this XCD's part of them, as the numbers x + 8 i of its tiles
            last = 8 * max(0, min(share, total - static_cast<int>(blockIdx.x & 7) * share));
        } else {
            share = (tiles + 7) >> 3;
            last = grp.count * 8 * share;
        }
    }
    // The tile of number t < last, or (COLUMNS) the first that exists of t, t + step, ...: its number.
    auto next_tile = [&](int t, int step) {
        if constexpr (KIND == COLUMNS)
            while (t < last && (t & 7) * share + ((t % (8 * share)) >> 3) >= tiles) t += step;
        return t;
    };
    auto locate = [&](int t) {
        Place p{};
        int tm, tn;
        p.real = (K + 127) >> 7;
        p.end = M;
        if constexpr (KIND == ONE) {
            map_tile(t, tiles_m, tiles_n, 8, &tm, &tn);
            p.m0 = tm * T::ROWS_A;
        } else if constexpr (KIND == ROWS) {
            t = (t & 7) * share + (t >> 3);
            // the group whose tiles include row tile q of all: 16 groups, then one
            const int q = t / tiles_n;
            const uint64_t far = __ballot(tables.of[min(16 * (lane + 1), grp.count)] > q);
            const int e0 = 16 * __builtin_ctzll(far);
            const uint64_t near = __ballot(tables.of[min(e0 + (lane & 15) + 1, grp.count)] > q);
            p.e = e0 + __builtin_ctzll(near);
            const int first = __builtin_amdgcn_readfirstlane(tables.of[p.e]);
            const int count = __builtin_amdgcn_readfirstlane(tables.of[p.e + 1]) - first;
            t -= first * tiles_n;
            const int g = t / (8 * tiles_n), rows = min(8, count - 8 * g), r = t - g * 8 * tiles_n;
            tm = 8 * g + r % rows;
            tn = r / rows;
            p.m0 = __builtin_amdgcn_readfirstlane(tables.at[p.e]) + tm * T::ROWS_A;
            p.end = __builtin_amdgcn_readfirstlane(tables.at[p.e + 1]);
        } else {
            p.e = t / (8 * share);
            t = (t & 7) * share + ((t - p.e * 8 * share) >> 3);
            const int g = t / (8 * tiles_n), rows = min(8, tiles_m - 8 * g), r = t - g * 8 * tiles_n;
            tm = 8 * g + r % rows;
            tn = r / rows;
            p.m0 = tm * T::ROWS_A;
            p.block = __builtin_amdgcn_readfirstlane(tables.at[p.e]);
            p.word = __builtin_amdgcn_readfirstlane(tables.of[p.e]);
            // what the buffers hold, whatever the offsets are
            const int room = static_cast<int>(min(static_cast<int64_t>((K >> 7) - p.block), 4 * (grp.words - p.word)));
            p.real = max(0, min(__builtin_amdgcn_readfirstlane(tables.at[p.e + 1]) - p.block, room));
        }
        p.n0 = tn * T::ROWS_B;
        return p;
    };
    Place here;
    int tile = next_tile(blockIdx.x, gridDim.x);
    if (KIND != ONE && tile >= last) return;
    here = locate(tile);

    // The loader: two stages ahead of the MFMAs, running on into the next tile.
    // The resources start at the tile's first row and end after its last row
    // inside the matrix: rows past the edge read as zero (all of them past the
    // last tile), offsets stay below 256 K < 2^31.
    int l_tile = tile, l_stage = 0, l_stages = stages(here), l_span = K;
    __amdgpu_buffer_rsrc_t rs_a, rs_b;
    auto aim = [&](const Place& p, bool any) {
        const uint8_t* pa = A + static_cast<int64_t>(p.m0) * K;
        const uint8_t* pb = B + static_cast<int64_t>(p.n0) * K;
        int size_a = min(T::ROWS_A, p.end - p.m0) * K, size_b = min(T::ROWS_B, N - p.n0) * K;
        if constexpr (KIND == ROWS) pb += static_cast<int64_t>(p.e) * N * K;
        if constexpr (KIND == COLUMNS) {
            // the group's part of the last row ends them
            l_span = 128 * p.real;
            pa += static_cast<int64_t>(p.block) * 128;
            pb += static_cast<int64_t>(p.block) * 128;
            size_a += l_span - K;
            size_b += l_span - K;
            any = any && l_span > 0;
        }
        rs_a = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pa), 0, any ? size_a : 0, 0x00020000);
        rs_b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pb), 0, any ? size_b : 0, 0x00020000);
    };
    auto advance = [&]() {
        if (++l_stage == l_stages) {
            l_stage = 0;
            // the search and the lookup are the compiler's code, which may move what it takes as
            // written: no fragment may still be on its way to a register
            lds_wait();
            l_tile = next_tile(l_tile + gridDim.x, gridDim.x);
            const bool any = l_tile < last;
            Place p{};
            if (any) p = locate(l_tile);
            if constexpr (KIND == COLUMNS) l_stages = stages(p);
            aim(p, any);
        }
    };
    // Direct load j of wave w fills rows 8 g .. 8 g + 7 of A (j < 2 TA) or B,
    // g = 4 (j or j - 2 TA) + w.  Lane l brings row 8 g + l / 8 and the chunk that
    // belongs at position l % 8: chunk c of row R sits at c ^ ((R >> 1) & 7).
    // Chunks past K are given an out-of-range offset and read as zero.
    const int drow = lane >> 3;
    const int dchunk = (lane & 7) ^ (((8 * wave + drow) >> 1) & 7);
    const uint32_t dma_row = static_cast<uint32_t>((8 * wave + drow) * K + dchunk * 16);
    const uint32_t dma_grp = static_cast<uint32_t>(32 * K);
    auto dma_one = [&](auto J, auto BUF) {
        constexpr int j = J;
        constexpr int buf = BUF;
        // A and B in turn as long as both have loads left
        constexpr int both = 4 * (TA < TB ? TA : TB);
        constexpr bool is_a = j < both ? (j & 1) == 0 : TA > TB;
        constexpr int gi = j < both ? j >> 1 : j - both / 2;
        const uint32_t vo = l_stage * 128 + dchunk * 16 < (KIND == COLUMNS ? l_span : K) ? dma_row + gi * dma_grp : 0x80000000u;
        lds_void* dst = (lds_void*)(lds + buf * T::STAGE_BYTES + (is_a ? 0 : T::A_BYTES) + (4 * gi + wave) * 1024);
        if constexpr (is_a)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, dst, 16, vo, l_stage * 128, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, dst, 16, vo, l_stage * 128, 0, 0);
    };
    // Scale words of a group of K blocks of a tile: wave w brings rows
    // 16 TA w .. of A (q = 0), 16 TB w .. of B (q = 1); rows past the edge take
    // one that exists.
    int slot = 0;                                    // LDS slot of the group in use
    auto scale_dma = [&](const Place& p, int group, int to, int q) {
        const int per = q == 0 ? 16 * TA : 16 * TB;
        const int row = min((q == 0 ? p.m0 : p.n0) + per * wave + min(lane, per - 1), (q == 0 ? p.end : N) - 1);
        const uint32_t* src = q == 0 ? sA.words + group * sA.rows + (row >> sA.shift)
                                     : sB.words + group * sB.rows + (row >> sB.shift);
        if constexpr (KIND == ROWS) src += q == 0 ? 0 : static_cast<int64_t>(p.e) * ((((K + 127) >> 7) + 3) >> 2) * sB.rows;
        // (a group without rows has no words; what is read in their place is not used)
        if constexpr (KIND == COLUMNS)
            src = p.real ? src + p.word * (q == 0 ? sA.rows : sB.rows) : reinterpret_cast<const uint32_t*>(grp.offsets);
        lds_void* dst = (lds_void*)(lds + T::SCALES + to * T::SCALE_GROUP + (q == 0 ? 0 : T::ROWS_A * 4) + wave * per * 4);
        if (lane < per) __builtin_amdgcn_global_load_lds(src, dst, 4, 0, 0);
    };

    // Fragment reads of step ks: lane (frag_row r, half h) reads chunks 4 ks + h
    // and 4 ks + 2 + h of rows wm 32 TA + 32 t + r (A), wn 32 TB + 32 t + r (B).
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_byte*)lds));
    const int frag_row = lane & 31;
    const int half = lane >> 5;
    const int sw = (frag_row >> 1) & 7;
    uint32_t rd_a[2][2][2], rd_b[2][2][2];           // [buffer][ks][low, high chunk]
#pragma unroll
    for (int bf = 0; bf < 2; ++bf)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t pos = static_cast<uint32_t>(((4 * ks + 2 * q + half) ^ sw) * 16);
                rd_a[bf][ks][q] = lds0 + bf * T::STAGE_BYTES + (wm * 32 * TA + frag_row) * kRowBytes + pos;
                rd_b[bf][ks][q] = lds0 + bf * T::STAGE_BYTES + T::A_BYTES + (wn * 32 * TB + frag_row) * kRowBytes + pos;
            }

    v16f acc[TB][TA];
    // zeros by the matrix core (0 x 0 + 0), straight into the accumulation
    // registers: through VGPRs they cost the main loop's registers
    auto clear = [&]() {
        u32x4 z = {0u, 0u, 0u, 0u};
        asm volatile("s_nop 4" : "+v"(z));
#pragma unroll
        for (int i = 0; i < TB; ++i)
#pragma unroll
            for (int j = 0; j < TA; ++j) asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %1, 0" : "=a"(acc[i][j]) : "v"(z));
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    };
    clear();

    struct Frag { u32x4 xl[TB], xh[TB], yl[TA], yh[TA]; };
    Frag fr[2];                                      // 16-bit outputs: a step's fragments
    // read piece R (0 .. NR - 1) of step KS of the stage in buffer BUF: B first
    auto read_one = [&](auto R, Frag& dst, auto BUF, auto KS) {
        constexpr int r = R;
        constexpr int t = (r < 2 * TB ? r : r - 2 * TB) >> 1;
        constexpr int hi = r & 1;
        constexpr int off = t * 32 * kRowBytes;
        if constexpr (r < 2 * TB) lds_read16<off>(hi ? dst.xh[t] : dst.xl[t], rd_b[BUF][KS][hi]);
        else lds_read16<off>(hi ? dst.yh[t] : dst.yl[t], rd_a[BUF][KS][hi]);
    };
    // the scale words of this lane's rows: nxt as read from LDS, cur in use
    uint32_t nxt[TA + TB], cur[TA + TB];
    const uint32_t srd_a = lds0 + T::SCALES + (wm * 32 * TA + frag_row) * 4;
    const uint32_t srd_b = lds0 + T::SCALES + T::ROWS_A * 4 + (wn * 32 * TB + frag_row) * 4;
    auto read_scale = [&](auto I, int from) {
        constexpr int t = I;
        if constexpr (t < TA) lds_read4<t * 128>(nxt[t], srd_a + from * T::SCALE_GROUP);
        else lds_read4<(t - TA) * 128>(nxt[t], srd_b + from * T::SCALE_GROUP);
    };
    auto name_scales = [&](uint32_t (&v)[TA + TB]) {
#pragma unroll
        for (int t = 0; t < TA + TB; ++t) asm volatile("" : "+v"(v[t]));
    };
    // bytes past the last K block (their codes are zero) become a unit scale
    auto take_scales = [&](const Place& p, int group) {
        const uint32_t used = (p.real & 3) ? (1u << (8 * (p.real & 3))) - 1u : KIND == COLUMNS && p.real == 0 ? 0u : 0xFFFFFFFFu;
        // named after the wait for their reads: the compiler takes them as
        // written when the read is issued
        name_scales(nxt);
        const uint32_t keep = group == ((stages(p) + 3) >> 2) - 1 ? used : 0xFFFFFFFFu;
#pragma unroll
        for (int t = 0; t < TA + TB; ++t) cur[t] = (nxt[t] & keep) | (0x7F7F7F7Fu & ~keep);
        // VALU writes settle before an MFMA of the assembly reads them
        name_scales(cur);
        asm volatile("s_nop 4");
    };

    constexpr auto C0 = std::integral_constant<int, 0>{};
    constexpr auto C1 = std::integral_constant<int, 1>{};

    // FP32 output: a stage is 8 quarter steps of 16 K.  Half fragments (step ks,
    // low or high chunk: two quarters' codes) alternate between two sets; the
    // bf16 operands of a quarter are widened during the MFMAs of the one before.
    struct Half { u32x4 x[TB], y[TA]; };
    Half hs[2], wd[2];
    float fs[TA + TB];                               // the scales of the codes being widened
    auto read_half = [&](auto R, Half& dst, auto BUF, auto H) {
        constexpr int r = R, h = H;
        if constexpr (r < TB) lds_read16<r * 32 * kRowBytes>(dst.x[r], rd_b[BUF][h >> 1][h & 1]);
        else lds_read16<(r - TB) * 32 * kRowBytes>(dst.y[r - TB], rd_a[BUF][h >> 1][h & 1]);
    };
    // piece P (0 .. 4 (TA + TB) - 1) of quarter Q's operands: B and A rows in turn
    auto widen_one = [&](auto P, auto Q) {
        constexpr int r = P >> 2, e = P & 3, q = Q;
        constexpr int both = 2 * (TA < TB ? TA : TB);
        constexpr bool is_b = r < both ? (r & 1) == 0 : TB > TA;
        constexpr int t = r < both ? r >> 1 : r - both / 2;
        constexpr int word = 2 * (q & 1) + (e >> 1);
        const Half& f = hs[(q >> 1) & 1];
        Half& w = wd[q & 1];
        if constexpr (is_b) w.x[t][e] = widen2<BF, e & 1>(f.x[t][word], fs[TA + t]);
        else w.y[t][e] = widen2<AF, e & 1>(f.y[t][word], fs[t]);
    };
    auto take_floats = [&](int byte) {
#pragma unroll
        for (int t = 0; t < TA + TB; ++t) {
            fs[t] = __uint_as_float(((cur[t] >> (8 * byte)) & 255u) << 23);
            asm volatile("" : "+v"(fs[t]));
        }
        asm volatile("s_nop 1");
    };

    // Prologue: stage 0, the first scale group and stage 1 on their way.
    aim(here, true);
    static_for<T::NL>([&](auto J) { dma_one(J, C0); });
    advance();
    scale_dma(here, 0, 0, 0);
    scale_dma(here, 0, 0, 1);
    static_for<T::NL>([&](auto J) { dma_one(J, C1); });
    advance();
    asm volatile("s_waitcnt vmcnt(%0)" :: "i"(T::NL) : "memory");
    lds_wait_barrier();
    static_for<TA + TB>([&](auto I) { read_scale(I, 0); });
    if constexpr (!WIDE) {
        static_for<T::NR>([&](auto R) { read_one(R, fr[0], C0, C0); });
        // (the lookup of the next tile follows: as in advance)
        lds_wait();
    } else {
        static_for<TA + TB>([&](auto R) { read_half(R, hs[0], C0, C0); });
        static_for<TA + TB>([&](auto R) { read_half(R, hs[1], C0, C1); });
        lds_wait();
        take_scales(here, 0);
        take_floats(0);
        static_for<4 * (TA + TB)>([&](auto P) { widen_one(P, C0); });
    }

    bool stores = false;                             // an epilogue's stores may be in flight
    for (;;) {
        Place there = here;
        const int next = next_tile(tile + gridDim.x, gridDim.x), nst = stages(here), ngr = (nst + 3) >> 2;
        const bool more = next < last;
        if (more) there = locate(next);
        auto run_stage = [&](int s, auto U) {
            constexpr int u = U;                     // stage within its scale group
            constexpr auto cb = std::integral_constant<int, u & 1>{};
            constexpr auto nb = std::integral_constant<int, (u & 1) ^ 1>{};
            lds_wait();
            if constexpr (u == 0) {
                take_scales(here, s >> 2);
            }
            const bool group_end = u == 3 || (u == 1 && s + 1 == nst);
            static_for<2 * T::NM>([&](auto N_) {
                constexpr int n = N_;
                constexpr int ks = n / T::NM;
                constexpr int ti = n % T::NM / TA, tj = n % TA;
                const Frag& f = fr[ks];
                const u32x8 x = __builtin_shufflevector(f.xl[ti], f.xh[ti], 0, 1, 2, 3, 4, 5, 6, 7);
                const u32x8 y = __builtin_shufflevector(f.yl[tj], f.yh[tj], 0, 1, 2, 3, 4, 5, 6, 7);
                mfma_scaled<u, mfma_fmt<BF>(), mfma_fmt<AF>()>(acc[ti][tj], x, y, cur[TA + ti], cur[tj]);
                if constexpr (n * T::RPS < T::NR)
                    static_for<T::RPS>([&](auto Q) {
                        if constexpr (n * T::RPS + Q < T::NR)
                            read_one(std::integral_constant<int, n * T::RPS + Q>{}, fr[1], cb, C1);
                    });
                if constexpr (n == T::FREE) lds_wait_barrier();
                static_for<T::NL>([&](auto J) {
                    if constexpr (T::load_slot(J) == n) dma_one(J, cb);
                });
                if constexpr (n == T::READY) {
                    // stage s + 1 has landed once only the loads issued in this
                    // stage (and, in a tile's first, the last tile's stores,
                    // which are younger than it) are outstanding
                    if (u == 0 && stores) {
                        asm volatile("s_waitcnt vmcnt(%0)" :: "i"(T::newer() + T::STORES) : "memory");
                        stores = false;
                    } else {
                        asm volatile("s_waitcnt vmcnt(%0)" :: "i"(T::newer()) : "memory");
                    }
                    lds_wait_barrier();
                }
                if constexpr (n > T::READY && (n - T::READY - 1) * T::RPS < T::NR)
                    static_for<T::RPS>([&](auto Q) {
                        if constexpr ((n - T::READY - 1) * T::RPS + Q < T::NR)
                            read_one(std::integral_constant<int, (n - T::READY - 1) * T::RPS + Q>{}, fr[0], nb, C0);
                    });
                // the next group's scales, or the next tile's first: loaded in a
                // group's first stage, read in its last
                if constexpr (u == 0 && n == T::READY + 1) {
                    const bool in = (s >> 2) + 1 < ngr;
                    scale_dma(in ? here : there, in ? (s >> 2) + 1 : 0, slot ^ 1, 0);
                    scale_dma(in ? here : there, in ? (s >> 2) + 1 : 0, slot ^ 1, 1);
                }
                if constexpr ((u & 1) && n == 2 * T::NM - 2) {
                    if (group_end) {
                        slot ^= 1;
                        static_for<TA + TB>([&](auto I) { read_scale(I, slot); });
                    }
                }
            });
            advance();
        };
        // FP32 output, a stage: quarter q runs its MFMAs, widens quarter q + 1, and
        //   q = 1, 3  reads half 2, 3 of this stage;
        //   q = 5     starts with the barrier: every wave has read this stage, and
        //             the next one has landed (its loads ended five quarters, some
        //             2500 cycles, ago); then half 0 of the next stage is read, and
        //             the loads of stage s + 2 go out over the last three quarters;
        //   q = 7     takes the next stage's scales and reads its half 1.
        auto run_stage_wide = [&](int s, auto CB) {
            constexpr auto cb = std::integral_constant<int, CB>{};
            constexpr auto nb = std::integral_constant<int, CB ^ 1>{};
            const int u = s & 3;                     // stage within its scale group
            const bool group_end = u == 3 || s + 1 == nst;
            static_for<8>([&](auto Q_) {
                constexpr int q = Q_;
                if constexpr (q & 1) lds_wait();
                if constexpr (q == 5) {
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    lds_wait_barrier();
                    if constexpr (cb == 0) {
                        if (u == 0) {
                            const bool in = (s >> 2) + 1 < ngr;
                            scale_dma(in ? here : there, in ? (s >> 2) + 1 : 0, slot ^ 1, 0);
                            scale_dma(in ? here : there, in ? (s >> 2) + 1 : 0, slot ^ 1, 1);
                        }
                    } else if (group_end) {
                        slot ^= 1;
                        static_for<TA + TB>([&](auto I) { read_scale(I, slot); });
                    }
                }
                if constexpr (q == 7) {
                    if constexpr (cb == 1) {
                        if (group_end) take_scales(s + 1 == nst ? there : here, s + 1 == nst ? 0 : (s + 1) >> 2);
                    }
                    take_floats(group_end ? 0 : u + 1);
                }
                static_for<T::NM>([&](auto N_) {
                    constexpr int n = N_;
                    constexpr int ti = n / TA, tj = n % TA;
                    constexpr int W = 4 * (TA + TB);
                    mfma_bf16_k16(acc[ti][tj], wd[q & 1].x[ti], wd[q & 1].y[tj]);
                    static_for<W>([&](auto P) {
                        if constexpr (P * T::NM / W == n) widen_one(P, std::integral_constant<int, (q + 1) & 7>{});
                    });
                    if constexpr (q & 1)
                        static_for<TA + TB>([&](auto R) {
                            if constexpr (R * T::NM / (TA + TB) == n) {
                                if constexpr (q == 1) read_half(R, hs[0], cb, std::integral_constant<int, 2>{});
                                if constexpr (q == 3) read_half(R, hs[1], cb, std::integral_constant<int, 3>{});
                                if constexpr (q == 5) read_half(R, hs[0], nb, C0);
                                if constexpr (q == 7) read_half(R, hs[1], nb, C1);
                            }
                        });
                    static_for<T::NL>([&](auto J) {
                        if constexpr (5 * T::NM + J * 3 * T::NM / T::NL == q * T::NM + n) dma_one(J, cb);
                    });
                });
            });
            advance();
        };
        if constexpr (WIDE) {
            for (int s = 0; s < nst; s += 2) {
                run_stage_wide(s, C0);
                run_stage_wide(s + 1, C1);
            }
        } else {
            for (int s = 0; s < nst; s += 4) {
                run_stage(s, C0);
                run_stage(s + 1, C1);
                if (s + 2 < nst) {
                    run_stage(s + 2, std::integral_constant<int, 2>{});
                    run_stage(s + 3, std::integral_constant<int, 3>{});
                }
            }
        }
        // The next tile's first fragments and scales are in their registers
        // before the compiler's own code runs (it may move them); MFMA results
        // must settle before the accumulation registers are read.
        lds_wait();
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
        for (int i = 0; i < TB; ++i)
#pragma unroll
            for (int j = 0; j < TA; ++j) asm volatile("" : "+a"(acc[i][j]));
        if constexpr (!T::PERSISTENT) {
            // the strips reuse the stages: no wave reads them any more and no
            // load is on its way there
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            lds_wait_barrier();
        }

        // Epilogue, each wave by itself through its own strip of LDS, so that
        // stores write whole lines.  acc[ti][tj][4 q + e] is row 32 tj +
        // frag_row, column 32 ti + 8 q + 4 half + e of the wave's part.  Chunk c
        // (16 bytes) of strip row R sits at c ^ ((R >> 1) & 7).
        // (The lane is opaque here, so that the epilogue's addresses are not kept
        // in registers through the main loop.)
        uint8_t* strip = lds + T::STRIPS + wave * kStripBytes;
        const int mw = here.m0 + wm * 32 * TA, nw = here.n0 + wn * 32 * TB;
        void* out = D;
        Epilogue fin = ep;
        if constexpr (KIND == COLUMNS) {
            constexpr int es = OUT == BSFP8_OUT_F32 ? 4 : 2;
            out = static_cast<uint8_t*>(D) + here.e * grp.d_group * es;
            if (ep.c) fin.c = static_cast<const uint8_t*>(ep.c) + here.e * grp.c_group * es;
        }
        int el = lane;
        asm volatile("" : "+v"(el));
        const int srow = el >> 3, schunk = el & 7;
        uint8_t* put = strip + (el & 31) * 128;
        const int psw = (el >> 1) & 7, phalf = el >> 5;
        if constexpr (FAST && WIDE) {
            // strips of 32 rows x 32 columns; C, if any, kAhead strips ahead of its use (one
            // ahead, a CU has 16 KB of it in flight, where HBM needs some 40)
            constexpr int es = 4, STRIPS = TA * TB, kAhead = STRIPS < 4 ? STRIPS : 4;
            const __amdgpu_buffer_rsrc_t rs_d = __builtin_amdgcn_make_buffer_rsrc(
                static_cast<uint8_t*>(out) + static_cast<int64_t>(here.m0) * ldd * es, 0,
                min(T::ROWS_A, here.end - here.m0) * static_cast<int>(ldd) * es, 0x00020000);
            const __amdgpu_buffer_rsrc_t rs_c = __builtin_amdgcn_make_buffer_rsrc(
                static_cast<uint8_t*>(const_cast<void*>(fin.c)) + static_cast<int64_t>(here.m0) * fin.ldc * es, 0,
                min(T::ROWS_A, here.end - here.m0) * static_cast<int>(fin.ldc) * es, 0x00020000);
            const uint32_t ld4 = static_cast<uint32_t>(ldd) * es, lc4 = static_cast<uint32_t>(fin.ldc) * es;
            const int row = wm * 32 * TA + srow;
            const bool edge = (N & 3) && here.n0 + T::ROWS_B > N;
            auto column = [&](int ti) { return nw + 32 * ti + 4 * schunk; };
            u32x4 c[kAhead][4];
            auto fetch_c = [&](auto S) {
                constexpr int tj = S / TB, ti = S % TB;
                const uint32_t at = column(ti) + 4 <= N ? row * lc4 + column(ti) * es : 0x80000000u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const auto w = __builtin_amdgcn_raw_buffer_load_b128(rs_c, at + (32 * tj + 8 * i) * lc4, 0, 0);
                    c[S % kAhead][i] = u32x4{w[0], w[1], w[2], w[3]};
                }
            };
            if (fin.beta != 0.0f) static_for<kAhead>([&](auto S) { fetch_c(S); });
            static_for<STRIPS>([&](auto S) {
                constexpr int tj = S / TB, ti = S % TB;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v16f& a = acc[ti][tj];
                    *reinterpret_cast<float4*>(put + (((2 * q + phalf) ^ psw) << 4)) =
                        make_float4(a[4 * q + 0], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
                }
                __builtin_amdgcn_wave_barrier();
                const uint32_t at = column(ti) + 4 <= N ? row * ld4 + column(ti) * es : 0x80000000u;
                u32x4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int R = 8 * i + srow;
                    const float4 v = *reinterpret_cast<const float4*>(strip + R * 128 + ((schunk ^ ((R >> 1) & 7)) << 4));
                    w[i] = u32x4{__float_as_uint(fin.alpha * v.x), __float_as_uint(fin.alpha * v.y),
                                 __float_as_uint(fin.alpha * v.z), __float_as_uint(fin.alpha * v.w)};
                }
                if (fin.beta != 0.0f) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[i][j] = __float_as_uint(fmaf(fin.beta, __uint_as_float(c[S % kAhead][i][j]), __uint_as_float(w[i][j])));
                    if constexpr (S + kAhead < STRIPS) fetch_c(std::integral_constant<int, S + kAhead>{});
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    __builtin_amdgcn_raw_buffer_store_b128(w[i], rs_d, at + (32 * tj + 8 * i) * ld4, 0, 0);
                // the last N % 4 columns, in the lanes of the chunk that they begin (its C is not in w)
                if (edge) {
                    const bool mine = column(ti) < N && column(ti) + 4 > N;
#pragma unroll 1
                    for (int e = 0; e < (N & 3); ++e)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t o = mine ? (column(ti) + e) * es + row * ld4 : 0x80000000u;
                            const uint32_t oc = mine ? (column(ti) + e) * es + row * lc4 : 0x80000000u;
                            float v = __uint_as_float(e == 0 ? w[i][0] : e == 1 ? w[i][1] : w[i][2]);
                            if (fin.beta != 0.0f)
                                v = fmaf(fin.beta, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs_c, oc + (32 * tj + 8 * i) * lc4, 0, 0)), v);
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rs_d, o + (32 * tj + 8 * i) * ld4, 0, 0);
                        }
                }
                __builtin_amdgcn_wave_barrier();
            });
        } else if constexpr (FAST) {
            static_assert(OUT != BSFP8_OUT_F32 && TB % 2 == 0, "16-bit output, column pairs");
            // strips of 32 rows x 64 columns of 16-bit outputs
            const __amdgpu_buffer_rsrc_t rs_d = __builtin_amdgcn_make_buffer_rsrc(
                static_cast<uint16_t*>(out) + static_cast<int64_t>(here.m0) * ldd, 0,
                min(T::ROWS_A, here.end - here.m0) * static_cast<int>(ldd) * 2, 0x00020000);
            // byte offset of this lane's first chunk of each column pair; past
            // column N one that stays out of range whatever rows are added
            const uint32_t ld2 = static_cast<uint32_t>(ldd) * 2;
            uint32_t at[TB / 2];
#pragma unroll
            for (int tp = 0; tp < TB / 2; ++tp) {
                const int col = nw + 64 * tp + 8 * schunk;
                at[tp] = (KIND == ONE ? col : col + 7) < N ? (wm * 32 * TA + srow) * ld2 + col * 2 : 0x80000000u;
            }
            // (groups' products take any N: the last N % 8 columns go one by one, beside the count of
            // stores that the main loop allows for, which may be more)
            const bool edge = KIND != ONE && (N & 7) && here.n0 + T::ROWS_B > N;
#pragma unroll
            for (int tj = 0; tj < TA; ++tj)
#pragma unroll
                for (int tp = 0; tp < TB / 2; ++tp) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const v16f& a = acc[2 * tp + t][tj];
                            uint2 w;
                            if constexpr (KIND == ONE)
                                w = make_uint2(bf16_pair(a[4 * q + 0], a[4 * q + 1]), bf16_pair(a[4 * q + 2], a[4 * q + 3]));
                            else
                                w = make_uint2(half_pair<OUT>(ep.alpha * a[4 * q + 0], ep.alpha * a[4 * q + 1]),
                                               half_pair<OUT>(ep.alpha * a[4 * q + 2], ep.alpha * a[4 * q + 3]));
                            *reinterpret_cast<uint2*>(put + (((4 * t + q) ^ psw) << 4) + 8 * phalf) = w;
                        }
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int R = 8 * i + srow;
                        const u32x4 w = *reinterpret_cast<const u32x4*>(strip + R * 128 + ((schunk ^ ((R >> 1) & 7)) << 4));
                        __builtin_amdgcn_raw_buffer_store_b128(w, rs_d, at[tp] + (32 * tj + 8 * i) * ld2, 0, 0);
                    }
                    if (edge) {
                        const int col = nw + 64 * tp + 8 * schunk;
                        const uint32_t o = col < N && col + 8 > N ? (wm * 32 * TA + srow) * ld2 + col * 2 : 0x80000000u;
#pragma unroll 1
                        for (int e = 0; e < (N & 7); ++e)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int R = 8 * i + srow;
                                const uint16_t w = *reinterpret_cast<const uint16_t*>(strip + R * 128 + ((schunk ^ ((R >> 1) & 7)) << 4) + 2 * e);
                                __builtin_amdgcn_raw_buffer_store_b16(w, rs_d, o + 2 * e + (32 * tj + 8 * i) * ld2, 0, 0);
                            }
                    }
                    __builtin_amdgcn_wave_barrier();
                }
            stores = T::PERSISTENT;
        } else {
            // strips of 32 rows x 32 columns in FP32; alpha, beta C and the
            // conversion row by row, masked at the edges
#pragma unroll
            for (int tj = 0; tj < TA; ++tj)
#pragma unroll
                for (int ti = 0; ti < TB; ++ti) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const v16f& a = acc[ti][tj];
                        *reinterpret_cast<float4*>(put + (((2 * q + phalf) ^ psw) << 4)) =
                            make_float4(a[4 * q + 0], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
                    }
                    __builtin_amdgcn_wave_barrier();
                    if constexpr (KIND == ONE) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int R = 8 * i + srow;
                            const float4 v = *reinterpret_cast<const float4*>(strip + R * 128 + ((schunk ^ ((R >> 1) & 7)) << 4));
                            const float a4[4] = {v.x, v.y, v.z, v.w};
                            finish_row_chunk<OUT, 4>(out, ldd, fin, mw + 32 * tj + R, nw + 32 * ti + 4 * schunk, here.end, N, vec_ok, a4);
                        }
                    } else {
                        // (not unrolled: with every strip's edges written out, this tile took minutes to compile)
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            const int R = 8 * i + srow;
                            const float4 v = *reinterpret_cast<const float4*>(strip + R * 128 + ((schunk ^ ((R >> 1) & 7)) << 4));
                            finish_chunk<OUT>(out, ldd, fin, mw + 32 * tj + R, nw + 32 * ti + 4 * schunk, here.end, N, v);
                        }
                    }
                    __builtin_amdgcn_wave_barrier();
                }
            // a masked store may not have been issued: none is left in flight
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        if (!T::PERSISTENT || !more) break;
        clear();
        tile = next;
        here = there;
    }
    // no direct load may still be writing LDS when the workgroup ends, and the
    // last reads, which have no consumer, are named after the wait so that
    // their registers are not reused while in flight
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if constexpr (WIDE) {
#pragma unroll
        for (int t = 0; t < TB; ++t) asm volatile("" :: "v"(hs[0].x[t]), "v"(hs[1].x[t]), "v"(wd[0].x[t]));
#pragma unroll
        for (int t = 0; t < TA; ++t) asm volatile("" :: "v"(hs[0].y[t]), "v"(hs[1].y[t]), "v"(wd[0].y[t]));
    } else {
#pragma unroll
        for (int t = 0; t < TB; ++t) asm volatile("" :: "v"(fr[0].xl[t]), "v"(fr[0].xh[t]));
#pragma unroll
        for (int t = 0; t < TA; ++t) asm volatile("" :: "v"(fr[0].yl[t]), "v"(fr[0].yh[t]));
    }
    name_scales(nxt);
}

// Persistent workgroups: one per CU.
constexpr int64_t kPersistent = 256;

template <int AF, int BF, int OUT, int TA, int TB, bool FAST>
hipError_t launch_typed(const TileArgs& t) {
    const int64_t tm = (t.M + 64 * TA - 1) / (64 * TA), tn = (t.N + 64 * TB - 1) / (64 * TB);
    const int64_t grid = Tile<TA, TB>::PERSISTENT && tm * tn > kPersistent ? kPersistent : tm * tn;
    hipLaunchKernelGGL((gemm_block128_tile_kernel<AF, BF, OUT, TA, TB, FAST>), dim3(static_cast<uint32_t>(grid)),
                       dim3(kThreads), 0, t.stream, static_cast<int>(t.M), static_cast<int>(t.N),
                       static_cast<int>(t.K), t.a, t.sa, t.b, t.sb, t.d, t.ldd, t.ep, static_cast<int>(tm),
                       static_cast<int>(tn), vec16_ok(OUT, t.d, t.ldd, t.ep), GroupsArg{});
    return hipGetLastError();
}

// F32: FP32 output is wanted on this tile.
template <int AF, int BF, int TA, int TB, bool F32>
hipError_t launch_out(const TileArgs& t) {
    if constexpr (F32) {
        if (t.out == BSFP8_OUT_F32) return launch_typed<AF, BF, BSFP8_OUT_F32, TA, TB, false>(t);
    } else if (t.out == BSFP8_OUT_F32) {
        return hipErrorInvalidValue;
    }
    if (t.out == BSFP8_OUT_F16) return launch_typed<AF, BF, BSFP8_OUT_F16, TA, TB, false>(t);
    // the buffer stores' offsets within a tile's rows are 32-bit
    if (t.ep.alpha == 1.0f && t.ep.beta == 0.0f && vec16_ok(t.out, t.d, t.ldd, t.ep) && t.N % 8 == 0 && t.ldd < (int64_t(1) << 21))
        return launch_typed<AF, BF, BSFP8_OUT_BF16, TA, TB, true>(t);
    return launch_typed<AF, BF, BSFP8_OUT_BF16, TA, TB, false>(t);
}

template <int TA, int TB, bool F32 = true>
hipError_t launch_tile(const TileArgs& t) {
    if (t.a_fmt == BSFP8_E4M3)
        return t.b_fmt == BSFP8_E4M3 ? launch_out<BSFP8_E4M3, BSFP8_E4M3, TA, TB, F32>(t)
                                     : launch_out<BSFP8_E4M3, BSFP8_E5M2, TA, TB, F32>(t);
    return t.b_fmt == BSFP8_E4M3 ? launch_out<BSFP8_E5M2, BSFP8_E4M3, TA, TB, F32>(t)
                                 : launch_out<BSFP8_E5M2, BSFP8_E5M2, TA, TB, F32>(t);
}

// The same for products grouped by rows and by columns.  Workgroups: one per CU, or (the smallest tile)
// one per tile, as many as there can be; a multiple of 8, so that a workgroup's tiles stay on its XCD.
inline int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

template <int AF, int BF, int OUT, int TA, int TB, bool FAST>
hipError_t launch_rows(const GroupedArgs& t) {
    const int64_t tn = (t.N + 64 * TB - 1) / (64 * TB), tiles = (t.M / (64 * TA) + (t.M < t.groups ? t.M : t.groups)) * tn;
    const int64_t grid = Tile<TA, TB>::PERSISTENT && tiles > kPersistent ? kPersistent : up8(tiles);
    hipLaunchKernelGGL((gemm_block128_tile_kernel<AF, BF, OUT, TA, TB, FAST, ROWS>), dim3(static_cast<uint32_t>(grid)),
                       dim3(kThreads), 0, t.stream, static_cast<int>(t.M), static_cast<int>(t.N),
                       static_cast<int>(t.K), t.a, t.sa, t.b, t.sb, t.d, t.ldd, t.ep, 0, static_cast<int>(tn),
                       0, GroupsArg{t.offsets, t.groups, 0, 0, 0});
    return hipGetLastError();
}

template <int AF, int BF, int OUT, int TA, int TB, bool FAST>
hipError_t launch_columns(const GroupedKArgs& t) {
    const int64_t tm = (t.M + 64 * TA - 1) / (64 * TA), tn = (t.N + 64 * TB - 1) / (64 * TB);
    const int64_t tiles = up8(tm * tn) * t.groups;
    const int64_t grid = Tile<TA, TB>::PERSISTENT && tiles > kPersistent ? kPersistent : tiles;
    const ScaleRows sa{t.sa, t.M, 0}, sb{t.sb, t.N, 0};
    hipLaunchKernelGGL((gemm_block128_tile_kernel<AF, BF, OUT, TA, TB, FAST, COLUMNS>), dim3(static_cast<uint32_t>(grid)),
                       dim3(kThreads), 0, t.stream, static_cast<int>(t.M), static_cast<int>(t.N),
                       static_cast<int>(t.columns), t.a, sa, t.b, sb, t.d, t.ldd, t.ep, static_cast<int>(tm),
                       static_cast<int>(tn), 0, GroupsArg{t.offsets, t.groups, t.words, t.d_group, t.c_group});
    return hipGetLastError();
}

// FAST where the call allows it (fast_ok), else the general form, where the tile has one (GENERAL).
template <int TA, int TB, bool GENERAL>
hipError_t launch_grouped_tile(const GroupedArgs& t) {
    return by_type(t, [](auto AF, auto BF, auto OUT, const GroupedArgs& g) {
        if constexpr (!GENERAL && OUT == BSFP8_OUT_F32) return hipErrorInvalidValue;
        else if (g.fast_ok()) return launch_rows<AF, BF, OUT, TA, TB, true>(g);
        else if constexpr (GENERAL) return launch_rows<AF, BF, OUT, TA, TB, false>(g);
        else return hipErrorInvalidValue;
    });
}

}  // namespace
}  // namespace bsfp8
