// quantize_grouped.hip -- FP8 quantisation, one power-of-two scale per 128 elements,
// of rows sorted into groups (gfx950): by rows and, group by group, transposed.
//
// Sorted row i is row index[i] of x (or row i), so that the copy that sorts a
// router's tokens by expert is this kernel's read.  The codes by rows are those of
// quantize_block128.hip for the sorted matrix.  The transpose is the operand of a
// product over each group's rows: a block of 128 must lie in one group, so each
// group's columns start at a multiple of 128 (zeros up to the next one) and its scale
// bytes at a word.  Where that is depends on the offsets, which are on the device: each
// wave finds its tile's group by a scan over them, 64 groups at a time.
#include "block128_codec.h"
#include "groups.h"

namespace bsfp8 {

namespace {

using namespace block128;

constexpr int kThreads = 256;
constexpr int kPitch = 132;      // LDS bytes per row of the transposed tile (128 codes + 4)
constexpr int64_t kSmallItems = 16384;

struct Args {
    const void* x;
    const int32_t* index;
    const int32_t* offsets;
    int64_t source, k, ld, columns, words;
    int rows, groups;
    bool aligned;                // rows of x start at multiples of 16 bytes
    uint8_t* codes;
    uint8_t* scales;
    uint8_t* codes_t;
    uint8_t* scales_t;
};

// The row of x that sorted row i is, or -1: outside x it counts as a row of zeros.
__device__ __forceinline__ int source_row(const Args& a, int i) {
    const int s = a.index ? a.index[i] : i;
    return s >= 0 && s < a.source ? s : -1;
}

// load_eight at any element's address (rows of an odd length start anywhere): the hardware takes a
// 16-byte load there.  1111 x 4001 bf16 in 64 groups, both orientations: 37 us element by element, 25.2
// so (29.1 past the caches, since neighbouring tiles share lines; aligned rows go past them:
// 16384 x 4096 bf16 by index, both, 66 us against 68.6).
template <int XT>
__device__ __forceinline__ Eight<XT> load_any(const void* x, int64_t row, int64_t c0, int c, int64_t k, bool whole, bool aligned) {
    typedef u4v u4u __attribute__((aligned(2)));
    if (aligned || !whole) return load_eight<XT>(x, row, c0, c, k, whole);
    Eight<XT> v;
    if constexpr (XT == BSFP8_OUT_F32) {
        const float* p = static_cast<const float*>(x) + row + c0 + 4 * c;
        v.w[0] = *reinterpret_cast<const u4u*>(p);
        v.w[1] = *reinterpret_cast<const u4u*>(p + 64);
    } else {
        v.w = *reinterpret_cast<const u4u*>(static_cast<const uint16_t*>(x) + row + c0 + 8 * c);
    }
    return v;
}

// 1 x 128 blocks of the sorted rows alone, as quantize_block128_rows_kernel: 16 lanes
// take four K blocks of a row.
template <int XT, int FMT>
__global__ void quantize_grouped_rows_kernel(Args a, int64_t items_per_row) {
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4;
    const int c = threadIdx.x & 15;
    const int64_t r = item / items_per_row;
    const int64_t g = item - r * items_per_row;
    if (r >= a.rows || r < a.offsets[0] || r >= a.offsets[a.groups]) return;
    const int64_t kp = (a.k + 31) & ~static_cast<int64_t>(31);
    const int64_t s = source_row(a, static_cast<int>(r));
    Eight<XT> v[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int64_t c0 = g * 512 + b * 128;
        v[b] = load_any<XT>(a.x, s < 0 ? 0 : s * a.ld, c0, c, s < 0 ? 0 : a.k, s >= 0 && c0 + col_of<XT>(c, 7) < a.k, a.aligned);
    }
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint32_t byte = scale_byte<FMT>(Eight<XT>::bits(max16(v[b].abs().widest())));
        word |= byte << (8 * b);
        const float f = inverse_scale(byte);
        uint32_t w0 = fp8_pack4<FMT>(v[b][0] * f, v[b][1] * f, v[b][2] * f, v[b][3] * f);
        uint32_t w1 = fp8_pack4<FMT>(v[b][4] * f, v[b][5] * f, v[b][6] * f, v[b][7] * f);
        if (byte == 255u) w0 = w1 = kNanCodes;
        put_codes<XT>(a.codes + r * kp, g * 512 + b * 128, kp, c, w0, w1);
    }
    if (c == 0) reinterpret_cast<uint32_t*>(a.scales)[g * a.rows + r] = word;
}

// One workgroup takes 128 rows of a group x 128 columns, as quantize_block128_kernel.  (Several column
// tiles per workgroup, so as to find the group once, took more registers than that
// saved: 16384 x 4096 bf16 by index, both orientations, 75.7 us with two, 83.4 with four.)
template <int XT, int FMT>
__global__ __launch_bounds__(kThreads) void quantize_grouped_kernel(Args a, int sr, int sc, int supers_c) {
    __shared__ uint32_t red[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t tl[128 * kPitch];
    const int64_t nkb = (a.k + 127) >> 7;
    // tiles that share scale words on one XCD at about the same time
    const int idx = blockIdx.x >> 3;
    const int super = idx / (sr * sc) * 8 + (blockIdx.x & 7), within = idx % (sr * sc);
    const int rt = (super / supers_c) * sr + within / sc;
    const int64_t ct = static_cast<int64_t>(super % supers_c) * sc + within % sc;
    if (ct >= nkb || rt >= (a.columns >> 7)) return;
    const groups::Lane own = groups::of_tile<128>(a.offsets, a.groups, a.rows, rt);
    if (own.rows == 0) return;
    const int j = rt - own.tile;                     // tile of the group
    const int r0 = own.start + 128 * j, rows = own.rows - 128 * j;
    if (own.word + (j >> 2) >= a.words) return;
    const int64_t kp = (a.k + 31) & ~static_cast<int64_t>(31);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = tid & 15, g = tid >> 4;
    const int64_t c0 = ct * 128;

    Eight<XT> v[8];
    const bool whole = c0 + col_of<XT>(c, 7) < a.k;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t s = 8 * g + i < rows ? source_row(a, r0 + 8 * g + i) : -1;
        v[i] = load_any<XT>(a.x, s < 0 ? 0 : s * a.ld, c0, c, s < 0 ? 0 : a.k, s >= 0 && whole, a.aligned);
    }
    if (a.codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t byte = scale_byte<FMT>(Eight<XT>::bits(max16(v[i].abs().widest())));
            if (8 * g + i >= rows) continue;
            const int64_t r = r0 + 8 * g + i;
            if (c == 0) put_scale(a.scales, a.rows, r, ct, nkb, byte);
            const float f = inverse_scale(byte);
            uint32_t w0 = fp8_pack4<FMT>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f);
            uint32_t w1 = fp8_pack4<FMT>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f);
            if (byte == 255u) w0 = w1 = kNanCodes;
            put_codes<XT>(a.codes + r * kp, c0, kp, c, w0, w1);
        }
    }
    Eight<XT> m8 = v[0].abs();
#pragma unroll
    for (int i = 1; i < 8; ++i) m8.take_max(v[i].abs());
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint32_t m = max_rows(m8.magnitude(q));
        if (lane < 16) red[wave][col_of<XT>(c, q)] = m;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int cc = col_of<XT>(c, q);
        const uint32_t m = umax(umax(red[0][cc], red[1][cc]), umax(red[2][cc], red[3][cc]));
        const uint32_t byte = scale_byte<FMT>(Eight<XT>::bits(m));
        // (the group's word: block j of the tiles that the group has)
        if (g == 0 && c0 + cc < a.k) put_scale(a.scales_t + own.word * a.k * 4, a.k, c0 + cc, j, own.tiles, byte);
        const float f = inverse_scale(byte);
        uint32_t w0 = fp8_pack4<FMT>(v[0][q] * f, v[1][q] * f, v[2][q] * f, v[3][q] * f);
        uint32_t w1 = fp8_pack4<FMT>(v[4][q] * f, v[5][q] * f, v[6][q] * f, v[7][q] * f);
        if (byte == 255u) w0 = w1 = kNanCodes;
        uint32_t* d = reinterpret_cast<uint32_t*>(tl + cc * kPitch + 8 * g);
        d[0] = w0;
        d[1] = w1;
    }
    __syncthreads();
    const int part = tid & 7;
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const int r = pass * 32 + (tid >> 3);
        if (c0 + r >= a.k) continue;
        const uint32_t* p = reinterpret_cast<const uint32_t*>(tl + r * kPitch + 16 * part);
        *reinterpret_cast<uint4*>(a.codes_t + (c0 + r) * a.columns + static_cast<int64_t>(rt) * 128 + 16 * part) =
            make_uint4(p[0], p[1], p[2], p[3]);
    }
}

template <int XT, int FMT>
hipError_t launch_typed(Args a, hipStream_t stream) {
    const int64_t es = XT == BSFP8_OUT_F32 ? 4 : 2;
    a.aligned = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.source == 1 || (a.ld * es) % 16 == 0);
    if (!a.codes_t) {
        const int64_t per_row = (a.k + 511) >> 9, items = a.rows * per_row;
        const int threads = items <= kSmallItems ? 64 : kThreads;
        hipLaunchKernelGGL((quantize_grouped_rows_kernel<XT, FMT>),
                           dim3(static_cast<uint32_t>((items * 16 + threads - 1) / threads)), dim3(threads), 0, stream, a,
                           per_row);
        return hipGetLastError();
    }
    const int64_t nkb = (a.k + 127) >> 7, nrb = a.columns >> 7;
    const int sr = nrb >= 4 ? 4 : 1, sc = nkb >= 4 ? 4 : 1;
    const int64_t supers_c = (nkb + sc - 1) / sc, supers = (nrb + sr - 1) / sr * supers_c;
    hipLaunchKernelGGL((quantize_grouped_kernel<XT, FMT>), dim3(static_cast<uint32_t>((supers + 7) / 8 * 8 * sr * sc)),
                       dim3(kThreads), 0, stream, a, sr, sc, static_cast<int>(supers_c));
    return hipGetLastError();
}

template <int XT>
hipError_t launch_fmt(const Args& a, int fmt, hipStream_t stream) {
    return fmt == BSFP8_E4M3 ? launch_typed<XT, BSFP8_E4M3>(a, stream) : launch_typed<XT, BSFP8_E5M2>(a, stream);
}

}  // namespace

hipError_t launch_quantize_grouped(const void* x, int x_type, int64_t source, int64_t k, int64_t ld,
                                   const int32_t* index, int64_t rows, const int32_t* offsets, int groups, int fmt,
                                   uint8_t* codes, uint8_t* scales, uint8_t* codes_t, int64_t columns,
                                   uint8_t* scales_t, int64_t words, hipStream_t stream) {
    const Args a{x, index, offsets, source, k, ld, columns, words, static_cast<int>(rows), groups, false, codes, scales,
                 codes_t, scales_t};
    if (x_type == BSFP8_OUT_F32) return launch_fmt<BSFP8_OUT_F32>(a, fmt, stream);
    if (x_type == BSFP8_OUT_BF16) return launch_fmt<BSFP8_OUT_BF16>(a, fmt, stream);
    return launch_fmt<BSFP8_OUT_F16>(a, fmt, stream);
}

}  // namespace bsfp8
