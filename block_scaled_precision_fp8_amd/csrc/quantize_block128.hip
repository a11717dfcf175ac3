// quantize_block128.hip -- FP8 quantisation with one power-of-two scale per
// 1 x 128 or 128 x 128 block, of a matrix, its transpose, or both (gfx950).
//
// Per block: e = the smallest integer with F 2^e >= max |x| (F = 448 or 57344,
// both 1.75 times a power of two, so e is read off the exponent of the maximum
// plus one where its fraction is above 0.75), code = RNE(x 2^-e).  The product
// x 2^-e is exact (or far below half the smallest code), so each code is
// rounded once.  A block that holds an infinity or a NaN gets the scale byte
// 0xFF (NaN) and NaN codes: the maximum is taken over the bit patterns of |x|,
// where NaN > infinity > every finite value.
#include "block128_codec.h"

namespace bsfp8 {

namespace {

using namespace block128;

constexpr int kThreads = 256;
constexpr int kPitch = 132;      // LDS bytes per row of the transposed tile (128 codes + 4)
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;   // a launch's threads are counted in 32 bits
constexpr int64_t kSmallItems = 16384;

// 1 x 128 blocks of x alone: 16 lanes take four K blocks of a row (512 values,
// one scale word), all their loads in flight at once, and need nothing from
// anyone else.  16 x 8192 bf16 (16 decoded tokens): 3.1 us, against 8.0 by the
// tile kernel below, where most of a 128-row tile's lanes have no row.
// 16384 x 4096 bf16: 34 us, 5.9 TB/s (items along a row side by side; with the
// rows side by side 38.6 us).
template <int XT, int FMT>
__global__ void quantize_block128_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t k, int64_t ld, int vec,
                                              uint8_t* __restrict__ codes, uint32_t* __restrict__ scales, int64_t groups) {
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4;
    const int c = threadIdx.x & 15;
    const int64_t r = item / groups;
    const int64_t g = item - r * groups;
    if (r >= rows) return;
    const int64_t kp = (k + 31) & ~static_cast<int64_t>(31);
    Eight<XT> v[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int64_t c0 = g * 512 + b * 128;
        v[b] = load_eight<XT>(x, r * ld, c0, c, k, vec && c0 + col_of<XT>(c, 7) < k);
    }
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint32_t m = max16(v[b].abs().widest());
        const uint32_t byte = scale_byte<FMT>(Eight<XT>::bits(m));        // 127 for a block past k: its values are zeros
        word |= byte << (8 * b);
        const float f = inverse_scale(byte);
        uint32_t w0 = fp8_pack4<FMT>(v[b][0] * f, v[b][1] * f, v[b][2] * f, v[b][3] * f);
        uint32_t w1 = fp8_pack4<FMT>(v[b][4] * f, v[b][5] * f, v[b][6] * f, v[b][7] * f);
        if (byte == 255u) w0 = w1 = kNanCodes;
        put_codes<XT>(codes + r * kp, g * 512 + b * 128, kp, c, w0, w1);
    }
    if (c == 0) scales[g * rows + r] = word;
}

// One workgroup takes a 128 x 128 tile.  Thread (c = t % 16, g = t / 16) holds
// eight columns (col_of) of rows 8 g .. 8 g + 7 in registers: the tile is read
// once, and the row maxima (over the 16 lanes of a row), the column maxima
// (over g) or the tile's maximum come from there.  The transposed codes, eight
// consecutive rows of a column in two words, pass through LDS so that they are
// written as rows of 128 bytes.
template <int XT, int FMT, bool SQUARE>
__global__ __launch_bounds__(kThreads) void quantize_block128_kernel(
    const void* __restrict__ x, int64_t rows, int64_t k, int64_t ld, int vec, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales, uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t, int sr, int sc,
    int supers_c) {
    __shared__ uint32_t red[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t tl[128 * kPitch];
    const int64_t nkb = (k + 127) >> 7, nrb = (rows + 127) >> 7;
    // Workgroups go to the 8 XCDs round-robin: the sr x sc tiles (4 x 4 where
    // there are as many) that share scale words run on one XCD at about the same
    // time, so that their single bytes meet in its L2 and leave as whole words.
    // In plain order, where a word's bytes came from four L2s, 16384 x 4096 bf16
    // transposed took 40.3 us instead of 38.4, both orientations 62.4 instead of 61.3.
    const int idx = blockIdx.x >> 3;
    const int super = idx / (sr * sc) * 8 + (blockIdx.x & 7), within = idx % (sr * sc);
    const int64_t rt = static_cast<int64_t>(super / supers_c) * sr + within / sc;
    const int64_t ct = static_cast<int64_t>(super % supers_c) * sc + within % sc;
    if (rt >= nrb || ct >= nkb) return;
    const int64_t kp = (k + 31) & ~static_cast<int64_t>(31), rp = (rows + 31) & ~static_cast<int64_t>(31);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = tid & 15, g = tid >> 4;
    const int64_t r0 = rt * 128 + 8 * g, c0 = ct * 128;

    Eight<XT> v[8];
    const bool whole = vec && c0 + col_of<XT>(c, 7) < k;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool in = r0 + i < rows;
        v[i] = load_eight<XT>(x, in ? (r0 + i) * ld : 0, c0, c, in ? k : 0, in && whole);
    }

    uint32_t byte_r[8], byte_c[8];
    if constexpr (SQUARE) {
        Eight<XT> a = v[0].abs();
#pragma unroll
        for (int i = 1; i < 8; ++i) a.take_max(v[i].abs());
        uint32_t m = max_rows(max16(a.widest()));
        if (lane == 0) red[0][wave] = m;
        __syncthreads();
        m = umax(umax(red[0][0], red[0][1]), umax(red[0][2], red[0][3]));
        const uint32_t b = scale_byte<FMT>(Eight<XT>::bits(m));
#pragma unroll
        for (int i = 0; i < 8; ++i) byte_r[i] = byte_c[i] = b;
        if (tid == 0) {
            if (codes) put_scale(scales, nrb, rt, ct, nkb, b);
            if (codes_t) put_scale(scales_t, nkb, ct, rt, nrb, b);
        }
    } else {
        if (codes) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                byte_r[i] = scale_byte<FMT>(Eight<XT>::bits(max16(v[i].abs().widest())));
                if (c == 0 && r0 + i < rows) put_scale(scales, rows, r0 + i, ct, nkb, byte_r[i]);
            }
        }
        if (codes_t) {
            Eight<XT> a = v[0].abs();
#pragma unroll
            for (int i = 1; i < 8; ++i) a.take_max(v[i].abs());
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = max_rows(a.magnitude(j));
                if (lane < 16) red[wave][col_of<XT>(c, j)] = m;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int cc = col_of<XT>(c, j);
                const uint32_t m = umax(umax(red[0][cc], red[1][cc]), umax(red[2][cc], red[3][cc]));
                byte_c[j] = scale_byte<FMT>(Eight<XT>::bits(m));
                if (g == 0 && c0 + cc < k) put_scale(scales_t, k, c0 + cc, rt, nrb, byte_c[j]);
            }
        }
    }

    if (codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r0 + i >= rows) break;
            const float f = inverse_scale(byte_r[i]);
            uint32_t w0 = fp8_pack4<FMT>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f);
            uint32_t w1 = fp8_pack4<FMT>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f);
            if (byte_r[i] == 255u) w0 = w1 = kNanCodes;
            put_codes<XT>(codes + (r0 + i) * kp, c0, kp, c, w0, w1);
        }
    }
    if (codes_t) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = inverse_scale(byte_c[j]);
            uint32_t w0 = fp8_pack4<FMT>(v[0][j] * f, v[1][j] * f, v[2][j] * f, v[3][j] * f);
            uint32_t w1 = fp8_pack4<FMT>(v[4][j] * f, v[5][j] * f, v[6][j] * f, v[7][j] * f);
            if (byte_c[j] == 255u) w0 = w1 = kNanCodes;
            uint32_t* d = reinterpret_cast<uint32_t*>(tl + col_of<XT>(c, j) * kPitch + 8 * g);
            d[0] = w0;
            d[1] = w1;
        }
        __syncthreads();
        const int part = tid & 7;
#pragma unroll
        for (int pass = 0; pass < 4; ++pass) {
            const int r = pass * 32 + (tid >> 3);
            const int64_t orow = c0 + r, ocol = rt * 128 + 16 * part;
            if (orow >= k || ocol >= rp) continue;
            const uint32_t* s = reinterpret_cast<const uint32_t*>(tl + r * kPitch + 16 * part);
            *reinterpret_cast<uint4*>(codes_t + orow * rp + ocol) = make_uint4(s[0], s[1], s[2], s[3]);
        }
    }
}

template <int XT, int FMT>
hipError_t launch_typed(const void* x, int64_t rows, int64_t k, int64_t ld, int square, uint8_t* codes,
                        uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, hipStream_t stream) {
    const int64_t es = XT == BSFP8_OUT_F32 ? 4 : 2;
    const int vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (rows == 1 || (ld * es) % 16 == 0) ? 1 : 0;
    if (!square && !codes_t) {
        const int64_t groups = (k + 511) >> 9, items = rows * groups;
        // few items: a wave per workgroup, so that they spread over the CUs
        const int threads = items <= kSmallItems ? 64 : kThreads;
        if ((items * 16 + threads - 1) / threads <= kMaxGroups) {
            hipLaunchKernelGGL((quantize_block128_rows_kernel<XT, FMT>),
                               dim3(static_cast<uint32_t>((items * 16 + threads - 1) / threads)), dim3(threads), 0,
                               stream, x, rows, k, ld, vec, codes, reinterpret_cast<uint32_t*>(scales), groups);
            return hipGetLastError();
        }
    }
    const int64_t nkb = (k + 127) >> 7, nrb = (rows + 127) >> 7;
    const int sr = nrb >= 4 ? 4 : 1, sc = nkb >= 4 ? 4 : 1;
    const int64_t supers_c = (nkb + sc - 1) / sc, supers = (nrb + sr - 1) / sr * supers_c;
    const dim3 grid(static_cast<uint32_t>((supers + 7) / 8 * 8 * sr * sc));
    if (square)
        hipLaunchKernelGGL((quantize_block128_kernel<XT, FMT, true>), grid, dim3(kThreads), 0, stream, x, rows, k, ld,
                           vec, codes, scales, codes_t, scales_t, sr, sc, static_cast<int>(supers_c));
    else
        hipLaunchKernelGGL((quantize_block128_kernel<XT, FMT, false>), grid, dim3(kThreads), 0, stream, x, rows, k, ld,
                           vec, codes, scales, codes_t, scales_t, sr, sc, static_cast<int>(supers_c));
    return hipGetLastError();
}

template <int XT>
hipError_t launch_fmt(const void* x, int64_t rows, int64_t k, int64_t ld, int square, int fmt, uint8_t* codes,
                      uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, hipStream_t stream) {
    if (fmt == BSFP8_E4M3)
        return launch_typed<XT, BSFP8_E4M3>(x, rows, k, ld, square, codes, scales, codes_t, scales_t, stream);
    return launch_typed<XT, BSFP8_E5M2>(x, rows, k, ld, square, codes, scales, codes_t, scales_t, stream);
}

}  // namespace

hipError_t launch_quantize_block128(const void* x, int x_type, int64_t rows, int64_t k, int64_t ld, int block_rows,
                                    int fmt, uint8_t* codes, uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                                    hipStream_t stream) {
    const int square = block_rows == 128 ? 1 : 0;
    if (x_type == BSFP8_OUT_F32)
        return launch_fmt<BSFP8_OUT_F32>(x, rows, k, ld, square, fmt, codes, scales, codes_t, scales_t, stream);
    if (x_type == BSFP8_OUT_BF16)
        return launch_fmt<BSFP8_OUT_BF16>(x, rows, k, ld, square, fmt, codes, scales, codes_t, scales_t, stream);
    return launch_fmt<BSFP8_OUT_F16>(x, rows, k, ld, square, fmt, codes, scales, codes_t, scales_t, stream);
}

}  // namespace bsfp8
