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
#include "fp8_codec.h"

namespace bsfp8 {

namespace {

constexpr int kThreads = 256;
constexpr int kPitch = 132;      // LDS bytes per row of the transposed tile (128 codes + 4)
constexpr uint32_t kNanCodes = 0x7F7F7F7Fu;

// E8M0 byte of a block whose largest |x| has the bit pattern amax.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    constexpr int top = FMT == BSFP8_E4M3 ? 8 : 15;
    if (amax == 0) return 127u;
    if (amax >= 0x7F800000u) return 255u;
    const int b = static_cast<int>(amax >> 23) - top + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(b < 0 ? 0 : b);
}
// 2^-e for a scale byte e + 127 (the value for 255 is not used)
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Eight values of a row: elements col(0) .. col(7) of this thread's columns.
// 16-bit types: 8 consecutive columns (one 16-byte load); FP32: 4 + 4 columns
// 64 apart, so that each 16-byte load of a 16-lane group covers 256 bytes.
template <int XT>
__device__ __forceinline__ int col_of(int c, int j) {
    return XT == BSFP8_OUT_F32 ? (j >> 2) * 64 + 4 * c + (j & 3) : 8 * c + j;
}
template <int XT>
__device__ __forceinline__ float load_one(const void* x, int64_t i) {
    if constexpr (XT == BSFP8_OUT_F32) return static_cast<const float*>(x)[i];
    else return from_half_bits<XT>(static_cast<const uint16_t*>(x)[i]);
}
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
template <int XT>
__device__ __forceinline__ void load_eight(const void* x, int64_t row_off, int64_t c0, int c, float* v) {
    if constexpr (XT == BSFP8_OUT_F32) {
        const float* p = static_cast<const float*>(x) + row_off + c0 + 4 * c;
        const u4v a = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(p));
        const u4v b = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(p + 64));
#pragma unroll
        for (int j = 0; j < 4; ++j) { v[j] = __uint_as_float(a[j]); v[4 + j] = __uint_as_float(b[j]); }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + row_off + c0 + 8 * c;
        const u4v a = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(p));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = from_half_bits<XT>(static_cast<uint16_t>(a[j >> 1] >> (16 * (j & 1))));
    }
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Writes the scale byte of K block kb of scale row r (of R rows); the last K
// block also fills the rest of its word with 127.
__device__ __forceinline__ void put_scale(uint8_t* scales, int64_t R, int64_t r, int64_t kb, int64_t nkb, uint32_t byte) {
    uint8_t* w = scales + ((kb >> 2) * R + r) * 4;
    w[kb & 3] = static_cast<uint8_t>(byte);
    if (kb == nkb - 1)
        for (int64_t j = (kb & 3) + 1; j < 4; ++j) w[j] = 127;
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
    uint8_t* __restrict__ scales, uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t, int64_t nkb) {
    __shared__ uint32_t red[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t tl[128 * kPitch];
    const int64_t rt = blockIdx.x / nkb;
    const int64_t ct = blockIdx.x - rt * nkb;
    const int64_t nrb = (rows + 127) >> 7;
    const int64_t kp = (k + 31) & ~static_cast<int64_t>(31), rp = (rows + 31) & ~static_cast<int64_t>(31);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = tid & 15, g = tid >> 4;
    const int64_t r0 = rt * 128 + 8 * g, c0 = ct * 128;

    float v[8][8];
    const bool whole = vec && c0 + col_of<XT>(c, 7) < k;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t off = (r0 + i) * ld;
        if (r0 + i < rows && whole) {
            load_eight<XT>(x, off, c0, c, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t col = c0 + col_of<XT>(c, j);
                v[i][j] = r0 + i < rows && col < k ? load_one<XT>(x, off + col) : 0.0f;
            }
        }
    }

    uint32_t byte_r[8], byte_c[8];
    if constexpr (SQUARE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(v[i][j]));
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) m = umax(m, __shfl_xor(m, s));
        if (lane == 0) red[0][wave] = m;
        __syncthreads();
        m = umax(umax(red[0][0], red[0][1]), umax(red[0][2], red[0][3]));
        const uint32_t b = scale_byte<FMT>(m);
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
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(v[i][j]));
#pragma unroll
                for (int s = 1; s < 16; s <<= 1) m = umax(m, __shfl_xor(m, s));
                byte_r[i] = scale_byte<FMT>(m);
                if (c == 0 && r0 + i < rows) put_scale(scales, rows, r0 + i, ct, nkb, byte_r[i]);
            }
        }
        if (codes_t) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = umax(m, abs_bits(v[i][j]));
                m = umax(m, __shfl_xor(m, 16));
                m = umax(m, __shfl_xor(m, 32));
                if (lane < 16) red[wave][col_of<XT>(c, j)] = m;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int cc = col_of<XT>(c, j);
                byte_c[j] = scale_byte<FMT>(umax(umax(red[0][cc], red[1][cc]), umax(red[2][cc], red[3][cc])));
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
            uint8_t* d = codes + (r0 + i) * kp;
            if constexpr (XT == BSFP8_OUT_F32) {
                if (c0 + 4 * c < kp) *reinterpret_cast<uint32_t*>(d + c0 + 4 * c) = w0;
                if (c0 + 64 + 4 * c < kp) *reinterpret_cast<uint32_t*>(d + c0 + 64 + 4 * c) = w1;
            } else {
                if (c0 + 8 * c < kp) *reinterpret_cast<uint2*>(d + c0 + 8 * c) = make_uint2(w0, w1);
            }
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
    const int64_t nkb = (k + 127) >> 7;
    const dim3 grid(static_cast<uint32_t>(nkb * ((rows + 127) >> 7)));
    if (square)
        hipLaunchKernelGGL((quantize_block128_kernel<XT, FMT, true>), grid, dim3(kThreads), 0, stream, x, rows, k, ld,
                           vec, codes, scales, codes_t, scales_t, nkb);
    else
        hipLaunchKernelGGL((quantize_block128_kernel<XT, FMT, false>), grid, dim3(kThreads), 0, stream, x, rows, k, ld,
                           vec, codes, scales, codes_t, scales_t, nkb);
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
