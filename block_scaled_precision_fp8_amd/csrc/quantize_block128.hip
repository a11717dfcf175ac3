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
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;   // a launch's threads are counted in 32 bits
constexpr int64_t kSmallItems = 16384;

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
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// Maximum over the 16 lanes of a row, in each of them: within quads, then
// mirrored within 8 and within 16 lanes.  Lane moves on the VALU instead of
// shuffles through LDS, and packed 16-bit maxima: 16384 x 4096 bf16 by rows
// 39.4 -> 34.2 us, transposed 49.7 -> 40.3, both 66.8 -> 62.4.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t m) {
    return umax(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), CTRL, 0xF, 0xF, false)));
}
__device__ __forceinline__ uint32_t max16(uint32_t m) {
    return max_dpp<0x140>(max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(m))));
}
// Maximum over the four 16-lane rows of a wave, lane by lane.
__device__ __forceinline__ uint32_t max_rows(uint32_t m) {
    const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = umax(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return umax(b[0], b[1]);
}

// Eight columns of one row, as loaded, and their magnitudes.  16-bit types stay
// packed: two magnitudes per maximum.  Magnitudes order as unsigned integers;
// bits() of one is the FP32 pattern that scale_byte takes.
template <int XT>
struct Eight {
    u4v w;
    typedef uint16_t u2h __attribute__((ext_vector_type(2)));
    __device__ __forceinline__ float operator[](int j) const {
        return from_half_bits<XT>(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
    }
    __device__ __forceinline__ Eight abs() const { return {w & 0x7FFF7FFFu}; }
    __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u2h, a), __builtin_bit_cast(u2h, b)));
    }
    __device__ __forceinline__ void take_max(const Eight& o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = max2(w[i], o.w[i]);
    }
    __device__ __forceinline__ uint32_t magnitude(int j) const { return (w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu; }
    __device__ __forceinline__ uint32_t widest() const {
        const uint32_t m = max2(max2(w[0], w[1]), max2(w[2], w[3]));
        return umax(m & 0xFFFFu, m >> 16);
    }
    __device__ __forceinline__ static uint32_t bits(uint32_t m) {
        return __float_as_uint(from_half_bits<XT>(static_cast<uint16_t>(m)));
    }
};
template <>
struct Eight<BSFP8_OUT_F32> {
    u4v w[2];
    __device__ __forceinline__ float operator[](int j) const { return __uint_as_float(w[j >> 2][j & 3]); }
    __device__ __forceinline__ Eight abs() const { return {{w[0] & 0x7FFFFFFFu, w[1] & 0x7FFFFFFFu}}; }
    __device__ __forceinline__ void take_max(const Eight& o) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j >> 2][j & 3] = umax(w[j >> 2][j & 3], o.w[j >> 2][j & 3]);
    }
    __device__ __forceinline__ uint32_t magnitude(int j) const { return w[j >> 2][j & 3]; }
    __device__ __forceinline__ uint32_t widest() const {
        uint32_t m = w[0][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) m = umax(m, w[j >> 2][j & 3]);
        return m;
    }
    __device__ __forceinline__ static uint32_t bits(uint32_t m) { return m; }
};
// Columns c0 + col_of(c, 0 .. 7) of the row at element offset row: with 16-byte
// loads where all eight exist (whole), else one by one, zeros past k.
template <int XT>
__device__ __forceinline__ Eight<XT> load_eight(const void* x, int64_t row, int64_t c0, int c, int64_t k, bool whole) {
    Eight<XT> v;
    if constexpr (XT == BSFP8_OUT_F32) {
        const float* p = static_cast<const float*>(x) + row + c0 + 4 * c;
        if (whole) {
            v.w[0] = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(p));
            v.w[1] = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(p + 64));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v.w[j >> 2][j & 3] = c0 + col_of<XT>(c, j) < k ? __float_as_uint(p[(j >> 2) * 64 + (j & 3)]) : 0u;
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + row + c0 + 8 * c;
        if (whole) {
            v.w = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(p));
        } else {
            v.w = u4v{0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + 8 * c + j < k) v.w[j >> 1] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
        }
    }
    return v;
}

// The two code words of load_eight's columns, into row d of kp codes.
template <int XT>
__device__ __forceinline__ void put_codes(uint8_t* d, int64_t c0, int64_t kp, int c, uint32_t w0, uint32_t w1) {
    if constexpr (XT == BSFP8_OUT_F32) {
        if (c0 + 4 * c < kp) *reinterpret_cast<uint32_t*>(d + c0 + 4 * c) = w0;
        if (c0 + 64 + 4 * c < kp) *reinterpret_cast<uint32_t*>(d + c0 + 64 + 4 * c) = w1;
    } else {
        if (c0 + 8 * c < kp) *reinterpret_cast<uint2*>(d + c0 + 8 * c) = make_uint2(w0, w1);
    }
}

// Writes the scale byte of K block kb of scale row r (of R rows); the last K
// block also fills the rest of its word with 127.
__device__ __forceinline__ void put_scale(uint8_t* scales, int64_t R, int64_t r, int64_t kb, int64_t nkb, uint32_t byte) {
    uint8_t* w = scales + ((kb >> 2) * R + r) * 4;
    w[kb & 3] = static_cast<uint8_t>(byte);
    if (kb == nkb - 1)
        for (int64_t j = (kb & 3) + 1; j < 4; ++j) w[j] = 127;
}

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
