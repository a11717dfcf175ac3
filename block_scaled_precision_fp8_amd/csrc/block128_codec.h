// block128_codec.h -- the pieces of FP8 quantisation with one power-of-two scale per
// 128 elements that its kernels share: eight values per lane, their magnitudes' maxima
// over a block, the scale byte, and where codes and scale bytes go (gfx950).
#pragma once

#include "fp8_codec.h"

namespace bsfp8 {
namespace block128 {

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

}  // namespace block128
}  // namespace bsfp8
