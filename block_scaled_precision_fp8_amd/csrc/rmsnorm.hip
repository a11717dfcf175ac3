// rmsnorm.hip -- root-mean-square norm with the residual's addition, to FP8 codes with
// one power-of-two scale per 1 x 128 block and to 16 or 32 bits, and its gradient (gfx950).
//
//   h = x + residual, rounded to the residual's type     rstd = (mean_k h^2 + eps)^(-1/2)
//   y = (h rstd) w                                       codes and scales: those of y
//
// The norm is taken of the rounded h, the values that a later backward pass reads, so that
// the gradient is that of the function that ran.  y stays in FP32 until it is encoded
// or converted: each output is rounded once.  With g = w dy, xh = h rstd:
//
//   dx = rstd (g - xh mean_k(g xh)) + dh                 dw = sum_rows dy xh
//
// dh being the gradient that reaches h along the residual.  Sums are FP32, in an order that depends on
// k alone (dw's on the rows, too): a lane's eight columns, then trees over lanes and pieces.
//
// A row is held in registers between its two passes, so each input is read once: HBM
// bounds the large calls.  Waves take 512 columns at a time, eight per lane: four blocks of
// 128 (16 lanes each) are one word of scale bytes, and a lane's eight codes one 8-byte store.
#include "block128_codec.h"

namespace bsfp8 {

namespace {

using namespace block128;

constexpr int kWaveColumns = 512;
constexpr int kMaxWaves = 16;
typedef u4v u4u __attribute__((aligned(2)));     // 16 bytes at any element's address
enum { NONE = 0, HALF = 1, WIDE = 2 };           // absent, a 16-bit type, FP32

// Eight elements of a row as loaded.
template <int W>
struct Raw { u4v w[W == WIDE ? 2 : 1]; };

// Elements at .. at + 7 of p, of which n (or all) exist; zeros for the others.
template <int W>
__device__ __forceinline__ Raw<W> load_raw(const void* p, int64_t at, int64_t n) {
    Raw<W> r;
    if constexpr (W == WIDE) {
        const uint32_t* q = static_cast<const uint32_t*>(p) + at;
        if (n >= 8) {
            r.w[0] = __builtin_nontemporal_load(reinterpret_cast<const u4u*>(q));
            r.w[1] = __builtin_nontemporal_load(reinterpret_cast<const u4u*>(q + 4));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r.w[j >> 2][j & 3] = j < n ? q[j] : 0u;
        }
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(p) + at;
        if (n >= 8) {
            r.w[0] = __builtin_nontemporal_load(reinterpret_cast<const u4u*>(q));
        } else {
            r.w[0] = u4v{0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) r.w[0][j >> 1] |= static_cast<uint32_t>(q[j]) << (16 * (j & 1));
        }
    }
    return r;
}
template <int T>
__device__ __forceinline__ void half_values(const u4v& w, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = from_half_bits<T>(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
}
template <int W>
__device__ __forceinline__ void values(const Raw<W>& r, int type, float (&v)[8]) {
    if constexpr (W == WIDE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.w[j >> 2][j & 3]);
    } else if (type == BSFP8_OUT_BF16) {
        half_values<BSFP8_OUT_BF16>(r.w[0], v);
    } else {
        half_values<BSFP8_OUT_F16>(r.w[0], v);
    }
}
template <int T>
__device__ __forceinline__ u4v half_words(const float (&v)[8]) {
    u4v w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = to_half_bits<T>(v[2 * j]) | (static_cast<uint32_t>(to_half_bits<T>(v[2 * j + 1])) << 16);
    return w;
}
template <int W>
__device__ __forceinline__ Raw<W> rounded(const float (&v)[8], int type) {
    Raw<W> r;
    if constexpr (W == WIDE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j >> 2][j & 3] = __float_as_uint(v[j]);
    } else if (type == BSFP8_OUT_BF16) {
        r.w[0] = half_words<BSFP8_OUT_BF16>(v);
    } else {
        r.w[0] = half_words<BSFP8_OUT_F16>(v);
    }
    return r;
}
template <int W>
__device__ __forceinline__ void store_raw(void* p, int64_t at, int64_t n, const Raw<W>& r) {
    if constexpr (W == WIDE) {
        uint32_t* q = static_cast<uint32_t*>(p) + at;
        if (n >= 8) {
            *reinterpret_cast<u4u*>(q) = r.w[0];
            *reinterpret_cast<u4u*>(q + 4) = r.w[1];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) q[j] = r.w[j >> 2][j & 3];
        }
    } else {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        if (n >= 8) {
            *reinterpret_cast<u4u*>(q) = r.w[0];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) q[j] = static_cast<uint16_t>(r.w[0][j >> 1] >> (16 * (j & 1)));
        }
    }
}
// Eight weights (ones without an array), raw: their type is only known here.
__device__ __forceinline__ Raw<WIDE> load_weight(const void* w, int type, int64_t col, int64_t n) {
    Raw<WIDE> r;
    r.w[0] = r.w[1] = u4v{0x3F800000u, 0x3F800000u, 0x3F800000u, 0x3F800000u};
    if (!w) return r;
    if (type == BSFP8_OUT_F32) return load_raw<WIDE>(w, col, n);
    r.w[0] = load_raw<HALF>(w, col, n).w[0];
    return r;
}
__device__ __forceinline__ void weight_values(const Raw<WIDE>& r, bool given, int type, float (&v)[8]) {
    if (given && type != BSFP8_OUT_F32) values<HALF>(Raw<HALF>{{r.w[0]}}, type, v);
    else values<WIDE>(r, type, v);
}

// The sum over the four 16-lane rows of a wave, lane by lane, in each of them.
__device__ __forceinline__ float add_rows(float v) {
    const uint32_t m = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    const uint32_t n = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(n, n, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// The sum over a wave, in each of its lanes: within quads, mirrored within 8 and 16 lanes, across rows.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    return add_rows(add_dpp<0x140>(add_dpp<0x141>(add_dpp<0x4E>(add_dpp<0xB1>(v)))));
}
// v^(-1/2), rounded once (to within 2^-18 of a step): the hardware's estimate r, off by up to a step and not
// made for subnormal v, moved by r (1 - v r^2) / 2, that difference formed from the exact product v r.
// 1 / sqrt(v), which rounds twice, is another value than the nearest one for a quarter of all v.
__device__ __forceinline__ float reciprocal_root(float v) {
    const bool tiny = v < 0x1p-100f;
    const float e = __builtin_amdgcn_rsqf(tiny ? v * 0x1p100f : v), r = tiny ? e * 0x1p50f : e;
    const float t = v * r, low = fmaf(v, r, -t);
    const float off = fmaf(-low, r, fmaf(-t, r, 1.0f));
    // (zero and infinity have theirs already, and NaN stays)
    return r > 0.0f && r < INFINITY ? fmaf(0.5f * r, off, r) : r;
}
// The sum over a row: each piece's 512 columns, then the pieces, both in a tree that is the same however
// pieces are spread over waves, so that a row's results do not depend on how many rows a call has.
// One barrier is enough where calls in turn alternate between two arrays `part`.
constexpr int kMaxPieces = 64;
template <int C>
__device__ __forceinline__ float row_sum(const float (&v)[C], float* part, int wave, int group) {
    const int lane = threadIdx.x & 63;
    if (C == 1 && group == 1) return wave_sum(v[0]);
    part += wave / group * kMaxPieces;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const float s = wave_sum(v[c]);
        if (lane == 0) part[c * group + wave % group] = s;
    }
    __syncthreads();
    return wave_sum(lane < C * group ? part[lane] : 0.0f);
}

struct NormArgs {
    const void* x;
    const void* r;
    const void* w;
    uint8_t* codes;
    uint32_t* scales;
    void* y;
    void* h;
    float* rstd;
    int64_t rows, k, ldx, ldr, ldy, ldh;
    int x_type, h_type, w_type, y_type, group;
    float eps;
};

// X: x's width, R: the residual's, C: pieces of 512 columns per wave.
template <int X, int R, int FMT, int C>
__global__ __launch_bounds__(64 * kMaxWaves) void rmsnorm_kernel(NormArgs a) {
    __shared__ float part[2][4 * kMaxPieces];   // (up to four rows at once)
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = (blockDim.x >> 6) / a.group;     // rows at once
    const int64_t kp = (a.k + 31) & ~static_cast<int64_t>(31);
    const int w0 = wave % a.group;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per;
    int turn = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * per; base < a.rows; base += step, turn ^= 1) {
        const int64_t row = base + wave / a.group;
        const bool in = row < a.rows;
        Raw<X> xr[C];
        Raw<R> rr[C];
        Raw<WIDE> wr[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = static_cast<int64_t>(c * a.group + w0) * kWaveColumns + 8 * lane;
            const int64_t n = in ? a.k - col : 0;
            xr[c] = load_raw<X>(a.x, row * a.ldx + col, n);
            if constexpr (R != NONE) rr[c] = load_raw<R>(a.r, row * a.ldr + col, n);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = static_cast<int64_t>(c * a.group + w0) * kWaveColumns + 8 * lane;
            wr[c] = load_weight(a.w, a.w_type, col, a.k - col);
        }
        float h[C][8], part_sum[C] = {};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = static_cast<int64_t>(c * a.group + w0) * kWaveColumns + 8 * lane;
            values<X>(xr[c], a.x_type, h[c]);
            if constexpr (R != NONE) {
                float q[8];
                values<R>(rr[c], a.h_type, q);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[c][j] += q[j];
                const Raw<R> hr = rounded<R>(h[c], a.h_type);
                values<R>(hr, a.h_type, h[c]);
                if (in) store_raw<R>(a.h, row * a.ldh + col, a.k - col, hr);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) part_sum[c] = fmaf(h[c][j], h[c][j], part_sum[c]);
        }
        const float sum = row_sum<C>(part_sum, part[turn], wave, a.group);
        if (!in) continue;
        const float rstd = reciprocal_root(sum / static_cast<float>(a.k) + a.eps);
        if (a.rstd && w0 == 0 && lane == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int g = c * a.group + w0;
            const int64_t col = static_cast<int64_t>(g) * kWaveColumns + 8 * lane;
            if (static_cast<int64_t>(g) * kWaveColumns >= a.k) break;
            float w[8], y[8];
            weight_values(wr[c], a.w != nullptr, a.w_type, w);
            // (columns past k: zeros, whatever rstd is)
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = col + j < a.k ? (h[c][j] * rstd) * w[j] : 0.0f;
            if (a.y) {
                if (a.y_type == BSFP8_OUT_F32) store_raw<WIDE>(a.y, row * a.ldy + col, a.k - col, rounded<WIDE>(y, a.y_type));
                else store_raw<HALF>(a.y, row * a.ldy + col, a.k - col, rounded<HALF>(y, a.y_type));
            }
            if (a.codes) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = umax(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
                const uint32_t byte = scale_byte<FMT>(max16(m));
                const float f = inverse_scale(byte);
                uint32_t c0 = fp8_pack4<FMT>(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
                uint32_t c1 = fp8_pack4<FMT>(y[4] * f, y[5] * f, y[6] * f, y[7] * f);
                if (byte == 255u) c0 = c1 = kNanCodes;
                if (col < kp) *reinterpret_cast<uint2*>(a.codes + row * kp + col) = make_uint2(c0, c1);
                const uint32_t word = __builtin_amdgcn_readlane(byte, 0) | (__builtin_amdgcn_readlane(byte, 16) << 8) |
                                      (__builtin_amdgcn_readlane(byte, 32) << 16) | (__builtin_amdgcn_readlane(byte, 48) << 24);
                if (lane == 0) a.scales[g * a.rows + row] = word;
            }
        }
    }
}

struct GradArgs {
    const void* dy;
    const void* h;
    const float* rstd;
    const void* w;
    const void* dh;
    void* dx;
    float* partial;              // null: the weight's gradient is not wanted
    int64_t rows, k, ldy, ldh, lda, ldx;
    int dy_type, h_type, w_type, dh_type, group;
};

// Y: dy's width, H: h's and dx's, A: dh's.
template <int Y, int H, int A, int C>
__global__ __launch_bounds__(64 * kMaxWaves) void rmsnorm_grad_kernel(GradArgs a) {
    __shared__ float part[2][4 * kMaxPieces];   // (up to four rows at once)
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = (blockDim.x >> 6) / a.group;
    const int w0 = wave % a.group;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per;
    // With one piece per wave there is room for its weights and for the next row's loads
    // ahead of this one's sum (16384 x 4096 bf16 with dh: 142 -> 97 us, 94 with the sums by lane moves); with more they would spill.
    constexpr bool AHEAD = C == 1;
    float acc[C][8] = {}, w[C][8];
    auto column = [&](int c) { return static_cast<int64_t>(c * a.group + w0) * kWaveColumns + 8 * lane; };
    auto weigh = [&](int c) {
        weight_values(load_weight(a.w, a.w_type, column(c), a.k - column(c)), a.w != nullptr, a.w_type, w[c]);
    };
    if constexpr (AHEAD) weigh(0);
    Raw<Y> yr[C];
    Raw<H> hr[C];
    Raw<A> ar[C];
    float rstd;
    auto fetch = [&](int64_t row) {
        const bool in = row < a.rows;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t n = in ? a.k - column(c) : 0;
            yr[c] = load_raw<Y>(a.dy, row * a.ldy + column(c), n);
            hr[c] = load_raw<H>(a.h, row * a.ldh + column(c), n);
            if constexpr (A != NONE) ar[c] = load_raw<A>(a.dh, row * a.lda + column(c), n);
        }
        rstd = in ? a.rstd[row] : 0.0f;
    };
    int turn = 0;
    int64_t row = static_cast<int64_t>(blockIdx.x) * per + wave / a.group;
    if constexpr (AHEAD) fetch(row);
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * per; base < a.rows; base += step, row += step, turn ^= 1) {
        const bool in = row < a.rows;
        if constexpr (!AHEAD) fetch(row);
        const float r = rstd;
        float part_sum[C] = {};
        float g[C][8], xh[C][8], along[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (!AHEAD) weigh(c);
            values<Y>(yr[c], a.dy_type, g[c]);
            values<H>(hr[c], a.h_type, xh[c]);
            if constexpr (A != NONE) values<A>(ar[c], a.dh_type, along[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // (columns past k: zeros, whatever rstd is)
                const bool there = column(c) + j < a.k;
                xh[c][j] = there ? xh[c][j] * r : 0.0f;
                if (in) acc[c][j] = fmaf(g[c][j], xh[c][j], acc[c][j]);
                g[c][j] = there ? g[c][j] * w[c][j] : 0.0f;
                part_sum[c] = fmaf(g[c][j], xh[c][j], part_sum[c]);
            }
        }
        if (AHEAD && base + step < a.rows) fetch(row + step);
        const float sum = row_sum<C>(part_sum, part[turn], wave, a.group);
        if (!in) continue;
        const float mean = sum / static_cast<float>(a.k);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float dx[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dx[j] = r * fmaf(-xh[c][j], mean, g[c][j]);
                if constexpr (A != NONE) dx[j] += along[c][j];
            }
            store_raw<H>(a.dx, row * a.ldx + column(c), a.k - column(c), rounded<H>(dx, a.h_type));
        }
    }
    if (!a.partial) return;
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * per + wave / a.group) * a.k;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t col = static_cast<int64_t>(c * a.group + w0) * kWaveColumns + 8 * lane;
        store_raw<WIDE>(a.partial, at + col, a.k - col, rounded<WIDE>(acc[c], BSFP8_OUT_F32));
    }
}

// dw[c] (+)= the sum of `count` partial rows: 16 columns per workgroup, each of a column's 64 lanes
// taking every 64th row, eight loads in flight; their sums added as a tree.  (Added one after another
// they left 777 x 5001 FP32 1.6e-7 from the exact gradients, 0.9e-7 so; a sum in FP32 by torch 1.2e-7.)
__global__ __launch_bounds__(64 * kMaxWaves) void column_sum_kernel(const float* __restrict__ partial, int64_t count,
                                                                    int64_t k, int accumulate, float* __restrict__ dw) {
    __shared__ float part[kMaxWaves][16];
    const int c = threadIdx.x & 15, first = threadIdx.x >> 4;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + c;
    float sum = 0.0f;
    if (col < k) {
        const float* p = partial + col;
        int64_t r = first;
        for (; r + 7 * 4 * kMaxWaves < count; r += 8 * 4 * kMaxWaves) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[(r + i * 4 * kMaxWaves) * k];
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
        for (; r < count; r += 4 * kMaxWaves) sum += p[r * k];
    }
    sum = add_rows(sum);                             // over the wave's four
    if ((first & 3) == 0) part[first >> 2][c] = sum;
    __syncthreads();
    if (first >= 4) return;                          // one wave: four sums each, then across its rows
    const float* p = &part[4 * first][c];
    sum = add_rows((p[0] + p[16]) + (p[32] + p[48]));
    if (first == 0 && col < k) dw[col] = accumulate ? dw[col] + sum : sum;
}

// How a row is spread: `pieces` of 512 columns per wave, `group` waves per row, `per`
// rows per workgroup at once, `grid` workgroups.
struct Spread { int pieces, group, per, grid; };

// One piece per wave spreads a row over the most waves, which small calls need; more rows in flight per
// workgroup suit large ones.  bf16 with residual (one piece, two, four): 16 x 8192 5.3, 5.2, 6.8 us; 512 x 4096
// 6.2, 6.3, 8.1; 512 x 8192 12.0, 10.2, 12.1; 1024 x 8192 21.6, 16.2, 16.6; 2048 x 4096 17.2, 16.1, 16.5;
// 16384 x 4096 99.8, 87.5, 94.2; 16384 x 8192 284, 175, 179; of up to 2048 columns 2048 x 2048 10.1, 10.1,
// 12.0, 16384 x 2048 49.0, 43.1, 48.4.  (Two, four): 2048 x 12288 38, 55; 2048 x 16384 60, 55.  Beyond
// 16384 columns a workgroup's 16 waves need four.
Spread norm_spread(int64_t rows, int64_t k) {
    const int n = static_cast<int>((k + kWaveColumns - 1) / kWaveColumns);
    const int pieces = n <= 4 || (n <= kMaxWaves && rows <= 512) ? 1 : n <= 2 * kMaxWaves ? 2 : 4;
    const int group = (n + pieces - 1) / pieces, per = group >= 4 ? 1 : 4 / group;
    const int64_t grid = (rows + per - 1) / per;
    return {pieces, group, per, static_cast<int>(grid < (1 << 20) ? grid : 1 << 20)};
}

Spread grad_spread(int64_t rows, int64_t k) {
    const int n = static_cast<int>((k + kWaveColumns - 1) / kWaveColumns);
    const int pieces = n <= kMaxWaves ? 1 : n <= 2 * kMaxWaves ? 2 : 4;
    const int group = (n + pieces - 1) / pieces, per = group >= 4 ? 1 : 4 / group;
    // Each workgroup writes a partial row of dw: two per CU where rows are many, else one, and as few as
    // give each the same number of rows.  bf16 without dh (256 workgroups, 512): 777 x 4096 12.2, 13.1 us;
    // 2500 x 4096 19.9, 21.4; 3500 x 4096 24.3, 24.6; 4096 x 4096 26.3, 25.1; 16384 x 4096 75.3, 70.7;
    // 16384 x 5001 199, 143.  FP32: 2500 x 5001 45.0, 44.3; 6000 x 5001 94.8, 87.5.  (With 8192 columns and
    // more one per CU stays ahead up to 6000 rows: 6000 x 8192 56, 64.)
    // Pieces as few as fit: two in place of one took 4096 x 4096 from 25 to 36 us, four in place of two
    // 4096 x 12288 from 80 to 179.  With two and more there is no look-ahead, and four spill (58 to 212
    // registers, at the 128 of a workgroup of 16 waves): rows past 8192 columns run, but not near the time of
    // their bytes (1500 x 20001 bf16 131 us, 37 at a copy's rate).
    const int64_t groups = (rows + per - 1) / per, most = rows >= 4096 ? 512 : 256, turns = (groups + most - 1) / most;
    return {pieces, group, per, static_cast<int>(turns ? (groups + turns - 1) / turns : 0)};
}

template <int X, int R, int FMT>
hipError_t launch_norm(const NormArgs& a, const Spread& s, hipStream_t stream) {
    const dim3 grid(s.grid), threads(64 * s.group * s.per);
    if (s.pieces == 1) hipLaunchKernelGGL((rmsnorm_kernel<X, R, FMT, 1>), grid, threads, 0, stream, a);
    else if (s.pieces == 2) hipLaunchKernelGGL((rmsnorm_kernel<X, R, FMT, 2>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((rmsnorm_kernel<X, R, FMT, 4>), grid, threads, 0, stream, a);
    return hipGetLastError();
}

template <int X, int R>
hipError_t launch_norm_fmt(const NormArgs& a, int fmt, const Spread& s, hipStream_t stream) {
    return fmt == BSFP8_E4M3 ? launch_norm<X, R, BSFP8_E4M3>(a, s, stream) : launch_norm<X, R, BSFP8_E5M2>(a, s, stream);
}

template <int Y, int H, int A>
hipError_t launch_grad(const GradArgs& a, const Spread& s, hipStream_t stream) {
    const dim3 grid(s.grid), threads(64 * s.group * s.per);
    if (s.pieces == 1) hipLaunchKernelGGL((rmsnorm_grad_kernel<Y, H, A, 1>), grid, threads, 0, stream, a);
    else if (s.pieces == 2) hipLaunchKernelGGL((rmsnorm_grad_kernel<Y, H, A, 2>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((rmsnorm_grad_kernel<Y, H, A, 4>), grid, threads, 0, stream, a);
    return hipGetLastError();
}

template <int Y, int H>
hipError_t launch_grad_dh(const GradArgs& a, const Spread& s, hipStream_t stream) {
    if (!a.dh) return launch_grad<Y, H, NONE>(a, s, stream);
    return a.dh_type == BSFP8_OUT_F32 ? launch_grad<Y, H, WIDE>(a, s, stream) : launch_grad<Y, H, HALF>(a, s, stream);
}

}  // namespace

hipError_t launch_rmsnorm(const void* x, int x_type, int64_t rows, int64_t k, int64_t ldx, const void* residual,
                          int h_type, int64_t ldr, const void* weight, int w_type, float eps, int fmt, uint8_t* codes,
                          uint8_t* scales, void* y, int y_type, int64_t ldy, void* h, int64_t ldh, float* rstd,
                          hipStream_t stream) {
    const Spread s = norm_spread(rows, k);
    const NormArgs a{x, residual, weight, codes, reinterpret_cast<uint32_t*>(scales), y, h, rstd, rows, k, ldx, ldr,
                     ldy, ldh, x_type, h_type, w_type, y_type, s.group, eps};
    if (x_type == BSFP8_OUT_F32) {
        if (!residual) return launch_norm_fmt<WIDE, NONE>(a, fmt, s, stream);
        return h_type == BSFP8_OUT_F32 ? launch_norm_fmt<WIDE, WIDE>(a, fmt, s, stream)
                                       : launch_norm_fmt<WIDE, HALF>(a, fmt, s, stream);
    }
    if (!residual) return launch_norm_fmt<HALF, NONE>(a, fmt, s, stream);
    return h_type == BSFP8_OUT_F32 ? launch_norm_fmt<HALF, WIDE>(a, fmt, s, stream)
                                   : launch_norm_fmt<HALF, HALF>(a, fmt, s, stream);
}

int64_t rmsnorm_grad_workspace(int64_t rows, int64_t k) {
    const Spread s = grad_spread(rows, k);
    return static_cast<int64_t>(s.grid) * s.per * k * 4;
}

hipError_t launch_rmsnorm_grad(const void* dy, int dy_type, int64_t ldy, const void* h, int h_type, int64_t ldh,
                               const float* rstd, const void* weight, int w_type, const void* dh, int dh_type,
                               int64_t lda, int64_t rows, int64_t k, void* dx, int64_t ldx, float* dweight,
                               int accumulate, void* workspace, hipStream_t stream) {
    const Spread s = grad_spread(rows, k);
    const GradArgs a{dy, h, rstd, weight, dh, dx, dweight ? static_cast<float*>(workspace) : nullptr, rows, k, ldy,
                     ldh, lda, ldx, dy_type, h_type, w_type, dh_type, s.group};
    hipError_t e = hipSuccess;
    if (rows == 0) e = hipSuccess;                   // only the weight's gradient: zeros
    else if (dy_type == BSFP8_OUT_F32)
        e = h_type == BSFP8_OUT_F32 ? launch_grad_dh<WIDE, WIDE>(a, s, stream) : launch_grad_dh<WIDE, HALF>(a, s, stream);
    else
        e = h_type == BSFP8_OUT_F32 ? launch_grad_dh<HALF, WIDE>(a, s, stream) : launch_grad_dh<HALF, HALF>(a, s, stream);
    if (e != hipSuccess || !dweight) return e;
    hipLaunchKernelGGL(column_sum_kernel, dim3(static_cast<uint32_t>((k + 15) / 16)), dim3(64 * kMaxWaves), 0, stream,
                       a.partial, static_cast<int64_t>(s.grid) * s.per, k, accumulate, dweight);
    return hipGetLastError();
}

}  // namespace bsfp8
