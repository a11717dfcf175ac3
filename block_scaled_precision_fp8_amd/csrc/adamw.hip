// adamw.hip -- one AdamW step over many tensors, states in FP32 or in FP8 (gfx950).
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,
//   p' = (1 - lr wd) p - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
//
// One pass: every element is read once and written once.  Each operation is
// rounded to FP32 by itself (no contraction to FMAs), so that the result does
// not depend on what a compiler fuses.
//
// FP8 states are E4M3 codes with one E8M0 scale per 128 elements: of m, and of
// r = sqrt(v), whose range of exponents is half that of v.  They are rounded
// stochastically.  Rounding to nearest would freeze them: beta2 = 0.999 moves r
// by at most 0.05% of itself per step where the gradients shrink, against half
// a code step of 3 to 6%.  The random bits come from a hash of (seed, step,
// tensor) and the index of a group of 8 elements, advanced by one xorshift per
// element: about 8 integer operations an element, no state and no traffic.
//
// The tensors' addresses and sizes go by value in the kernel's arguments: no
// copy to the device, nothing to keep alive, and a launch can be captured.
#include "fp8_codec.h"

#include <math.h>

namespace bsfp8 {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                          // elements per thread: one random group
constexpr int kUnit = kThreads * kPer;           // elements per workgroup
constexpr int kTensors = 48;                     // per launch: 48 x 72 bytes of the 4 KB of arguments
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;   // a launch's threads are counted in 32 bits

struct Entry {
    void* p;
    const void* g;
    void* m;
    void* v;
    uint8_t* ms;
    uint8_t* vs;
    int64_t n;
    int64_t start;       // first element of this launch
    uint32_t first;      // first workgroup
    uint32_t index;      // position in the call, and bit 31: 16-byte loads are allowed
};
struct Table {
    Entry e[kTensors];
    int count;
};
struct Constants {
    float b1, c1, b2, c2, decay, size, rbc, eps;
    uint32_t key;        // of (seed, step)
};
struct Dynamic {
    const float* lr;
    const int64_t* step;
    const float* grad_scale;
    const float* found_inf;
    double lr0, beta1, beta2, weight_decay;
    int64_t step0;
    uint32_t seed;
};

// The 32-bit finalizer of MurmurHash3 (Austin Appleby, public domain).
__host__ __device__ inline uint32_t mix(uint32_t h) {
    h ^= h >> 16;
    h *= 0x85EBCA6Bu;
    h ^= h >> 13;
    h *= 0xC2B2AE35u;
    return h ^ (h >> 16);
}
// Marsaglia's 32-bit xorshift generator, shifts 13, 17, 5.
__device__ __forceinline__ uint32_t xorshift(uint32_t s) {
    s ^= s << 13;
    s ^= s >> 17;
    return s ^ (s << 5);
}

__host__ __device__ inline void set_rates(Constants& c, double lr, double beta1, double beta2, double wd, int64_t step,
                                          uint32_t seed) {
    // 1 - lr wd with the product rounded by itself, as the host does: contracted to an
    // FMA on the device, a rate there and the same rate as an argument could differ
#pragma clang fp contract(off)
    const double t = static_cast<double>(step);
    c.decay = static_cast<float>(1.0 - lr * wd);
    c.size = static_cast<float>(lr / (1.0 - pow(beta1, t)));
    c.rbc = static_cast<float>(1.0 / sqrt(1.0 - pow(beta2, t)));
    c.key = mix(mix(seed) ^ static_cast<uint32_t>(step));
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// E8M0 byte of a block whose largest |x| has the bit pattern amax (E4M3).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    if (amax == 0) return 127u;
    if (amax >= 0x7F800000u) return 255u;
    const int b = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(b < 0 ? 0 : b);
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
}

// The E4M3 code of x times the exact power of two f (|x f| <= 448), rounded up
// where its bits below the code, cut to 20, carry when 16 b is added.
__device__ __forceinline__ uint32_t encode(float x, float f, uint32_t b16) {
    const uint32_t y = __float_as_uint(x * f);
    const uint32_t a = y & 0x7FFFFFFFu;
    // normal codes keep the exponent (rebiased by 120) and 3 fraction bits;
    // below 2^-6 the step is 2^-9, and a value in units of 2^-29 lines up the same way
    const uint32_t normal = a - (120u << 23);
    const uint32_t small = static_cast<uint32_t>(__uint_as_float(a) * 0x1p29f);
    const uint32_t t = ((a >= (121u << 23) ? normal : small) + b16) >> 20;
    return t | ((y >> 24) & 0x80u);
}

template <int T>
__device__ __forceinline__ float get(const void* p, int64_t i) {
    if constexpr (T == BSFP8_OUT_F32) return static_cast<const float*>(p)[i];
    else return from_half_bits<T>(static_cast<const uint16_t*>(p)[i]);
}
// eight elements at i, 16-byte aligned
template <int T>
__device__ __forceinline__ void get8(const void* p, int64_t i, float (&x)[8]) {
    if constexpr (T == BSFP8_OUT_F32) {
        const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[0];
        const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = from_half_bits<T>(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
    }
}
__device__ __forceinline__ void put8(float* p, int64_t i, const float (&x)[8]) {
    reinterpret_cast<float4*>(p + i)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p + i)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

template <int PT, int GT, bool FP8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Table table, Constants c, Dynamic dyn) {
#pragma clang fp contract(off)
    if (dyn.found_inf && *dyn.found_inf != 0.0f) return;
    const int tid = threadIdx.x;
    if (dyn.step || dyn.lr) {
        // rates that live on the device: formed once per workgroup
        __shared__ Constants shared;
        if (tid == 0) {
            const double lr = dyn.lr ? static_cast<double>(*dyn.lr) : dyn.lr0;
            shared = c;
            set_rates(shared, lr, dyn.beta1, dyn.beta2, dyn.weight_decay, dyn.step ? *dyn.step : dyn.step0, dyn.seed);
        }
        __syncthreads();
        c = shared;
    }
    // this workgroup's tensor: the last whose first workgroup is not after it
    int lo = 0, hi = table.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table.e[mid].first <= blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const Entry& t = table.e[lo];
    const int64_t n = t.n;
    const int64_t base = t.start + static_cast<int64_t>(blockIdx.x - t.first) * kUnit;
    const int64_t i0 = base + tid * kPer;
    const bool whole = (t.index >> 31) && base + kUnit <= n;
    const float gs = dyn.grad_scale ? *dyn.grad_scale : 1.0f;

    float p[8], g[8], m[8], r[8];
    if (whole) {
        get8<PT>(t.p, i0, p);
        get8<GT>(t.g, i0, g);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = i0 + j < n ? get<PT>(t.p, i0 + j) : 0.0f;
            g[j] = i0 + j < n ? get<GT>(t.g, i0 + j) : 0.0f;
        }
    }
    if constexpr (FP8) {
        uint2 cm = make_uint2(0, 0), cv = make_uint2(0, 0);
        uint32_t bm = 127, bv = 127;
        if (whole) {
            cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i0);
            cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i0);
        } else {
            uint32_t wm[2] = {0, 0}, wv[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + j < n) {
                    wm[j >> 2] |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.m)[i0 + j]) << (8 * (j & 3));
                    wv[j >> 2] |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[i0 + j]) << (8 * (j & 3));
                }
            cm = make_uint2(wm[0], wm[1]);
            cv = make_uint2(wv[0], wv[1]);
        }
        if (i0 < n) {
            bm = t.ms[i0 >> 7];
            bv = t.vs[i0 >> 7];
        }
        const float fm = scale_value(bm), fv = scale_value(bv);
        const uint32_t wm[2] = {cm.x, cm.y}, wv[2] = {cv.x, cv.y};
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(wm[j >> 2], false);
            const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(wm[j >> 2], true);
            const auto d = __builtin_amdgcn_cvt_pk_f32_fp8(wv[j >> 2], false);
            const auto e = __builtin_amdgcn_cvt_pk_f32_fp8(wv[j >> 2], true);
            m[j] = a[0] * fm; m[j + 1] = a[1] * fm; m[j + 2] = b[0] * fm; m[j + 3] = b[1] * fm;
            r[j] = d[0] * fv; r[j + 1] = d[1] * fv; r[j + 2] = e[0] * fv; r[j + 3] = e[1] * fv;
        }
    } else if (whole) {
        get8<BSFP8_OUT_F32>(t.m, i0, m);
        get8<BSFP8_OUT_F32>(t.v, i0, r);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = i0 + j < n ? static_cast<const float*>(t.m)[i0 + j] : 0.0f;
            r[j] = i0 + j < n ? static_cast<const float*>(t.v)[i0 + j] : 0.0f;
        }
    }

    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float gj = g[j] * gs;
        const float v0 = FP8 ? r[j] * r[j] : r[j];
        m[j] = c.b1 * m[j] + c.c1 * gj;
        v[j] = c.b2 * v0 + (c.c2 * gj) * gj;
        r[j] = sqrtf(v[j]);
        p[j] = p[j] * c.decay - (c.size * m[j]) / (r[j] * c.rbc + c.eps);
    }

    // 32 random bits per element; a launch that rounds nothing leaves them unused
    uint32_t bits[8];
    {
        const int64_t q = i0 >> 3;
        const uint32_t key = mix(c.key ^ (t.index & 0x7FFFFFFFu));
        bits[0] = mix(static_cast<uint32_t>(q) * 0x9E3779B1u + key) | 1u;
#pragma unroll
        for (int j = 1; j < 8; ++j) bits[j] = xorshift(bits[j - 1]);
    }

    if constexpr (PT == BSFP8_OUT_F32) {
        if (whole) {
            put8(static_cast<float*>(t.p), i0, p);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + j < n) static_cast<float*>(t.p)[i0 + j] = p[j];
        }
    } else {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // infinities and NaN keep their upper half (a NaN stays one)
            const uint32_t w = __float_as_uint(p[j]);
            const bool odd = (w & 0x7FFFFFFFu) >= 0x7F800000u;
            h[j] = (odd ? w | ((w & 0xFFFFu) != 0 ? 0x400000u : 0u) : w + (bits[j] & 0xFFFFu)) >> 16;
        }
        uint16_t* d = static_cast<uint16_t*>(t.p) + i0;
        if (whole) {
            *reinterpret_cast<uint4*>(d) = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                                                      h[6] | (h[7] << 16));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + j < n) d[j] = static_cast<uint16_t>(h[j]);
        }
    }

    if constexpr (FP8) {
        // the 16 lanes of a block of 128 agree on its scales
        uint32_t am = 0, ar = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = whole || i0 + j < n;
            am = umax(am, in ? __float_as_uint(m[j]) & 0x7FFFFFFFu : 0u);
            ar = umax(ar, in ? __float_as_uint(r[j]) & 0x7FFFFFFFu : 0u);
        }
#pragma unroll
        for (int s = 1; s < 16; s <<= 1) {
            am = umax(am, __shfl_xor(am, s));
            ar = umax(ar, __shfl_xor(ar, s));
        }
        const uint32_t bm = scale_byte(am), bv = scale_byte(ar);
        const float fm = __uint_as_float((254u - bm) << 23), fv = __uint_as_float((254u - bv) << 23);
        uint32_t wm[2] = {0, 0}, wv[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t a = encode(m[j], fm, (bits[j] & 0xFFFFu) << 4);
            uint32_t b = encode(r[j], fv, (bits[j] >> 16) << 4);
            // r' > 0 keeps a code: a zero would let m / (0 + eps) explode
            if (b == 0 && r[j] > 0.0f) b = 1;
            wm[j >> 2] |= (bm == 255u ? 0x7Fu : a) << (8 * (j & 3));
            wv[j >> 2] |= (bv == 255u ? 0x7Fu : b) << (8 * (j & 3));
        }
        uint8_t* dm = static_cast<uint8_t*>(t.m) + i0;
        uint8_t* dv = static_cast<uint8_t*>(t.v) + i0;
        if (whole) {
            *reinterpret_cast<uint2*>(dm) = make_uint2(wm[0], wm[1]);
            *reinterpret_cast<uint2*>(dv) = make_uint2(wv[0], wv[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + j < n) {
                    dm[j] = static_cast<uint8_t>(wm[j >> 2] >> (8 * (j & 3)));
                    dv[j] = static_cast<uint8_t>(wv[j >> 2] >> (8 * (j & 3)));
                }
        }
        if ((tid & 15) == 0 && i0 < n) {
            t.ms[i0 >> 7] = static_cast<uint8_t>(bm);
            t.vs[i0 >> 7] = static_cast<uint8_t>(bv);
        }
    } else if (whole) {
        put8(static_cast<float*>(t.m), i0, m);
        put8(static_cast<float*>(t.v), i0, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i0 + j < n) {
                static_cast<float*>(t.m)[i0 + j] = m[j];
                static_cast<float*>(t.v)[i0 + j] = v[j];
            }
    }
}

template <int PT, int GT>
void launch_state(int state, uint32_t grid, hipStream_t stream, const Table& t, const Constants& c, const Dynamic& d) {
    if (state == BSFP8_STATE_FP8)
        hipLaunchKernelGGL((adamw_kernel<PT, GT, true>), dim3(grid), dim3(kThreads), 0, stream, t, c, d);
    else
        hipLaunchKernelGGL((adamw_kernel<PT, GT, false>), dim3(grid), dim3(kThreads), 0, stream, t, c, d);
}
template <int PT>
void launch_grad(int g_type, int state, uint32_t grid, hipStream_t stream, const Table& t, const Constants& c,
                 const Dynamic& d) {
    if (g_type == BSFP8_OUT_F32) launch_state<PT, BSFP8_OUT_F32>(state, grid, stream, t, c, d);
    else if (g_type == BSFP8_OUT_BF16) launch_state<PT, BSFP8_OUT_BF16>(state, grid, stream, t, c, d);
    else launch_state<PT, BSFP8_OUT_F16>(state, grid, stream, t, c, d);
}

}  // namespace

hipError_t launch_adamw(const bsfp8_adamw_tensor* tensors, int64_t count, int p_type, int g_type, int state,
                        const bsfp8_adamw_args& args, hipStream_t stream) {
    Constants c{};
    c.b1 = static_cast<float>(args.beta1);
    c.c1 = static_cast<float>(1.0 - args.beta1);
    c.b2 = static_cast<float>(args.beta2);
    c.c2 = static_cast<float>(1.0 - args.beta2);
    c.eps = static_cast<float>(args.eps);
    set_rates(c, args.lr, args.beta1, args.beta2, args.weight_decay, args.step, args.seed);
    const Dynamic d{args.lr_dev, args.step_dev, args.grad_scale, args.found_inf, args.lr, args.beta1, args.beta2,
                    args.weight_decay, args.step, args.seed};
    Table t{};
    int64_t grid = 0;
    auto flush = [&]() -> hipError_t {
        if (t.count == 0) return hipSuccess;
        if (p_type == BSFP8_OUT_F32) launch_grad<BSFP8_OUT_F32>(g_type, state, static_cast<uint32_t>(grid), stream, t, c, d);
        else launch_grad<BSFP8_OUT_BF16>(g_type, state, static_cast<uint32_t>(grid), stream, t, c, d);
        t.count = 0;
        grid = 0;
        return hipGetLastError();
    };
    for (int64_t i = 0; i < count; ++i) {
        const bsfp8_adamw_tensor& x = tensors[i];
        const int64_t units = (x.n + kUnit - 1) / kUnit;
        auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
        const uint32_t wide = at16(x.p) && at16(x.g) && at16(x.m) && at16(x.v) ? 0x80000000u : 0u;
        for (int64_t u = 0; u < units;) {
            if (t.count == kTensors || grid == kMaxGroups) {
                const hipError_t e = flush();
                if (e != hipSuccess) return e;
            }
            const int64_t take = units - u < kMaxGroups - grid ? units - u : kMaxGroups - grid;
            t.e[t.count++] = Entry{x.p, x.g, x.m, x.v, x.m_scales, x.v_scales, x.n, u * kUnit,
                                   static_cast<uint32_t>(grid), static_cast<uint32_t>(i) | wide};
            grid += take;
            u += take;
        }
    }
    return flush();
}

}  // namespace bsfp8
