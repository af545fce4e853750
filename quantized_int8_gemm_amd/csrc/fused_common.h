// Activations, int8 blocks and the epilogue that the fused A8W8 kernels share.
#pragma once
#include "fused_kernels.h"
#include "mx_common.h"

namespace qg {

// ---------------------------------------------------------------------------
// Activations
// ---------------------------------------------------------------------------

// 1 / (1 + exp(-z)).  The exponential is 2^(z log2 e) with the product rounded to
// fp32, the reciprocal the hardware's: relative error below (|z| + 4) 2^-23.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// The normal distribution's Phi = (1 + erf(z / sqrt 2)) / 2 by density = exp(-z^2 / 2).  With
// a = |z|, t = 1 / (1 + 0.265 a) and w = a t, Phi(-a) = density t P(w): P is the polynomial of
// degree 8 whose largest relative error over 0 .. 16 is least (2.0e-8, found by exchange of its
// extrema).  Past 16 the density is 0.  w, unlike t, keeps its own significand next to zero, where P
// is 1/2 less a multiple of w, so that Phi is off by 3 2^-24 at most there; and no sum of
// like magnitudes cancels for z < 0, where Phi keeps (z^2 + 4) 2^-23 of itself, most of it the
// density's exponent.  (1 + erf in fp32 keeps 2^-24 of 1 there: nothing at all from -5.5 on.)  A
// formula of five terms, to 1.5e-7 of 1: 4096 x 8192 x 2048 forward with a checkpoint and back 255 us,
// 262 with this one; 300 x 5001 x 2048 10.4 and 10.7.
struct NormalTail {
    float t, w, p;
    __device__ __forceinline__ explicit NormalTail(float z) {
        const float a = __builtin_fminf(__builtin_fabsf(z), 16.0f);   // 16 for a NaN, which the density holds
        t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.265f, a, 1.0f));
        w = a * t;
        p = __builtin_fmaf(w, 7.317133849937818e-07f, -9.171379133476876e-06f);
        p = __builtin_fmaf(w, p, 2.353733179916162e-05f);
        p = __builtin_fmaf(w, p, 1.497743214713410e-04f);
        p = __builtin_fmaf(w, p, -3.358556423336267e-04f);
        p = __builtin_fmaf(w, p, -8.980181999504566e-03f);
        p = __builtin_fmaf(w, p, 7.367415726184845e-02f);
        p = __builtin_fmaf(w, p, -2.664422392845154e-01f);
        p = __builtin_fmaf(w, p, 0.5f);
    }
};
__device__ __forceinline__ float normal_density(float z) { return __builtin_amdgcn_exp2f(z * z * -0.72134752f); }   // times sqrt(2 pi)

template <int KIND>
__device__ __forceinline__ float activate(float z) {
    if constexpr (KIND == QG_ACT_RELU) return z < 0.f ? 0.f : z;
    else if constexpr (KIND == QG_ACT_SILU) return z * sigmoid(z);
    else if constexpr (KIND == QG_ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| Phi(-|z|), 3 instructions less than by Phi (4096 x 8192 x 1024 74.5 us,
        // 71.9 so).  The maximum by two exact halves, so that -infinity gives the formula's NaN.
        const NormalTail n(z);
        return __builtin_fmaf(-(n.w * normal_density(z)), n.p, __builtin_fmaf(0.5f, __builtin_fabsf(z), 0.5f * z));
    }
    // tanh y = 2 sigmoid(2 y) - 1; where z^3 passes fp32's range the sigmoid is 0 or 1 all the same
    else if constexpr (KIND == QG_ACT_GELU_TANH) return z * sigmoid(1.59576912f * z * __builtin_fmaf(0.044715f, z * z, 1.0f));
    else return z;
}

// The activation and its derivative at a checkpoint's value.
template <int KIND>
__device__ __forceinline__ void activate_both(float z, float& f, float& slope) {
    f = z;
    slope = 1.f;
    if constexpr (KIND == QG_ACT_RELU) {
        f = z < 0.f ? 0.f : z;
        slope = z > 0.f ? 1.f : (z != z ? z : 0.f);
    } else if constexpr (KIND == QG_ACT_SILU) {
        const float e = sigmoid(z);
        f = z * e;
        slope = __builtin_fmaf(f, 1.0f - e, e);
    } else if constexpr (KIND == QG_ACT_GELU) {
        const NormalTail n(z);
        const float density = normal_density(z), tail = n.p * n.t * density, c = z < 0.f ? tail : 1.0f - tail;
        f = z * c;
        slope = __builtin_fmaf(z * 0.39894228f, density, c);
    } else if constexpr (KIND == QG_ACT_GELU_TANH) {
        const float c = __builtin_amdgcn_fmed3f(z, -32.f, 32.f), sq = c * c;   // past 32 the sigmoid is 0 or 1
        const float e = sigmoid(1.59576912f * c * __builtin_fmaf(0.044715f, sq, 1.0f));
        f = z * e;
        slope = __builtin_fmaf(c * e * (1.0f - e) * 1.59576912f, __builtin_fmaf(0.134145f, sq, 1.0f), e);
        if (z != z) slope = z;   // the clamp drops a NaN
    }
}

// Calls f with the activation as a constant: one branch for a whole group of values.
template <typename F>
__device__ __forceinline__ void with_activation(int kind, F&& f) {
    switch (kind) {
        case QG_ACT_RELU: f(std::integral_constant<int, QG_ACT_RELU>()); break;
        case QG_ACT_SILU: f(std::integral_constant<int, QG_ACT_SILU>()); break;
        case QG_ACT_GELU: f(std::integral_constant<int, QG_ACT_GELU>()); break;
        case QG_ACT_GELU_TANH: f(std::integral_constant<int, QG_ACT_GELU_TANH>()); break;
        default: f(std::integral_constant<int, QG_ACT_NONE>()); break;
    }
}

// ---------------------------------------------------------------------------
// int8 with a shared scale
// ---------------------------------------------------------------------------

// 127 / x and x / 127, correctly rounded, for 2^-100 <= x <= fp32's largest: a
// reciprocal with one Newton step, a quotient and its remainder (P. Markstein, IBM J. Res.
// Dev. 34, 1990), 9 instructions for both where two divisions take 22.  Compared with
// the division for every mantissa of x.
__device__ __forceinline__ float quotient_127(float x) {
    float y = __builtin_amdgcn_rcpf(x);
    y = __builtin_fmaf(__builtin_fmaf(-x, y, 1.0f), y, y);
    const float q = 127.0f * y;
    return __builtin_fmaf(__builtin_fmaf(-x, q, 127.0f), y, q);
}
__device__ __forceinline__ float over_127(float x) {
    const float q = x * 0x1.020408p-7f;
    return __builtin_fmaf(__builtin_fmaf(-127.0f, q, x), 0x1.020408p-7f, q);
}

// The nearest whole number to a |v| < 2^22, ties to even, in the sum's low bits.  v, a product,
// is rounded first: in one instruction with the sum it would not be, and ties fall otherwise.
__device__ __forceinline__ uint32_t nearest_bits(float v) {
#pragma clang fp contract(off)
    return __float_as_uint(v + 12582912.0f);
}

// The low bytes of four words (shift 0) or the next ones (shift 1).
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d, int shift = 0) {
    const uint32_t sel = shift == 0 ? 0x0c0c0400u : 0x0c0c0501u;
    const uint32_t lo = __builtin_amdgcn_perm(b, a, sel), hi = __builtin_amdgcn_perm(d, c, sel);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// From the bits of the largest magnitude: codes are rint((v * up) * inv).  A NaN or an
// infinity makes inv 0, and so do zeros alone: then every code is 0 (a NaN's product with 0
// would keep the NaN's own low bits).
struct Int8Form {
    float inv, scale, up = 1.0f;
    // 2^-100 .. 2^120; outside: zeros, 127 / most not finite or its reciprocal not normal, most not
    // finite.
    __device__ __forceinline__ static bool ordinary(uint32_t top) { return top - 0x0d800000u <= 0x7b800000u - 0x0d800000u; }
    __device__ __forceinline__ explicit Int8Form(uint32_t top) {
        const float most = __uint_as_float(top);
        inv = quotient_127(most);
        scale = over_127(most);
        if (!ordinary(top)) {
            if (most < 1.0f) up = 0x1p60f;
            inv = top == 0u || top >= INF_BITS ? 0.f : 127.0f / (most * up);
            scale = top >= INF_BITS ? __uint_as_float(0x7fc00000u) : top == 0u ? 1.0f : most / 127.0f;
        }
    }
    // Codes of four values, in bytes.
    __device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) const {
        if (up != 1.0f) {
            a *= up;
            b *= up;
            c *= up;
            d *= up;
        }
        const uint32_t w = pack_bytes(nearest_bits(a * inv), nearest_bits(b * inv), nearest_bits(c * inv), nearest_bits(d * inv));
        return inv == 0.f ? 0u : w;
    }
};

// ---------------------------------------------------------------------------
// Four consecutive values of a row
// ---------------------------------------------------------------------------

typedef int v2i_any __attribute__((ext_vector_type(2), aligned(1)));

struct Raw4 { uint32_t w[4]; };

// As they lie in memory, of `count` that exist (the others 0).
__device__ __forceinline__ Raw4 load_raw4(const void* at, int type, int count) {
    Raw4 r = {};
    if (type == QG_FP32) {
        const float* p = reinterpret_cast<const float*>(at);
        if (count >= 4) {
            const v4i_any v = *reinterpret_cast<const v4i_any*>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e) r.w[e] = (uint32_t)v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < count) r.w[e] = __float_as_uint(p[e]);
        }
        return r;
    }
    const uint16_t* p = reinterpret_cast<const uint16_t*>(at);
    if (count >= 4) {
        const v2i_any v = *reinterpret_cast<const v2i_any*>(p);
        r.w[0] = (uint32_t)v[0];
        r.w[1] = (uint32_t)v[1];
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < count) r.w[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    return r;
}

__device__ __forceinline__ v4f values4(const Raw4& r, int type) {
    v4f v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (type == QG_FP32) v[e] = __uint_as_float(r.w[e]);
        else if (type == QG_BF16) v[e] = __uint_as_float(e & 1 ? r.w[e / 2] & 0xffff0000u : r.w[e / 2] << 16);
        else v[e] = half_value(r.w[e / 2], e & 1);
    }
    return v;
}

__device__ __forceinline__ v4f load4(const float* at, int count) { return values4(load_raw4(at, QG_FP32, count), QG_FP32); }

// Rounded once to the type; the first `count` of them.
__device__ __forceinline__ void store4(void* at, int type, int count, v4f v) {
    if (type == QG_FP32) {
        float* p = reinterpret_cast<float*>(at);
        if (count >= 4) {
            v4i_any w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = (int)__float_as_uint(v[e]);
            *reinterpret_cast<v4i_any*>(p) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < count) p[e] = v[e];
        }
        return;
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (type == QG_BF16) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        else w[i] = __builtin_bit_cast(uint32_t, (v2h){(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
    }
    uint16_t* p = reinterpret_cast<uint16_t*>(at);
    if (count >= 4) {
        v2i_any o = {(int)w[0], (int)w[1]};
        *reinterpret_cast<v2i_any*>(p) = o;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < count) p[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
}

// ---------------------------------------------------------------------------
// The epilogue
// ---------------------------------------------------------------------------

// Where four columns of a row go.
struct Goes {
    void* out;
    int8_t* code[2];
    float* scale[2];   // of the block that starts here
    bool starts;
};

__device__ __forceinline__ int size_of(int type) { return type == QG_FP32 ? 4 : 2; }

// From row m and column n of the output.
template <bool PAIR>
__device__ __forceinline__ Goes goes_to(const Epilogue& e, int64_t m, int n) {
    Goes g{};
    g.out = reinterpret_cast<char*>(e.out) + (m * e.ldo + n) * size_of(e.out_type);
    g.starts = n % INT8_BLOCK == 0;
#pragma unroll
    for (int h = 0; h < (PAIR ? 2 : 1); ++h) {
        g.code[h] = e.ckpt[h] + (m * e.ld_ckpt + n);
        g.scale[h] = e.ckpt_scale[h] + (m * e.ld_ckpt_scale + n / INT8_BLOCK);
    }
    return g;
}

// U times four columns of a row, `count` of them there (none or less: a row or columns
// outside): z0 (and z1 of a pair) the scaled products, res the residual as it lies.  FULL: all
// four are.  Several at once hide each other's latencies (one a time, the epilogue of a
// 4096 x 8192 x 2048 product with GELU and a checkpoint took 50 of 108 us).  With a checkpoint,
// eight lanes in a row from a multiple of eight hold one block of 32 columns, and all lanes of
// a wave have to be here, those outside the matrix too.  Each step rounds by itself: the
// checkpoint's codes are defined by these steps.
template <bool PAIR, bool FULL, int U>
__device__ __forceinline__ void finish(const Epilogue& e, const Goes* to, const int* counts, v4f* z0, const v4f* z1, v4f bias, const Raw4* res) {
#pragma clang fp contract(off)
    if (!PAIR && e.bias != nullptr) {
#pragma unroll
        for (int u = 0; u < U; ++u) z0[u] = z0[u] + bias;
    }
    if (e.ckpt[0] != nullptr) {
#pragma unroll
        for (int h = 0; h < (PAIR ? 2 : 1); ++h) {
            uint32_t top[U], w[U];
            float scale[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const v4f z = h == 0 ? z0[u] : z1[u];
                top[u] = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) top[u] = umax(top[u], FULL || i < counts[u] ? abs_bits(z[i]) : 0u);
                top[u] = quad_max(top[u]);
                top[u] = umax(top[u], (uint32_t)__builtin_amdgcn_mov_dpp((int)top[u], 0x141, 0xF, 0xF, true));   // the other four of eight
            }
            bool plain = true;
#pragma unroll
            for (int u = 0; u < U; ++u) plain = plain && Int8Form::ordinary(top[u]);
            if (__builtin_amdgcn_ballot_w64(!plain) == 0ull) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const v4f z = h == 0 ? z0[u] : z1[u];
                    const float inv = quotient_127(__uint_as_float(top[u]));
                    scale[u] = over_127(__uint_as_float(top[u]));
                    w[u] = pack_bytes(nearest_bits(z[0] * inv), nearest_bits(z[1] * inv), nearest_bits(z[2] * inv), nearest_bits(z[3] * inv));
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const v4f z = h == 0 ? z0[u] : z1[u];
                    const Int8Form f(top[u]);
                    scale[u] = f.scale;
                    w[u] = f.codes(z[0], z[1], z[2], z[3]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (FULL || counts[u] >= 4) {
                    __builtin_memcpy(to[u].code[h], &w[u], 4);
                } else {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (i < counts[u]) to[u].code[h][i] = (int8_t)(w[u] >> (8 * i));
                }
            }
            if (to[0].starts) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (FULL || counts[u] > 0) *to[u].scale[h] = scale[u];
            }
        }
    }
    v4f y[U];
    with_activation(e.activation, [&](auto kind) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[u][i] = activate<decltype(kind)::value>(z0[u][i]);
    });
    if constexpr (PAIR) {
#pragma unroll
        for (int u = 0; u < U; ++u) y[u] = y[u] * z1[u];
    } else if (e.res != nullptr) {
#pragma unroll
        for (int u = 0; u < U; ++u) y[u] = y[u] + values4(res[u], e.out_type);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (FULL || counts[u] > 0) store4(to[u].out, e.out_type, FULL ? 4 : counts[u], y[u]);
}

// The same from the int32 sums of row m, columns n .. n + 3, for kernels whose lanes have one item
// each; sums of a gradient's planes hi and lo give its value.
template <int FORM>
__device__ __forceinline__ void finish_sums(const Epilogue& e, int m, int n, int count, const v4i* s, float as, const v4f* ws, v4f bias,
                                            const Raw4& res) {
    constexpr bool PAIR = FORM == FUSED_PAIR;
    const Goes to = goes_to<PAIR>(e, m, n);
    v4f z[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if constexpr (FORM == FUSED_GRAD) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[0][i] = __builtin_fmaf((float)s[0][i], 256.f, (float)s[1][i]) * as;
        if (count > 0) store4(to.out, e.out_type, count, z[0]);
    } else {
#pragma unroll
        for (int h = 0; h < (PAIR ? 2 : 1); ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[h][i] = (float)s[h][i] * as * ws[h][i];
        finish<PAIR, false, 1>(e, &to, &count, &z[0], &z[1], bias, &res);
    }
}

// Where columns 4 c4 .. of a row lie in a tile of sums with C columns in LDS: the 16 rows that a
// fragment's store touches, 64 / C to 256 bytes, take distinct places (64 x 32 gated workgroups
// lost 5 us where they did not).
template <int C>
__device__ __forceinline__ int sums_at(int row, int c4) {
    return row * C + ((c4 ^ ((row / (64 / C)) & (C / 4 - 1))) << 2);
}

}  // namespace qg
