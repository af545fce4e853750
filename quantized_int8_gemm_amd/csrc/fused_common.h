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

// The argument of GELU_TANH's sigmoid (tanh y = 2 sigmoid(2 y) - 1): 2 sqrt(2 / pi) (z +
// 0.044715 z^3).  Past 32 the sigmoid is 0 or 1 to the last bit, and z^3 could pass
// fp32's range.
__device__ __forceinline__ float gelu_tanh_arg(float z, float& square) {
    const float c = __builtin_amdgcn_fmed3f(z, -32.f, 32.f);
    square = c * c;
    return 1.59576912f * c * __builtin_fmaf(0.044715f, square, 1.0f);
}

template <int KIND>
__device__ __forceinline__ float activate(float z) {
    if constexpr (KIND == QG_ACT_RELU) return z < 0.f ? 0.f : z;
    else if constexpr (KIND == QG_ACT_SILU) return z * sigmoid(z);
    else if constexpr (KIND == QG_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    else if constexpr (KIND == QG_ACT_GELU_TANH) {
        float sq;
        const float s = sigmoid(gelu_tanh_arg(z, sq));
        return z != z ? z : z * s;   // the clamp drops a NaN
    } else return z;
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
        slope = e * (1.0f + z * (1.0f - e));
    } else if constexpr (KIND == QG_ACT_GELU) {
        const float c = 0.5f * (1.0f + erff(z * 0.70710678f));
        f = z * c;
        slope = c + z * 0.39894228f * __builtin_amdgcn_exp2f(z * z * -0.72134752f);
    } else if constexpr (KIND == QG_ACT_GELU_TANH) {
        float sq;
        const float e = sigmoid(gelu_tanh_arg(z, sq));
        const float c = __builtin_amdgcn_fmed3f(z, -32.f, 32.f);
        f = z * e;
        slope = e + c * e * (1.0f - e) * 1.59576912f * __builtin_fmaf(0.134145f, sq, 1.0f);
        if (z != z) slope = z;
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

// From the bits of the largest magnitude: codes are rint((v * up) * inv).
struct Int8Form {
    float up, inv, scale;
    bool bad;
    __device__ __forceinline__ explicit Int8Form(uint32_t top) {
        const float most = __uint_as_float(top);
        bad = top >= INF_BITS;
        up = 1.0f;
        inv = quotient_127(most);
        scale = over_127(most);
        if (most < 0x1p-100f || most > 0x1p120f) {   // rare: 127 / most would not be finite, or its reciprocal not normal
            up = most < 1.0f ? 0x1p60f : 1.0f;
            inv = top == 0u ? 0.f : 127.0f / (most * up);
            scale = top == 0u ? 1.0f : most / 127.0f;
        }
        if (bad) {
            inv = 0.f;
            scale = __uint_as_float(0x7fc00000u);
        }
    }
    __device__ __forceinline__ uint32_t code(float v) const {
        const float t = bad ? 0.f : (v * up) * inv;
        return (uint32_t)(int)__builtin_rintf(t) & 0xffu;
    }
};

// ---------------------------------------------------------------------------
// Four consecutive values of a row
// ---------------------------------------------------------------------------

typedef int v2i_any __attribute__((ext_vector_type(2), aligned(1)));

struct Raw4 { uint32_t w[4]; };

// As they lie in memory, of `count` that exist (the others 0).
__device__ __forceinline__ Raw4 load_raw4(const void* base, int64_t at, int type, int count) {
    Raw4 r = {};
    if (type == QG_FP32) {
        const float* p = reinterpret_cast<const float*>(base) + at;
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
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
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

__device__ __forceinline__ v4f load4(const void* base, int64_t at, int type, int count) {
    return values4(load_raw4(base, at, type, count), type);
}

// Rounded once to the type; the first `count` of them.
__device__ __forceinline__ void store4(void* base, int64_t at, int type, int count, v4f v) {
    if (type == QG_FP32) {
        float* p = reinterpret_cast<float*>(base) + at;
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
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
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

// Four columns n .. n + 3 of row m, z0 (and z1 of a pair) the scaled products, res the
// residual as it lies.  With a
// checkpoint, eight lanes in a row from a multiple of eight hold one block of 32
// columns, and all lanes of a wave have to be here, those outside the matrix too.
// Each step rounds by itself: the checkpoint's codes are defined by these steps.
template <bool PAIR>
__device__ __forceinline__ void finish4(const Epilogue& e, int m, int n, v4f z0, v4f z1, v4f bias, const Raw4& res) {
#pragma clang fp contract(off)
    const bool live = m < e.M && n < e.N;
    const int count = live ? e.N - n : 0;
    if (!PAIR && e.bias != nullptr) z0 = z0 + bias;
    if (e.ckpt[0] != nullptr) {
#pragma unroll
        for (int h = 0; h < (PAIR ? 2 : 1); ++h) {
            const v4f z = h == 0 ? z0 : z1;
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = umax(top, i < count ? abs_bits(z[i]) : 0u);
            top = quad_max(top);
            top = umax(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x141, 0xF, 0xF, true));   // the other four of eight
            const Int8Form f(top);
            uint32_t w = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) w |= f.code(z[i]) << (8 * i);
            if (live) {
                int8_t* p = e.ckpt[h] + (int64_t)m * e.ld_ckpt + n;
                if (count >= 4) {
                    __builtin_memcpy(p, &w, 4);
                } else {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (i < count) p[i] = (int8_t)(w >> (8 * i));
                }
                if (n % INT8_BLOCK == 0) e.ckpt_scale[h][(int64_t)m * e.ld_ckpt_scale + n / INT8_BLOCK] = f.scale;
            }
        }
    }
    if (!live) return;
    v4f y;
    with_activation(e.activation, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = activate<decltype(kind)::value>(z0[i]);
    });
    if constexpr (PAIR) y = y * z1;
    if (!PAIR && e.res != nullptr) y = y + values4(res, e.out_type);
    store4(e.out, (int64_t)m * e.ldo + n, e.out_type, count, y);
}

}  // namespace qg
