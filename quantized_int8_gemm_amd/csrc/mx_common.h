// Element types, 8-value loads and stores, and the MX block conversion that
// the norm and the quantiser share.
#pragma once
#include "device_common.h"
#include "mx_kernels.h"

namespace qg {

typedef short v2s __attribute__((ext_vector_type(2)));

// Eight consecutive values as a lane moves them: one 16-byte access for 16-bit
// types, two for fp32.  The copies carry the type's alignment only: gfx950
// takes 16-byte accesses at any byte address, so odd widths and strides run
// the same code.
template <typename T> struct Pack8 { T v[8]; };

template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, Pack8<T>& r) {
    if (left >= 8) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = i < left ? p[i] : (T)0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int left, const Pack8<T>& r) {
    if (left >= 8) {
        __builtin_memcpy(p, &r, sizeof(r));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = r.v[i];
    }
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Bits of |v|: as integers they order like the magnitudes, with infinities
// above every finite value and NaN above those, so one integer maximum finds
// the largest magnitude and whether all values are finite.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t INF_BITS = 0x7f800000u;

// Maximum over the four lanes that share an MX block (quad permutes).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // lanes 1 0 3 2
    return umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// Scale byte of a block whose largest magnitude has these bits.  A subnormal
// maximum has exponent field 0 and takes byte 0, as the clamp asks.
template <bool FP4>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    const int e = (int)(top >> 23) - (FP4 ? 2 : 8);
    return top >= INF_BITS ? 255u : (uint32_t)(e > 0 ? e : 0);
}

// Eight values to MX elements under scale byte b: 4 (e2m1) or 8 bytes (e4m3).
// The hardware conversions divide by the scale's power of two and round to
// nearest even.  e2m1 saturates by itself; e4m3 would turn values past 464
// into NaN, so they are clamped to 448 first.
template <bool FP4>
__device__ __forceinline__ void mx_encode8(const float* v, uint32_t b, uint32_t* w) {
    const float scale = __uint_as_float((b == 255u ? 127u : b) << 23);
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = b == 255u ? 0.f : v[i];
    if constexpr (FP4) {
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, u[0], u[1], scale, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, u[2], u[3], scale, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, u[4], u[5], scale, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, u[6], u[7], scale, 3);
        w[0] = r;
    } else {
        const float top = __uint_as_float(b == 255u ? 0u : ((b + 8u) << 23) | 0x600000u);   // 448 * 2^(b-127)
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __builtin_amdgcn_fmed3f(u[i], -top, top);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            v2s r = {0, 0};
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, u[4 * q], u[4 * q + 1], scale, false);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, u[4 * q + 2], u[4 * q + 3], scale, true);
            w[q] = __builtin_bit_cast(uint32_t, r);
        }
    }
}

// 2^(b - 127), NaN for 255.
__device__ __forceinline__ float mx_factor(uint32_t b) {
    return __uint_as_float(b == 0u ? 0x00400000u : (b == 255u ? 0x7fc00000u : b << 23));
}

}  // namespace qg
