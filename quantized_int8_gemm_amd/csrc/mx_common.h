// Element types, 8-value loads and stores, and the MX block conversion that
// the norm and the quantiser share.
#pragma once
#include <type_traits>

#include "device_common.h"
#include "mx_kernels.h"

namespace qg {

typedef short v2s __attribute__((ext_vector_type(2)));

// Eight consecutive values as a lane moves them: one 16-byte access for 16-bit
// types, two for fp32.  The accesses carry no alignment: gfx950 takes 16-byte
// ones at any byte address, so odd widths and strides run the same code.  The
// values stay packed in dwords until they are used: as single 16-bit elements
// they would take a register each.
template <typename T> struct Pack8 { uint32_t w[2 * sizeof(T)]; };
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(1)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// One half of a dword as a float: v * 1 - 0, exact for every value.  From vector
// elements the compiler shifts high halves down first and keeps halves apart in
// registers (gradient 3691 x 4096 fp16 44.7 us so, 28.1 with this; norm 4000 x 8192 fp16
// to int8 44.8 and 41.0).
__device__ __forceinline__ float half_value(uint32_t pair, bool high) {
    float v;
    if (high) asm("v_fma_mix_f32 %0, %1, 1.0, neg(0) op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(v) : "v"(pair));
    else asm("v_fma_mix_f32 %0, %1, 1.0, neg(0) op_sel_hi:[1,0,0]" : "=v"(v) : "v"(pair));
    return v;
}

template <typename T>
__device__ __forceinline__ float value(const Pack8<T>& p, int e) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(p.w[e]);
    else if constexpr (std::is_same<T, __bf16>::value) return __uint_as_float(e & 1 ? p.w[e / 2] & 0xffff0000u : p.w[e / 2] << 16);
    else return half_value(p.w[e / 2], e & 1);
}

// Eight values rounded once to T.
template <typename T>
__device__ __forceinline__ Pack8<T> pack(const float* v) {
    Pack8<T> p;
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); ++i) {
        if constexpr (sizeof(T) == 4) p.w[i] = __float_as_uint(v[i]);
        else if constexpr (std::is_same<T, __bf16>::value) p.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        else p.w[i] = __builtin_bit_cast(uint32_t, (v2h){(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
    }
    return p;
}

// Rows that start at multiples of a cache line's 128 bytes.
inline bool whole_lines(const void* p, int64_t stride) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride) & 127) == 0;
}

// Values c .. c + 7 of a row of n, those past its end zero.  A row of eight or
// more is read by whole groups only: the one that would pass the end starts at
// n - 8 instead and its values move down, so every lane does one load and only
// the last group's wave a few instructions more.  TINY: rows of less than eight.
// NT: with the non-temporal policy, for what is read once (norm to int8 8192 x
// 8192 83.6 -> 73.6 us, gradient 8192 x 4096 52.2 -> 49.7; stores gain nothing
// by it, and the next kernel reads what they leave).  Only where every row is
// whole_lines: a line that two reads share is then fetched twice (norm to MXFP8,
// 1537 x 5000 fp16, 10.8 us without and 11.4 with it).
// Not for fp32, whose group of eight is two loads of the same lines (norm to int8 1024 x
// 8192 19.2 us, 24.5 with it; 8192 x 8192 155 and 170; gradient 512 x 12288 25.3 and 29.4).
template <bool TINY, bool NT = false, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int n, Pack8<T>& r) {
    constexpr int W = 2 * sizeof(T);
    if constexpr (TINY) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(T) == 4) {
                r.w[i] = c + i < n ? reinterpret_cast<const uint32_t*>(row)[c + i] : 0u;
            } else {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(row) + c;
                r.w[i] = (c + 2 * i < n ? (uint32_t)q[2 * i] : 0u) | (c + 2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
            }
        }
    } else {
        const int past = c + 8 - n;   // values past the end
        // 32-bit offset from a row that the waves of a row share: one scalar base
        const char* from = reinterpret_cast<const char*>(row) + (uint32_t)(past > 0 ? n - 8 : c) * (uint32_t)sizeof(T);
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const v4i_any* at = reinterpret_cast<const v4i_any*>(from) + i;
            v4i_any v;
            if constexpr (NT) v = __builtin_nontemporal_load(at);
            else v = *at;
#pragma unroll
            for (int k = 0; k < 4; ++k) r.w[4 * i + k] = (uint32_t)v[k];
        }
        if (past > 0) {
#pragma unroll
            for (int d = W / 2; d >= 1; d /= 2) {   // dwords: 4, 2, 1 of an fp32 group, 2, 1 of a 16-bit one
                const bool move = (past & d * 4 / (int)sizeof(T)) != 0;
#pragma unroll
                for (int i = 0; i < W; ++i) r.w[i] = move ? (i + d < W ? r.w[i + d] : 0u) : r.w[i];
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if constexpr (sizeof(T) == 2) {
                    const uint32_t next = i + 1 < W ? r.w[i + 1] : 0u;
                    r.w[i] = past & 1 ? (r.w[i] >> 16) | (next << 16) : r.w[i];
                }
                r.w[i] = past >= 8 ? 0u : r.w[i];
            }
        }
    }
}

// The values to c .. c + 7 of a row of n, those past its end left out; c < n.
template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int n, const Pack8<T>& r) {
    const int left = n - c;
    char* p = reinterpret_cast<char*>(row) + (uint32_t)c * (uint32_t)sizeof(T);
    if (left >= 8) {
        if constexpr (sizeof(T) == 1) {
            __builtin_memcpy(p, r.w, 8);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                v4i_any* at = reinterpret_cast<v4i_any*>(p) + i;
                const v4i_any v = {(int)r.w[4 * i], (int)r.w[4 * i + 1], (int)r.w[4 * i + 2], (int)r.w[4 * i + 3]};
                *at = v;
            }
        }
    } else {
        Pack8<T> t = r;
#pragma unroll
        for (int k = 4; k >= 1; k /= 2) {   // four values, two, one
            constexpr int W = 2 * sizeof(T);
            const int bytes = k * (int)sizeof(T);
            if ((left & k) == 0) continue;
            __builtin_memcpy(p, t.w, bytes);
            p += bytes;
            if (bytes >= 4) {
#pragma unroll
                for (int i = 0; i < W; ++i) t.w[i] = i + bytes / 4 < W ? t.w[i + bytes / 4] : 0u;
            } else {
                t.w[0] >>= 8 * bytes;
            }
        }
    }
}

// Keeps the compiler from holding the unpacked values from here on: they are
// unpacked again where they are used.
template <typename T>
__device__ __forceinline__ void stay_packed(Pack8<T>& p) {
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); ++i) asm volatile("" : "+v"(p.w[i]));
}

// Eight weights as floats.
template <typename W, bool TINY>
__device__ __forceinline__ void load_weights(const void* weight, int c, int n, float* w) {
    Pack8<W> p;
    load8<TINY>(reinterpret_cast<const W*>(weight), c, n, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = value(p, e);
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
