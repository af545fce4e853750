// The scaled matrix-core instructions as the MX product uses them, with W
// (always e2m1) as the first operand and A (e2m1 or e4m3) as the second, so a
// lane's results are consecutive columns of one output row.
//
// 32x32x64: lane l holds row l % 32 of its operand, g = l / 32.  e2m1: the 32
// values k = 32 g .. 32 g + 31 in 16 bytes; e4m3: k = 16 g .. + 15 and 32 + 16
// g .. + 15 in 32 bytes.  Either way the scale of values 32 g .. + 31 is taken
// from lane group g, byte `sel` of its scale register.  Result register i of
// lane l: W row 8 (i / 4) + 4 g + i % 4, A row l % 32.
// 16x16x128: the same with row l % 16, g = l / 16: e2m1 k = 32 g .. + 31, e4m3
// k = 16 g .. + 15 and 64 + 16 g .. + 15; result register i: W row 4 g + i, A
// row l % 16.
#pragma once
#include "mx_common.h"

namespace qg {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int FMT_E4M3 = 0, FMT_E2M1 = 4;

__device__ __forceinline__ v8i words4(u32x4 a) { return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0}; }
__device__ __forceinline__ v8i words8(u32x4 a, u32x4 b) {
    return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// An 8-bit operand's products are added in groups of 16 k, aligned to the
// largest, and what lies 2^-14 below that is cut off: where the largest cancel,
// most of the result (448 * 6 - 448 * 6 beside sums of 0.5 to 250 left the sums 2
// off).  e4m3 values split at 2 (bit 6, the exponent field's top bit) span eight
// binades each, and products with e2m1 values within eight binades fit those 14
// bits: two instructions, one for each half, lose nothing.
__device__ __forceinline__ void split_e4m3(v8i a, v8i& hi, v8i& lo) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // 0xff for each byte whose bit 6 is set: the byte permute's selectors 8 to 11
        // repeat the top bit of bytes 1, 3, 5 and 7 of its two operands
        const uint32_t x = (uint32_t)a[i];
        const uint32_t mask = __builtin_amdgcn_perm(x << 1, x << 9, 0x0b090a08u);
        hi[i] = (int)(x & mask);
        lo[i] = (int)(x ^ (x & mask));
    }
}

template <bool A8, int WSEL, int ASEL>
__device__ __forceinline__ v16f mfma_mx32(v8i w, uint32_t ws, v8i a, uint32_t as, v16f c) {
    if constexpr (A8) {
        v8i hi, lo;
        split_e4m3(a, hi, lo);
        c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, lo, c, FMT_E2M1, FMT_E4M3, WSEL, (int)ws, ASEL, (int)as);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, hi, c, FMT_E2M1, FMT_E4M3, WSEL, (int)ws, ASEL, (int)as);
    } else {
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, FMT_E2M1, FMT_E2M1, WSEL, (int)ws, ASEL, (int)as);
    }
}

template <bool A8>
__device__ __forceinline__ v4f mfma_mx16(v8i w, uint32_t ws, v8i a, uint32_t as, v4f c) {
    if constexpr (A8) {
        v8i hi, lo;
        split_e4m3(a, hi, lo);
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, lo, c, FMT_E2M1, FMT_E4M3, 0, (int)ws, 0, (int)as);
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, hi, c, FMT_E2M1, FMT_E4M3, 0, (int)ws, 0, (int)as);
    } else {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, FMT_E2M1, FMT_E2M1, 0, (int)ws, 0, (int)as);
    }
}

// One output element.
template <typename T>
__device__ __forceinline__ void put(void* out, int64_t at, float v) {
    reinterpret_cast<T*>(out)[at] = (T)v;
}

}  // namespace qg
