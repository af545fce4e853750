// Values to MX form and back.
//
// Bound by HBM: each lane moves eight consecutive values (16 bytes of a 16-bit
// type), four lanes hold one block of 32, and the block's largest magnitude
// comes from two quad permutes.  8192 x 8192 bf16 to MXFP4 and back: 57.5 us, 5.3
// TB/s over values in, codes and values out.  Lanes are numbered over the rows' groups of
// eight, so short and odd rows fill waves as well as long ones.
#include "mx_common.h"

namespace qg {
namespace {

constexpr int NT = 256;
constexpr int UNROLL = 4;   // groups of eight in flight per lane

// Row and group of eight in it of the groups that a workgroup moves.  Only the first one's
// are found by a division; the rest lie a few rows on.  2^31 / per, rounded up, finds how
// many exactly while x * per < 2^31: per < 1024, where x < 2048.  Longer rows: one at most.
struct Places {
    int64_t row0;
    uint32_t rem, per, part;
    __device__ __forceinline__ Places(uint32_t per_, uint32_t part_) : per(per_), part(part_) {
        const int64_t first = (int64_t)blockIdx.x * (NT * UNROLL);
        row0 = first / per;
        rem = (uint32_t)(first - row0 * per);
    }
    __device__ __forceinline__ void at(int u, int64_t& row, int& c) const {
        const uint32_t x = rem + threadIdx.x + u * NT;
        const uint32_t on = part != 0u ? __umulhi(x << 1, part) : (uint32_t)(x >= per);
        row = row0 + on;
        c = (int)(x - on * per) * 8;
    }
};

template <typename T, bool FP4, bool TINY, bool ONCE>
__global__ __launch_bounds__(NT) void mx_quantize_kernel(MxCodecArgs a, uint32_t gpr, uint32_t part, int64_t groups) {
    const int64_t g0 = (int64_t)blockIdx.x * (NT * UNROLL) + threadIdx.x;
    const Places places(gpr, part);
    Pack8<T> v[UNROLL];
    int64_t row[UNROLL];
    int c[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t g = g0 + u * NT;
        places.at(u, row[u], c[u]);
        if (g >= groups) row[u] = c[u] = 0;   // past the last one: read something that is there
        load8<TINY, ONCE>(reinterpret_cast<const T*>(a.x) + row[u] * a.ldx, c[u], (int)a.n, v[u]);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        float f[8];
        uint32_t m = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[e] = value(v[u], e);
            m = umax(m, abs_bits(f[e]));
        }
        m = quad_max(m);
        const uint32_t b = mx_scale_byte<FP4>(m);
        uint32_t q[2];
        mx_encode8<FP4>(f, b, q);
        if (g0 + u * NT < groups) {
            uint8_t* dst = a.codes + row[u] * a.ldc;
            if constexpr (FP4) __builtin_memcpy(dst + c[u] / 2, q, 4);
            else __builtin_memcpy(dst + c[u], q, 8);
            if ((threadIdx.x & 3) == 0) a.scale[row[u] * a.lds + c[u] / 32] = (uint8_t)b;
        }
    }
}

template <typename T, bool FP4>
__global__ __launch_bounds__(NT) void mx_dequantize_kernel(MxCodecArgs a, uint32_t gpr, uint32_t part, int64_t groups) {
    const int64_t g0 = (int64_t)blockIdx.x * (NT * UNROLL) + threadIdx.x;
    const Places places(gpr, part);
    uint32_t q[UNROLL][2];
    uint32_t b[UNROLL];
    int64_t row[UNROLL];
    int c[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t g = g0 + u * NT;
        places.at(u, row[u], c[u]);
        q[u][0] = q[u][1] = b[u] = 0u;
        if (g < groups) {
            const uint8_t* src = a.codes + row[u] * a.ldc;
            if constexpr (FP4) __builtin_memcpy(q[u], src + c[u] / 2, 4);
            else __builtin_memcpy(q[u], src + c[u], 8);
            b[u] = a.scale[row[u] * a.lds + c[u] / 32];
        }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        if (g0 + u * NT >= groups) continue;
        const float s = mx_factor(b[u]);
        v2f p[4];
        if constexpr (FP4) {
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u][0], 1.0f, 0);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u][0], 1.0f, 1);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u][0], 1.0f, 2);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u][0], 1.0f, 3);
        } else {
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[u][0], 1.0f, false);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[u][0], 1.0f, true);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[u][1], 1.0f, false);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[u][1], 1.0f, true);
        }
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = p[e / 2][e & 1] * s;
        store8(reinterpret_cast<T*>(a.out) + row[u] * a.ldo, c[u], (int)a.n, pack<T>(o));
    }
}

template <typename T, bool FP4>
hipError_t run(const MxCodecArgs& a, bool back, hipStream_t s) {
    // Quantising covers whole blocks (their padding is written), reading back
    // the n values.
    const int64_t gpr = back ? (a.n + 7) / 8 : (a.n + 31) / 32 * 4;
    const int64_t groups = a.M * gpr, blocks = (groups + NT * UNROLL - 1) / (NT * UNROLL);
    const uint32_t part = gpr < 1024 ? (uint32_t)((((int64_t)1 << 31) + gpr - 1) / gpr) : 0u;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    if (back)
        hipLaunchKernelGGL((mx_dequantize_kernel<T, FP4>), dim3((unsigned)blocks), dim3(NT), 0, s, a, (uint32_t)gpr, part, groups);
    else if (a.n < 8)
        hipLaunchKernelGGL((mx_quantize_kernel<T, FP4, true, false>), dim3((unsigned)blocks), dim3(NT), 0, s, a, (uint32_t)gpr, part, groups);
    else if (sizeof(T) == 2 && whole_lines(a.x, a.ldx * sizeof(T)))
        hipLaunchKernelGGL((mx_quantize_kernel<T, FP4, false, sizeof(T) == 2>), dim3((unsigned)blocks), dim3(NT), 0, s, a, (uint32_t)gpr, part, groups);
    else
        hipLaunchKernelGGL((mx_quantize_kernel<T, FP4, false, false>), dim3((unsigned)blocks), dim3(NT), 0, s, a, (uint32_t)gpr, part, groups);
    return hipGetLastError();
}

template <bool FP4>
hipError_t by_type(const MxCodecArgs& a, qg_dtype type, bool back, hipStream_t s) {
    if (type == QG_FP32) return run<float, FP4>(a, back, s);
    if (type == QG_BF16) return run<__bf16, FP4>(a, back, s);
    return run<_Float16, FP4>(a, back, s);
}

}  // namespace

hipError_t launch_mx_quantize(const MxCodecArgs& a, qg_dtype type, qg_dtype format, hipStream_t s, const char** name) {
    *name = format == QG_MXFP4 ? "mx_quantize_mxfp4" : "mx_quantize_mxfp8";
    return format == QG_MXFP4 ? by_type<true>(a, type, false, s) : by_type<false>(a, type, false, s);
}

hipError_t launch_mx_dequantize(const MxCodecArgs& a, qg_dtype type, qg_dtype format, hipStream_t s, const char** name) {
    *name = format == QG_MXFP4 ? "mx_dequantize_mxfp4" : "mx_dequantize_mxfp8";
    return format == QG_MXFP4 ? by_type<true>(a, type, true, s) : by_type<false>(a, type, true, s);
}

}  // namespace qg
