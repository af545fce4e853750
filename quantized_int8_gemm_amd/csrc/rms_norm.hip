// Root-mean-square norm with the residual's addition and an output in fp32,
// bf16 or fp16, in int8 with a scale per row, or in MX form.
//
// Mathematics: h = x + residual (stored in x's type), r = 1 / sqrt(mean h^2 +
// eps), y = h r w.  r is one factor of the whole row, so a quantised output
// never needs it: int8 codes are rint(t * 127 / max|t|) with t = h w, and r
// joins the row's scale; MX blocks hold t and r is handed on as the product's
// row scale.  The codes are then the same whatever order the sum of squares
// is added in, and MX blocks leave before the row's sum is known.
//
// Bound by HBM: every value is read once and kept in registers (at most 64 a
// lane), one barrier per row.  Past 32768 columns that is more than 1024 lanes have:
// fp32 spills (83 to 95 of a lane's 128 registers, 232 to 240 bytes), fp16 a little (8 to
// 20): 1000 x 65536 with a residual to int8 fp32 263 us, 3.2 TB/s, fp16 128, 3.6, bf16
// 102, 4.5; 1000 x 32768 fp32 88 us, 4.8.  A row is shared by G lanes: 16 up to 128 columns,
// 32 up to 256, a wave up to 1024 (16, 8 and 4 rows per workgroup), 256 lanes up to
// 8192, 512 up to 16384, 1024 beyond.  Up to 512 rows leave CUs without work, so the
// lanes of each take as little of it as they can: 512 up to 4096 columns, 1024 beyond
// (to int8, bf16: 1 x 8192 4.5 -> 3.7 us, 16 x 5000 5.2 -> 4.0, 256 x 4096 5.0 -> 4.6;
// 768 x 5000 8.5 -> 9.5, 1024 x 8192 13.0 -> 13.8).  Lanes that have nothing of a row
// cost as much as those that have: 8192 x 5120 bf16 54.9 us with the four groups a lane
// that 8192 columns take, 49.5 with three.
// 8192 x 8192 bf16 with a residual to int8: 75 us, 6.3 TB/s over what is read
// and written (a copy of 2 GiB runs at 4.85), where calls write the same outputs again,
// 81.5 where each allocates its own; one row of 4096 2.6 us, the launch's and one load's
// latency.
#include "mx_common.h"

namespace qg {
namespace {

enum { OUT_SAME = 0, OUT_F32 = 1, OUT_I8 = 2, OUT_MX8 = 3, OUT_MX4 = 4 };

// Sum of `ss` and maximum of `top` over the G lanes of a row; every lane
// receives both.
template <int G>
__device__ __forceinline__ void row_reduce(float& ss, uint32_t& top) {
#pragma unroll
    for (int off = G < 64 ? G / 2 : 32; off >= 1; off >>= 1) {
        ss += __shfl_xor(ss, off);
        top = umax(top, (uint32_t)__shfl_xor((int)top, off));
    }
    if constexpr (G > 64) {
        __shared__ float s_ss[G / 64];
        __shared__ uint32_t s_top[G / 64];
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            s_ss[wave] = ss;
            s_top[wave] = top;
        }
        __syncthreads();
        ss = s_ss[0];
        top = s_top[0];
#pragma unroll
        for (int w = 1; w < G / 64; ++w) {
            ss += s_ss[w];
            top = umax(top, s_top[w]);
        }
    }
}

// fp16: six waves a SIMD asked for, since its widened halves take registers that
// would leave five (4000 x 8192 fp16 to fp16 51.2 -> 48.5 us).
template <typename T, int G, int ITER, int OUT, bool WF32, bool TINY, bool NT>
__global__ __launch_bounds__(G < 256 ? 256 : G, ((std::is_same<T, _Float16>::value && G <= 512) ? 6 : 1)) void rms_norm_kernel(RmsNormArgs a) {
    constexpr int RPW = G < 256 ? 256 / G : 1;   // rows per workgroup
    const int t = threadIdx.x % G;
    const int sub = threadIdx.x / G;
    const int64_t row = (int64_t)blockIdx.x * RPW + (G < 64 ? sub : __builtin_amdgcn_readfirstlane(sub));
    if (row >= a.M) return;                      // whole groups (no barrier with several in a workgroup)
    const int n = a.n;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* res = a.res != nullptr ? reinterpret_cast<const T*>(a.res) + row * a.ldr : nullptr;

    Pack8<T> xv[ITER], rv[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * G + t) * 8;
        load8<TINY, NT>(x, c, n, xv[i]);
    }
    if (res != nullptr) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * G + t) * 8;
            load8<TINY, NT>(res, c, n, rv[i]);
        }
    }
    float ss = 0.f;
    uint32_t top = 0u;
    float y[ITER][8];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * G + t) * 8;
        if (res != nullptr) {
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = value(xv[i], e) + value(rv[i], e);
            xv[i] = pack<T>(h);
            if (c < n) store8(reinterpret_cast<T*>(a.h) + row * a.ldh, c, n, xv[i]);
        }
        float w[8];
        load_weights<typename std::conditional<WF32, float, T>::type, TINY>(a.weight, c, n, w);
        uint32_t m = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float h = value(xv[i], e);
            ss = __builtin_fmaf(h, h, ss);
            y[i][e] = h * w[e];
            m = umax(m, abs_bits(y[i][e]));
        }
        if constexpr (OUT == OUT_MX8 || OUT == OUT_MX4) {
            // four lanes hold one block of 32; columns past n are zeros
            m = quad_max(m);
            const uint32_t b = mx_scale_byte<OUT == OUT_MX4>(m);
            uint32_t q[2];
            mx_encode8<OUT == OUT_MX4>(y[i], b, q);
            if ((c & ~31) < n) {
                uint8_t* dst = reinterpret_cast<uint8_t*>(a.out) + row * a.ldo;
                if constexpr (OUT == OUT_MX4) __builtin_memcpy(dst + c / 2, q, 4);
                else __builtin_memcpy(dst + c, q, 8);
                if ((t & 3) == 0) a.block_scale[row * a.lds + c / 32] = (uint8_t)b;
            }
        }
        top = umax(top, m);
    }
    row_reduce<G>(ss, top);
    const float r = 1.0f / __builtin_sqrtf(ss / (float)n + a.eps);
    if constexpr (OUT == OUT_I8) {
        const bool bad = top >= INF_BITS;
        float most = __uint_as_float(top);
        // 127 / most stays finite: tiny rows are multiplied by 2^60, exactly
        const float up = most < 0x1p-100f ? 0x1p60f : 1.0f;
        const float inv = bad || top == 0u ? 0.f : 127.0f / (most * up);
        if (t == 0) a.row_scale[row] = bad ? __uint_as_float(0x7fc00000u) : (top == 0u ? 1.0f : most * r / 127.0f);
        int8_t* dst = reinterpret_cast<int8_t*>(a.out) + row * a.ldo;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * G + t) * 8;
            Pack8<int8_t> q = {};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = bad ? 0.f : (y[i][e] * up) * inv;
                q.w[e / 4] |= ((uint32_t)(int)__builtin_rintf(v) & 0xffu) << (8 * (e & 3));
            }
            if (c < n) store8(dst, c, n, q);
        }
    } else {
        if (t == 0 && a.row_scale != nullptr) a.row_scale[row] = r;
        if constexpr (OUT == OUT_SAME || OUT == OUT_F32) {
            typedef typename std::conditional<OUT == OUT_F32, float, T>::type O;
            O* dst = reinterpret_cast<O*>(a.out) + row * a.ldo;
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                const int c = (i * G + t) * 8;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = y[i][e] * r;
                if (c < n) store8(dst, c, n, pack<O>(v));
            }
        }
    }
}

template <typename T, int OUT, bool WF32>
hipError_t by_width(const RmsNormArgs& a, hipStream_t s) {
#define QG_NORM(G, ITER, LIMIT, TINY, NT)                                                                      \
    if (a.n <= LIMIT) {                                                                                        \
        constexpr int RPW = G < 256 ? 256 / G : 1;                                                             \
        hipLaunchKernelGGL((rms_norm_kernel<T, G, ITER, OUT, WF32, TINY, NT>),                                 \
                           dim3((unsigned)((a.M + RPW - 1) / RPW)), dim3(G < 256 ? 256 : G), 0, s, a);         \
        return hipGetLastError();                                                                              \
    }
    QG_NORM(16, 1, 7, true, false)
    QG_NORM(16, 1, 128, false, false)
    QG_NORM(32, 1, 256, false, false)
    QG_NORM(64, 1, 512, false, false)
    QG_NORM(64, 2, 1024, false, false)
    QG_NORM(256, 1, 2048, false, false)
    if (a.M <= 512) {
        if (a.n > 2048) QG_NORM(512, 1, 4096, false, false)
        if (a.n > (a.M <= 256 ? 4096 : 6144)) QG_NORM(1024, 1, 8192, false, false)
        if (a.n > 8192) QG_NORM(1024, 2, 16384, false, false)
    }
    if constexpr (sizeof(T) == 2) {
        if (whole_lines(a.x, a.ldx * sizeof(T)) && (a.res == nullptr || whole_lines(a.res, a.ldr * sizeof(T)))) {
            QG_NORM(256, 2, 4096, false, true)
            QG_NORM(256, 3, 6144, false, true)
            QG_NORM(256, 4, 8192, false, true)
            QG_NORM(512, 4, 16384, false, true)
        }
    }
    QG_NORM(256, 2, 4096, false, false)
    QG_NORM(256, 3, 6144, false, false)
    QG_NORM(256, 4, 8192, false, false)
    QG_NORM(512, 4, 16384, false, false)
    QG_NORM(1024, 4, 32768, false, false)
    QG_NORM(1024, 8, 65536, false, false)
#undef QG_NORM
    return hipErrorInvalidValue;
}

template <typename T, bool WF32>
hipError_t by_format(const RmsNormArgs& a, int out, hipStream_t s) {
    switch (out) {
        case OUT_SAME: return by_width<T, OUT_SAME, WF32>(a, s);
        case OUT_F32: return by_width<T, OUT_F32, WF32>(a, s);
        case OUT_I8: return by_width<T, OUT_I8, WF32>(a, s);
        case OUT_MX8: return by_width<T, OUT_MX8, WF32>(a, s);
        default: return by_width<T, OUT_MX4, WF32>(a, s);
    }
}

}  // namespace

namespace {

hipError_t by_type(const RmsNormArgs& a, qg_dtype type, bool weight_f32, int out, hipStream_t s) {
    if (type == QG_FP32) return by_format<float, false>(a, out, s);
    if (type == QG_BF16) return weight_f32 ? by_format<__bf16, true>(a, out, s) : by_format<__bf16, false>(a, out, s);
    return weight_f32 ? by_format<_Float16, true>(a, out, s) : by_format<_Float16, false>(a, out, s);
}

}  // namespace

hipError_t launch_rms_norm(const RmsNormArgs& all, qg_dtype type, bool weight_f32, qg_dtype format, hipStream_t s,
                           const char** name) {
    const int out = format == QG_INT8 ? OUT_I8 : format == QG_MXFP8 ? OUT_MX8 : format == QG_MXFP4 ? OUT_MX4
                  : format == type ? OUT_SAME : OUT_F32;
    static const char* names[] = {"rms_norm", "rms_norm", "rms_norm_int8", "rms_norm_mxfp8", "rms_norm_mxfp4"};
    *name = names[out];
    // a launch holds fewer than 2^32 threads, 1024 a row at most
    constexpr int64_t ROWS = (int64_t)1 << 21;
    const int in_size = type == QG_FP32 ? 4 : 2;
    const int out_size = out == OUT_SAME ? in_size : out == OUT_F32 ? 4 : 1;
    for (int64_t m = 0; m < all.M; m += ROWS) {
        RmsNormArgs a = all;
        a.M = all.M - m < ROWS ? all.M - m : ROWS;
        a.x = (const char*)all.x + m * all.ldx * in_size;
        if (all.res != nullptr) {
            a.res = (const char*)all.res + m * all.ldr * in_size;
            a.h = (char*)all.h + m * all.ldh * in_size;
        }
        a.out = (char*)all.out + m * all.ldo * out_size;
        if (all.block_scale != nullptr) a.block_scale = all.block_scale + m * all.lds;
        if (all.row_scale != nullptr) a.row_scale = all.row_scale + m;
        const hipError_t e = by_type(a, type, weight_f32, out, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qg
