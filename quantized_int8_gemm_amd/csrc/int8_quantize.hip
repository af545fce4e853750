// Values to int8 with a scale per row or per block of 32 columns, and back.
//
// Bound by HBM.  Whole rows: a row stays packed in the registers of the lanes that
// share it between its maximum and its codes, so it is read once.  Blocks: each lane
// moves eight values, four lanes share a block, whose maximum takes two quad
// permutes.
#include "fused_common.h"

namespace qg {
namespace {

constexpr int NT = 256;

template <typename T, int G, int ITER, bool TINY>
__global__ __launch_bounds__(G < 256 ? 256 : G) void int8_rows_kernel(Int8Args a) {
    constexpr int RPW = G < 256 ? 256 / G : 1;
    const int t = threadIdx.x % G, n = (int)a.n;
    const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / G;
    if (row >= a.M) return;   // whole groups (no barrier with several in a workgroup)
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    Pack8<T> v[ITER];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < ITER; ++i) load8<TINY>(x, (i * G + t) * 8, n, v[i]);
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = umax(top, abs_bits(value(v[i], e)));
#pragma unroll
    for (int off = G < 64 ? G / 2 : 32; off >= 1; off >>= 1) top = umax(top, (uint32_t)__shfl_xor((int)top, off));
    if constexpr (G > 64) {
        __shared__ uint32_t red[G / 64];
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
        __syncthreads();
        top = red[0];
#pragma unroll
        for (int w = 1; w < G / 64; ++w) top = umax(top, red[w]);
    }
    const Int8Form f(top);
    if (t == 0) a.scale[row * a.lds] = f.scale;
    int8_t* dst = a.codes + row * a.ldc;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * G + t) * 8;
        Pack8<int8_t> q = {};
#pragma unroll
        for (int h = 0; h < 2; ++h)
            q.w[h] = f.codes(value(v[i], 4 * h), value(v[i], 4 * h + 1), value(v[i], 4 * h + 2), value(v[i], 4 * h + 3));
        if (c < n) store8(dst, c, n, q);
    }
}

// Lanes are numbered over the rows' groups of eight, whole blocks of four to a row.
template <typename T, bool TINY>
__global__ __launch_bounds__(NT) void int8_blocks_kernel(Int8Args a, int64_t gpr) {
    const int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int64_t row = t / gpr;
    const int c = (int)(t - row * gpr) * 8, n = (int)a.n;
    const bool live = row < a.M;
    Pack8<T> v;
    load8<TINY>(reinterpret_cast<const T*>(a.x) + (live ? row : 0) * a.ldx, live ? c : 0, n, v);
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = umax(top, abs_bits(value(v, e)));
    const Int8Form f(quad_max(top));
    Pack8<int8_t> q = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) q.w[h] = f.codes(value(v, 4 * h), value(v, 4 * h + 1), value(v, 4 * h + 2), value(v, 4 * h + 3));
    if (!live || c >= n) return;
    store8(a.codes + row * a.ldc, c, n, q);
    if (c % INT8_BLOCK == 0) a.scale[row * a.lds + c / INT8_BLOCK] = f.scale;
}

template <typename T>
__global__ __launch_bounds__(NT) void int8_dequantize_kernel(Int8Args a, int64_t gpr) {
    const int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int64_t row = t / gpr;
    const int c = (int)(t - row * gpr) * 8, n = (int)a.n;
    if (row >= a.M) return;
    const int8_t* q = a.codes + row * a.ldc + c;
    const float s = a.scale[row * a.lds + (a.block != 0 ? c / INT8_BLOCK : 0)];
    float v[8];
    if (c + 8 <= n) {
        uint2 w;
        __builtin_memcpy(&w, q, 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) * s;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < n ? (float)q[e] * s : 0.f;
    }
    store8(reinterpret_cast<T*>(a.out) + row * a.ldo, c, n, pack<T>(v));
}

template <typename T>
hipError_t rows(const Int8Args& a, hipStream_t s) {
#define QG_ROWS(G, ITER, LIMIT, TINY)                                                                                \
    if (a.n <= LIMIT) {                                                                                              \
        constexpr int RPW = G < 256 ? 256 / G : 1;                                                                   \
        hipLaunchKernelGGL((int8_rows_kernel<T, G, ITER, TINY>), dim3((unsigned)((a.M + RPW - 1) / RPW)),            \
                           dim3(G < 256 ? 256 : G), 0, s, a);                                                        \
        return hipGetLastError();                                                                                    \
    }
    QG_ROWS(16, 1, 7, true)
    QG_ROWS(16, 1, 128, false)
    QG_ROWS(64, 1, 512, false)
    QG_ROWS(256, 1, 2048, false)
    QG_ROWS(256, 2, 4096, false)
    QG_ROWS(256, 4, 8192, false)
    QG_ROWS(512, 4, 16384, false)
    QG_ROWS(1024, 4, 32768, false)
    QG_ROWS(1024, 8, 65536, false)
#undef QG_ROWS
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t quantize(const Int8Args& a, hipStream_t s) {
    if (a.block == 0) return rows<T>(a, s);
    const int64_t gpr = (a.n + 31) / 32 * 4;
    const dim3 grid((unsigned)((a.M * gpr + NT - 1) / NT));
    if (a.n < 8) hipLaunchKernelGGL((int8_blocks_kernel<T, true>), grid, dim3(NT), 0, s, a, gpr);
    else hipLaunchKernelGGL((int8_blocks_kernel<T, false>), grid, dim3(NT), 0, s, a, gpr);
    return hipGetLastError();
}

template <typename T>
hipError_t dequantize(const Int8Args& a, hipStream_t s) {
    const int64_t gpr = (a.n + 7) / 8;
    hipLaunchKernelGGL((int8_dequantize_kernel<T>), dim3((unsigned)((a.M * gpr + NT - 1) / NT)), dim3(NT), 0, s, a, gpr);
    return hipGetLastError();
}

// A launch holds fewer than 2^32 threads: rows by pieces.
template <typename F>
hipError_t by_pieces(const Int8Args& all, int size, int64_t threads_a_row, F&& launch) {
    const int64_t piece = threads_a_row >= (int64_t)1 << 30 ? 1 : ((int64_t)1 << 31) / threads_a_row;
    for (int64_t m = 0; m < all.M; m += piece) {
        Int8Args a = all;
        a.M = all.M - m < piece ? all.M - m : piece;
        if (all.x != nullptr) a.x = (const char*)all.x + m * all.ldx * size;
        if (all.out != nullptr) a.out = (char*)all.out + m * all.ldo * size;
        a.codes = all.codes + m * all.ldc;
        a.scale = all.scale + m * all.lds;
        const hipError_t e = launch(a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_int8_quantize(const Int8Args& all, qg_dtype type, hipStream_t s) {
    return by_pieces(all, type == QG_FP32 ? 4 : 2, all.block == 0 ? 1024 : (all.n + 31) / 32 * 4, [&](const Int8Args& a) {
        return type == QG_FP32 ? quantize<float>(a, s) : type == QG_BF16 ? quantize<__bf16>(a, s) : quantize<_Float16>(a, s);
    });
}

hipError_t launch_int8_dequantize(const Int8Args& all, qg_dtype type, hipStream_t s) {
    return by_pieces(all, type == QG_FP32 ? 4 : 2, (all.n + 7) / 8, [&](const Int8Args& a) {
        return type == QG_FP32 ? dequantize<float>(a, s) : type == QG_BF16 ? dequantize<__bf16>(a, s) : dequantize<_Float16>(a, s);
    });
}

}  // namespace qg
