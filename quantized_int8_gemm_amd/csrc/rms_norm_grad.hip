// Gradient of the root-mean-square norm.
//
// Mathematics: with g = dy w, dx = r g - h r^3 / n sum(g h) (+ dh) and dw =
// sum over rows of dy h r.  Bound by HBM: dy, h (and dh) are read once.  A
// workgroup walks rows with a fixed set of columns per lane, so dw is added up
// in registers and leaves once, as one row of partial sums per workgroup; a
// second kernel adds those.  No atomics: the order of every sum is fixed.
#include "mx_common.h"

namespace qg {
namespace {

template <int G>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    if constexpr (G > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < G / 64; ++w) v += red[w];
    }
    return v;
}

// The lane's columns are (i * G + t) * 8 .. + 7.  Row groups of G < 256 lanes
// share a workgroup; their partial sums of dw are added through LDS.
template <typename T, int G, int ITER, bool WF32>
__global__ __launch_bounds__(G < 256 ? 256 : G) void rms_norm_grad_kernel(RmsNormGradArgs a) {
    constexpr int RPW = G < 256 ? 256 / G : 1;
    __shared__ float red[2][G / 64];
    __shared__ float part[RPW > 1 ? (RPW - 1) * G * ITER * 8 : 1];
    const int t = threadIdx.x % G, sub = threadIdx.x / G;
    const int n = a.n;
    float w[ITER][8], dw[ITER][8];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * G + t) * 8;
        if constexpr (WF32) {
            Pack8<float> p;
            load8(reinterpret_cast<const float*>(a.weight) + c, n - c, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[i][e] = p.v[e];
        } else {
            Pack8<T> p;
            load8(reinterpret_cast<const T*>(a.weight) + c, n - c, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[i][e] = (float)p.v[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPW + sub; row < a.M; row += (int64_t)gridDim.x * RPW, turn ^= 1) {
        const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.ldy;
        const T* h = reinterpret_cast<const T*>(a.h) + row * a.ldh;
        Pack8<T> yv[ITER], hv[ITER], sv[ITER];
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * G + t) * 8;
            load8(dy + c, n - c, yv[i]);
            load8(h + c, n - c, hv[i]);
        }
        if (a.dh != nullptr) {
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                const int c = (i * G + t) * 8;
                load8(reinterpret_cast<const T*>(a.dh) + row * a.lddh + c, n - c, sv[i]);
            }
        }
        const float r = a.rstd[row];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < ITER; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float yh = (float)yv[i].v[e] * (float)hv[i].v[e];
                dot = __builtin_fmaf(yh, w[i][e], dot);
                dw[i][e] = __builtin_fmaf(yh, r, dw[i][e]);
            }
        // two slots taken in turn: a wave may be one row ahead of the others' reads
        dot = row_sum<G>(dot, red[turn]);
        const float k = r * r * r * (dot / (float)n);
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * G + t) * 8;
            Pack8<T> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = r * ((float)yv[i].v[e] * w[i][e]) - k * (float)hv[i].v[e];
                if (a.dh != nullptr) v += (float)sv[i].v[e];
                o.v[e] = (T)v;
            }
            if (c < n) store8(reinterpret_cast<T*>(a.dx) + row * a.ldx + c, n - c, o);
        }
    }
    if constexpr (RPW > 1) {
        if (sub > 0) {
#pragma unroll
            for (int i = 0; i < ITER; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) part[(((sub - 1) * ITER + i) * 8 + e) * G + t] = dw[i][e];
        }
        __syncthreads();
        if (sub > 0) return;
#pragma unroll
        for (int q = 0; q < RPW - 1; ++q)
#pragma unroll
            for (int i = 0; i < ITER; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[i][e] += part[((q * ITER + i) * 8 + e) * G + t];
    }
    float* out = a.part + (int64_t)blockIdx.x * n;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * G + t) * 8;
        Pack8<float> o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = dw[i][e];
        if (c < n) store8(out + c, n - c, o);
    }
}

// dw[j] = sum of the partial rows: 32 columns a workgroup (one 128-byte line
// of each row), eight lanes a column, joined through LDS.
template <typename W>
__global__ __launch_bounds__(256) void rms_norm_grad_sum(const float* __restrict__ part, int parts, int n,
                                                         W* __restrict__ dw) {
    __shared__ float red[8][33];
    const int cl = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + cl;
    float s = 0.f;
    if (c < n) {
#pragma unroll 8
        for (int p = q; p < parts; p += 8) s += part[(int64_t)p * n + c];
    }
    red[q][cl] = s;
    __syncthreads();
    if (q == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][cl];
        dw[c] = (W)s;
    }
}

// Lanes per row for n columns: as the kernel table below.
int rows_per_group(int64_t n) { return n <= 1024 ? 4 : 1; }

template <typename T, bool WF32>
hipError_t by_width(const RmsNormGradArgs& a, hipStream_t s) {
    typedef typename std::conditional<WF32, float, T>::type W;
    bool done = a.M == 0;
#define QG_GRAD(G, ITER)                                                                                       \
    if (!done && a.n <= G * ITER * 8) {                                                                        \
        hipLaunchKernelGGL((rms_norm_grad_kernel<T, G, ITER, WF32>), dim3((unsigned)a.parts),                  \
                           dim3(G < 256 ? 256 : G), 0, s, a);                                                  \
        done = true;                                                                                           \
    }
    QG_GRAD(64, 1)
    QG_GRAD(64, 2)
    QG_GRAD(256, 1)
    QG_GRAD(256, 2)
    QG_GRAD(512, 2)
    QG_GRAD(1024, 2)
    QG_GRAD(1024, 4)
    QG_GRAD(1024, 8)
#undef QG_GRAD
    if (!done) return hipErrorInvalidValue;
    hipLaunchKernelGGL((rms_norm_grad_sum<W>), dim3((unsigned)((a.n + 31) / 32)), dim3(256), 0, s, a.part, a.parts, a.n,
                       reinterpret_cast<W*>(a.dweight));
    return hipGetLastError();
}

}  // namespace

// Workgroups of the row kernel, each with one partial row of dw: two per
// compute unit, none without rows.
int rms_norm_grad_parts(int64_t M, int64_t n) {
    const int64_t groups = (M + rows_per_group(n) - 1) / rows_per_group(n);
    return (int)(groups < 512 ? groups : 512);
}

hipError_t launch_rms_norm_grad(const RmsNormGradArgs& a, qg_dtype type, bool weight_f32, hipStream_t s,
                                const char** name) {
    *name = "rms_norm_grad";
    if (type == QG_FP32) return by_width<float, false>(a, s);
    if (type == QG_BF16) return weight_f32 ? by_width<__bf16, true>(a, s) : by_width<__bf16, false>(a, s);
    return weight_f32 ? by_width<_Float16, true>(a, s) : by_width<_Float16, false>(a, s);
}

}  // namespace qg
