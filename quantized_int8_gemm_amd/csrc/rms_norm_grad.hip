// Gradient of the root-mean-square norm.
//
// Mathematics: with g = dy w and u = h r, the normalised row, dx = r (g - u sum(g u)
// / n) (+ dh) and dw = sum over rows of dy u.  u is of ordinary size wherever the
// norm is; r^3, or dy h, leaves fp32's range on rows of 10^13 or 10^-13.  Bound by HBM: dy, h (and dh) are read once.  A
// workgroup walks rows with a fixed set of columns per lane, so dw is added up
// in registers and leaves once, as one row of partial sums per workgroup; a
// second kernel adds those.  No atomics: the order of every sum is fixed.
// 8192 x 4096 with dh: bf16 51.2 us both kernels, 5.2 TB/s, fp32 103.7, 5.2 (a copy of 2
// GiB runs at 4.85); bf16 86.9 us with one row at a time in the registers as single values, which
// left two waves per SIMD nothing in flight between the barrier and the stores.
#include "mx_common.h"

namespace qg {
namespace {

template <int G>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int off = G < 64 ? G / 2 : 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
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
// share a workgroup; their partial sums of dw are added through LDS.  How a row
// passes through the registers:
//  * AHEAD, up to 256 lanes, or 768 of 16-bit values, which have a CU to themselves and
//    so 168 registers: the next row's loads are in flight while this one's sum is
//    completed and its results are stored (3691 x 12288 bf16 67.1 us, HOLD 70.6; fp32
//    would spill, 168 against 145);
//  * HOLD, 512 to 1024 lanes: one row at a time, in at most 128 registers.  Of 512
//    lanes two workgroups share a CU, and one's loads cover the other's barrier (5000
//    x 6144 bf16 54.7 us, AHEAD 59.3); 768 (fp32) and 1024 have the CU to themselves
//    and nothing covers theirs, but with two rows in hand they spill (2000 x 16384
//    55.6, AHEAD 63.9); past 16384 columns of 16 bits too, the weights read again
//    where they are used (1000 x 32768 bf16 105 us, AGAIN 115);
//  * AGAIN, wider rows, where dw alone takes 32 or 64 registers: a row is read
//    once for its sum and again, from the caches, for its results (1000 x 32768 fp32
//    218 us, 2.4 TB/s; 1000 x 65536 bf16 410, 1.3).
// Registers spill from 16385 columns on, in fp32 from 12289 (4 of them, 20 bytes a lane:
// 1000 x 16384 60 us, 4.4 TB/s).  The pairs above are of one run each, before rows were
// normalised first, which costs 0 to 5 % (5000 x 6144 now 56.9, 2000 x 16384 56.4).
enum { AHEAD, HOLD, AGAIN };
constexpr int FEW = 256, MANY = 512;   // lanes of a workgroup that has several rows in hand

template <typename T, int G, int ITER, bool WF32, bool TINY, bool NT>
__global__ __launch_bounds__(G < 256 ? (ITER == 1 ? MANY : FEW) : G, (G < 256 && ITER == 1 ? 4 : G < 512 ? 1 : G == 768 && sizeof(T) == 2 ? 3 : 4)) void rms_norm_grad_kernel(RmsNormGradArgs a) {
    typedef typename std::conditional<WF32, float, T>::type W;
    constexpr int RPW = G < 256 ? (ITER == 1 ? MANY : FEW) / G : 1;   // rows in hand, at most
    constexpr int MODE = G < 512 || (G == 768 && sizeof(T) == 2) ? AHEAD : ITER <= (sizeof(T) == 2 ? 4 : 2) ? HOLD : AGAIN;
    constexpr bool WEIGHTS = ITER <= 2;   // in registers; else read again where they are used
    constexpr int WI = MODE == AGAIN ? 1 : ITER, BUFS = MODE == AHEAD ? 2 : 1;
    __shared__ float red[2][G < 64 ? 1 : G / 64];
    __shared__ float part[RPW > 1 ? (RPW - 1) * G * ITER * 8 : 1];
    const int t = threadIdx.x % G, group = threadIdx.x / G, sub = G < 64 ? group : __builtin_amdgcn_readfirstlane(group);
    const int n = a.n;
    float w[WEIGHTS ? ITER : 1][8], dw[ITER][8];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        if constexpr (WEIGHTS) load_weights<W, TINY>(a.weight, (i * G + t) * 8, n, w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    }
    Pack8<T> yv[BUFS][WI], hv[BUFS][WI], sv[BUFS][WI] = {};
    float rv[BUFS];
    const int rpw = RPW > 1 ? (int)blockDim.x / G : 1, step = (int)gridDim.x * rpw, M = (int)a.M;   // M + step < 2^31
    auto fetch = [&](int row, int i, int buf, int at, bool also) {
        const int c = (i * G + t) * 8;
        load8<TINY, NT && MODE != AGAIN>(reinterpret_cast<const T*>(a.dy) + (int64_t)row * a.ldy, c, n, yv[buf][at]);
        load8<TINY, NT && MODE != AGAIN>(reinterpret_cast<const T*>(a.h) + (int64_t)row * a.ldh, c, n, hv[buf][at]);
        if (also && a.dh != nullptr) load8<TINY, NT>(reinterpret_cast<const T*>(a.dh) + (int64_t)row * a.lddh, c, n, sv[buf][at]);
    };
    auto fetch_row = [&](int row, int buf) {
        if constexpr (MODE != AGAIN) {
#pragma unroll
            for (int i = 0; i < ITER; ++i) fetch(row, i, buf, i, true);
        }
        rv[buf] = a.rstd[row];
    };
    // The weights' address, new to the compiler each time, lest it keep what it read
    // for the next row in registers that are not there.
    auto weight_now = [&]() {
        const void* p = a.weight;
        asm volatile("" : "+s"(p));
        return p;
    };
    auto hold_packed = [&](int buf) {
#pragma unroll
        for (int i = 0; i < WI; ++i) {
            stay_packed(yv[buf][i]);
            stay_packed(hv[buf][i]);
            stay_packed(sv[buf][i]);
        }
    };
    // slot: two in turn, since a wave may be one row ahead of the others' reads
    auto finish_row = [&](int row, int buf, int slot) {
        const float r = rv[buf];
        float dot = 0.f;
        if constexpr (MODE != AGAIN) hold_packed(buf);
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int at = MODE == AGAIN ? 0 : i;
            const int wi = WEIGHTS ? i : 0;
            if constexpr (!WEIGHTS) load_weights<W, TINY>(weight_now(), (i * G + t) * 8, n, w[0]);
            if constexpr (MODE == AGAIN) fetch(row, i, buf, 0, false);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float yu = value(yv[buf][at], e) * (value(hv[buf][at], e) * r);
                dot = __builtin_fmaf(yu, w[wi][e], dot);
                dw[i][e] += yu;
            }
            __builtin_amdgcn_sched_barrier(0);   // one group unpacked at a time
        }
        dot = row_sum<G>(dot, red[slot]);
        const float k = dot / (float)n;
        if constexpr (MODE != AGAIN) hold_packed(buf);
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * G + t) * 8, at = MODE == AGAIN ? 0 : i, wi = WEIGHTS ? i : 0;
            if constexpr (!WEIGHTS) load_weights<W, TINY>(weight_now(), c, n, w[0]);
            if constexpr (MODE == AGAIN) fetch(row, i, buf, 0, true);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e] = r * (value(yv[buf][at], e) * w[wi][e] - value(hv[buf][at], e) * r * k);
                if (a.dh != nullptr) o[e] += value(sv[buf][at], e);
            }
            if (c < n) store8(reinterpret_cast<T*>(a.dx) + (int64_t)row * a.ldx, c, n, pack<T>(o));
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int row = (int)blockIdx.x * rpw + sub;
    if constexpr (MODE == AHEAD) {
        if (row < M) fetch_row(row, 0);
        while (row < M) {
            if (row + step < M) fetch_row(row + step, 1);
            finish_row(row, 0, 0);
            row += step;
            if (row >= M) break;
            if (row + step < M) fetch_row(row + step, 0);
            finish_row(row, 1, 1);
            row += step;
        }
    } else {
        for (int turn = 0; row < M; row += step, turn ^= 1) {
            fetch_row(row, 0);
            finish_row(row, 0, turn);
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
        for (int q = 0; q < rpw - 1; ++q)
#pragma unroll
            for (int i = 0; i < ITER; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[i][e] += part[((q * ITER + i) * 8 + e) * G + t];
    }
    float* out = a.part + (int64_t)blockIdx.x * n;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * G + t) * 8;
        if (c < n) store8(out, c, n, pack<float>(dw[i]));
    }
}

// dw[j] = sum of the partial rows: 32 columns a workgroup (one 128-byte line
// of each row), 32 lanes a column, joined through LDS.
constexpr int SUM_ROWS = 32;
template <typename W>
__global__ __launch_bounds__(32 * SUM_ROWS) void rms_norm_grad_sum(const float* __restrict__ part, int parts, int n,
                                                                   W* __restrict__ dw) {
    __shared__ float red[SUM_ROWS][33];
    const int cl = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + cl;
    float s = 0.f;
    if (c < n) {
#pragma unroll 8
        for (int p = q; p < parts; p += SUM_ROWS) s += part[(int64_t)p * n + c];
    }
    red[q][cl] = s;
    __syncthreads();
    if (q < 4) {
#pragma unroll
        for (int i = 4; i < SUM_ROWS; i += 4) s += red[q + i][cl];
        red[q][cl] = s;
    }
    __syncthreads();
    if (q == 0 && c < n) dw[c] = (W)(s + red[1][cl] + red[2][cl] + red[3][cl]);
}

// Lanes that share a row of up to 1024 columns: as the kernel table below.
int lanes_of(int64_t n) { return n <= 128 ? 16 : n <= 256 ? 32 : 64; }

// Workgroups of the row kernel, each with one partial row of dw: at most two per compute
// unit, or one for wide rows (2000 x 16384: the partial rows of 512 workgroups are a
// quarter of what the gradient itself moves) and for few rows of more than a wave's
// width (512 x 4096 bf16 10.6 us, one workgroup a row 12.2; 512 x 8192 13.5, 17.1; 768 x
// 4096 12.7, 13.6; but 1024 x 1368 12.5, 11.3).
int most_parts(int64_t M, int64_t n) { return n > 8192 || (n > 1024 && M <= 768) ? 256 : 512; }

// Rows that a workgroup has in hand at once.  Up to 512 columns its lanes follow from
// them: eight waves where four would take a second turn (12334 x 478 fp16 14.5 us, four
// 17.5; 7623 x 369 bf16 12.3, 14.7; 60000 x 64 16.7, 20); up to 1024, whose lanes hold
// twice as much, eight are slower (16384 x 1024 bf16 29.7, four 27.1).
int rows_per_group(int64_t M, int64_t n) {
    if (n > 1024) return 1;
    const int few = FEW / lanes_of(n);
    return n > 512 || M <= (int64_t)few * most_parts(M, n) ? few : MANY / lanes_of(n);
}

template <typename T, bool WF32>
hipError_t by_width(const RmsNormGradArgs& a, hipStream_t s) {
    typedef typename std::conditional<WF32, float, T>::type W;
    bool done = a.M == 0;
#define QG_GRAD(G, ITER, LIMIT, TINY, NT)                                                                      \
    if (!done && a.n <= LIMIT) {                                                                               \
        hipLaunchKernelGGL((rms_norm_grad_kernel<T, G, ITER, WF32, TINY, NT>), dim3((unsigned)a.parts),        \
                           dim3(G < 256 ? rows_per_group(a.M, a.n) * G : G), 0, s, a);                                                  \
        done = true;                                                                                           \
    }
    QG_GRAD(16, 1, 7, true, false)
    QG_GRAD(16, 1, 128, false, false)
    QG_GRAD(32, 1, 256, false, false)
    QG_GRAD(64, 1, 512, false, false)
    QG_GRAD(64, 2, 1024, false, false)
    QG_GRAD(256, 1, 2048, false, false)
    // a row or two a workgroup: as many lanes as take it in one piece (512 x 4096 bf16
    // 12.2 us, 256 lanes 13.0; 16 x 8192 fp32 7.2, 512 lanes 8.0)
    if (a.M <= 512) {
        if (a.n > 2048) QG_GRAD(512, 1, 4096, false, false)
        if (a.n > 4096) QG_GRAD(1024, 1, 8192, false, false)
    }
    if constexpr (sizeof(T) == 2) {
        if (whole_lines(a.dy, a.ldy * sizeof(T)) && whole_lines(a.h, a.ldh * sizeof(T)) &&
            (a.dh == nullptr || whole_lines(a.dh, a.lddh * sizeof(T)))) {
            QG_GRAD(256, 2, 4096, false, true)
            QG_GRAD(512, 2, 8192, false, true)
            QG_GRAD(768, 2, 12288, false, true)
            QG_GRAD(1024, 2, 16384, false, true)
        }
    }
    QG_GRAD(256, 2, 4096, false, false)
    QG_GRAD(512, 2, 8192, false, false)
    QG_GRAD(768, 2, 12288, false, false)
    QG_GRAD(1024, 2, 16384, false, false)
    QG_GRAD(1024, 4, 32768, false, false)
    QG_GRAD(1024, 8, 65536, false, false)
#undef QG_GRAD
    if (!done) return hipErrorInvalidValue;
    hipLaunchKernelGGL((rms_norm_grad_sum<W>), dim3((unsigned)((a.n + 31) / 32)), dim3(32 * SUM_ROWS), 0, s, a.part, a.parts, a.n,
                       reinterpret_cast<W*>(a.dweight));
    return hipGetLastError();
}

}  // namespace

// Workgroups of the row kernel, none without rows.
int rms_norm_grad_parts(int64_t M, int64_t n) {
    const int64_t rows = rows_per_group(M, n), groups = (M + rows - 1) / rows;
    return (int)(groups < most_parts(M, n) ? groups : most_parts(M, n));
}

hipError_t launch_rms_norm_grad(const RmsNormGradArgs& a, qg_dtype type, bool weight_f32, hipStream_t s,
                                const char** name) {
    *name = "rms_norm_grad";
    if (type == QG_FP32) return by_width<float, false>(a, s);
    if (type == QG_BF16) return weight_f32 ? by_width<__bf16, true>(a, s) : by_width<__bf16, false>(a, s);
    return weight_f32 ? by_width<_Float16, true>(a, s) : by_width<_Float16, false>(a, s);
}

}  // namespace qg
