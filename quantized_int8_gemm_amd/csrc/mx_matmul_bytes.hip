// MX product for operands of any stride and alignment: each wave computes a
// 16 x 16 tile of the output straight from memory, 128 values of K at a time,
// with 16-byte loads at any byte address.  It serves layouts that the tiled
// and the weight-streaming kernels do not take; nothing is reused between
// waves but through the caches: 4096 columns, K = 4160, MXFP8, 1, 64 and 4096 rows
// 15.9, 16.8 and 694 us a call, where they take 7.7, 10.2 and 101.
#include "mx_mfma.h"

namespace qg {
namespace {

__device__ __forceinline__ u32x4 load16_if(const uint8_t* p, bool ok) {
    u32x4 r{0u, 0u, 0u, 0u};
    if (ok) __builtin_memcpy(&r, p, 16);
    return r;
}

template <bool A8, typename T>
__global__ __launch_bounds__(256) void mx_matmul_bytes_kernel(MxMatmulArgs p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int m = blockIdx.y * 16 + r, n = (blockIdx.x * 4 + wave) * 16 + r;
    const bool m_ok = m < p.M, n_ok = n < p.N;
    const uint8_t* A = p.A + (int64_t)(m_ok ? m : 0) * p.lda;
    const uint8_t* W = p.W + (int64_t)(n_ok ? n : 0) * p.ldw;
    const uint8_t* as = p.as + (int64_t)(m_ok ? m : 0) * p.ldas;
    const uint8_t* ws = p.ws + (int64_t)(n_ok ? n : 0) * p.ldws;
    const int blocks = p.K / 32;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int b0 = 0; b0 < blocks; b0 += 4) {
        const int b = b0 + g;   // the block this lane's scales belong to
        const bool k_ok = b < blocks;
        const uint32_t sa = m_ok && k_ok ? as[b] : 127u, sw = n_ok && k_ok ? ws[b] : 127u;
        const v8i w = words4(load16_if(W + b * 16, n_ok && k_ok));
        v8i a;
        if constexpr (A8) {
            // k = 16 g .. + 15 of the first two blocks, then of the last two
            a = words8(load16_if(A + b0 * 32 + 16 * g, m_ok && b0 + g / 2 < blocks),
                       load16_if(A + b0 * 32 + 64 + 16 * g, m_ok && b0 + 2 + g / 2 < blocks));
        } else {
            a = words4(load16_if(A + b * 16, m_ok && k_ok));
        }
        acc = mfma_mx16<A8>(w, sw, a, sa, acc);
    }
    if (!m_ok) return;
    const float s = p.act_scale != nullptr ? p.act_scale[m] : 1.0f;
    const int c = (blockIdx.x * 4 + wave) * 16 + 4 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < p.N) put<T>(p.out, (int64_t)m * p.ldo + c + i, acc[i] * s);
}

template <bool A8>
hipError_t by_out(const MxMatmulArgs& p, hipStream_t s) {   // M <= ROWS, N <= COLUMNS
    const dim3 grid((unsigned)((p.N + 63) / 64), (unsigned)((p.M + 15) / 16));
    if (p.out_type == QG_FP32)
        hipLaunchKernelGGL((mx_matmul_bytes_kernel<A8, float>), grid, dim3(256), 0, s, p);
    else if (p.out_type == QG_BF16)
        hipLaunchKernelGGL((mx_matmul_bytes_kernel<A8, __bf16>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((mx_matmul_bytes_kernel<A8, _Float16>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_bytes(const MxMatmulArgs& all, bool a8, hipStream_t s, const char** name) {
    *name = "mx_matmul_bytes";
    // one launch's second grid dimension, and the threads of its first
    constexpr int ROWS = 65535 * 16, COLUMNS = 1 << 29;
    const int out_size = all.out_type == QG_FP32 ? 4 : 2;
    for (int n = 0; n < all.N; n += COLUMNS) {
        for (int m = 0; m < all.M; m += ROWS) {
            MxMatmulArgs a = all;
            a.M = all.M - m < ROWS ? all.M - m : ROWS;
            a.N = all.N - n < COLUMNS ? all.N - n : COLUMNS;
            a.A = all.A + m * all.lda;
            a.as = all.as + m * all.ldas;
            a.W = all.W + n * all.ldw;
            a.ws = all.ws + n * all.ldws;
            if (all.act_scale != nullptr) a.act_scale = all.act_scale + m;
            a.out = (char*)all.out + (m * all.ldo + n) * out_size;
            const hipError_t e = a8 ? by_out<true>(a, s) : by_out<false>(a, s);
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace qg
