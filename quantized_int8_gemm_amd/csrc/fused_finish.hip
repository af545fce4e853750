// The epilogue of the fused A8W8 products as a kernel of its own, behind products
// that qgemm_a8w8 left in memory in fp32: for operands that the fused kernels do
// not take (rows that are not whole 16-byte pieces).  Bound by memory.
#include "fused_common.h"

namespace qg {
namespace {

constexpr int NT = 256;

// gpr: groups of four columns a row, a multiple of eight, so that a block's eight
// lanes stay together.
template <bool PAIR>
__global__ __launch_bounds__(NT) void fused_finish_kernel(Epilogue e, const float* __restrict__ z0, const float* __restrict__ z1,
                                                          int m0, int rows, int gpr) {
    const int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int64_t row = t / gpr;
    const int n = (int)(t - row * gpr) * 4;
    const bool live = row < rows && n < e.N;
    const int count = live ? e.N - n : 0;
    const v4f a = load4(z0, row * e.N + n, QG_FP32, count);
    v4f b = {0.f, 0.f, 0.f, 0.f};
    if constexpr (PAIR) b = load4(z1, row * e.N + n, QG_FP32, count);
    v4f bias = {0.f, 0.f, 0.f, 0.f};
    if (!PAIR && e.bias != nullptr) bias = load4(e.bias, n, QG_FP32, count);
    Raw4 res = {};
    if (!PAIR && e.res != nullptr && live) res = load_raw4(e.res, (m0 + row) * e.ldr + n, e.out_type, count);
    finish4<PAIR>(e, live ? m0 + (int)row : e.M, n, a, b, bias, res);
}

__global__ __launch_bounds__(NT) void grad_sum_kernel(const float* __restrict__ z, int64_t stride, int count, int64_t rows, int K,
                                                      int gpr, void* dx, int64_t ld_dx, int type) {
    const int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int64_t row = t / gpr;
    const int n = (int)(t - row * gpr) * 4;
    if (row >= rows || n >= K) return;
    v4f s = load4(z, row * K + n, QG_FP32, K - n);
    for (int i = 1; i < count; ++i) s = s + load4(z + i * stride, row * K + n, QG_FP32, K - n);
    store4(dx, row * ld_dx + n, type, K - n, s);
}

__global__ void clear_kernel(uint32_t* words, int count) {
    const int i = blockIdx.x * NT + threadIdx.x;
    if (i < count) words[i] = 0u;
}

unsigned blocks(int64_t threads) { return (unsigned)((threads + NT - 1) / NT); }

}  // namespace

hipError_t launch_fused_finish(const Epilogue& e, bool pair, const float* z0, const float* z1, int m0, int rows, hipStream_t s) {
    const int gpr = (e.N + 31) / 32 * 8;
    const dim3 grid(blocks((int64_t)rows * gpr));
    if (pair) hipLaunchKernelGGL((fused_finish_kernel<true>), grid, dim3(NT), 0, s, e, z0, z1, m0, rows, gpr);
    else hipLaunchKernelGGL((fused_finish_kernel<false>), grid, dim3(NT), 0, s, e, z0, z1, m0, rows, gpr);
    return hipGetLastError();
}

hipError_t launch_grad_sum(const float* z, int64_t stride, int count, int64_t rows, int64_t K, void* dx, int64_t ld_dx,
                           bool bf16, hipStream_t s) {
    const int gpr = (int)((K + 3) / 4);
    hipLaunchKernelGGL(grad_sum_kernel, dim3(blocks(rows * gpr)), dim3(NT), 0, s, z, stride, count, rows, (int)K, gpr, dx, ld_dx,
                       bf16 ? QG_BF16 : QG_FP16);
    return hipGetLastError();
}

hipError_t launch_clear(uint32_t* words, int count, hipStream_t s) {
    hipLaunchKernelGGL(clear_kernel, dim3(blocks(count)), dim3(NT), 0, s, words, count);
    return hipGetLastError();
}

}  // namespace qg
