// The sums of a product whose K was divided among workgroups, added, with the epilogue.
// Bound by memory and the launch; int32 sums are exact in any order.
#include "fused_common.h"

namespace qg {
namespace {

constexpr int NT = 256;

// gpr: groups of four columns a row, a multiple of eight, so that a checkpoint block's
// eight lanes stay together.
template <int FORM>
__global__ __launch_bounds__(NT) void fused_join_kernel(FusedArgs p, int gpr) {
    constexpr int H = FORM == FUSED_ONE ? 1 : 2;
    const Epilogue& e = p.e;
    const int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int64_t row = t / gpr;
    const int n = (int)(t - row * gpr) * 4;
    const bool live = row < e.M && n < e.N;
    const int count = live ? e.N - n : 0;
    v4i s[H];
    v4f ws[H], bias = {0.f, 0.f, 0.f, 0.f};
    Raw4 res = {};
    float as = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) s[h] = v4i{0, 0, 0, 0};
    if (live) {
        const int* from = p.partial + row * p.ld_partial + n;
        const int64_t plane = (int64_t)e.M * p.ld_partial;
#pragma unroll 4
        for (int i = 0; i < p.splits; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const v4i v = *reinterpret_cast<const v4i*>(from + (i * H + h) * plane);
#pragma unroll
                for (int q = 0; q < 4; ++q) s[h][q] = (int)((uint32_t)s[h][q] + (uint32_t)v[q]);
            }
        as = e.act_scale[row * e.as_stride];
        if (FORM == FUSED_ONE && e.res != nullptr) res = load_raw4((const char*)e.res + (row * e.ldr + n) * size_of(e.out_type), e.out_type, count);
        if (FORM == FUSED_ONE && e.bias != nullptr) bias = load4(e.bias + n, count);
    }
    if constexpr (FORM != FUSED_GRAD) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) ws[h][i] = i < count ? e.w_scale[h][(int64_t)(n + i) * e.ws_stride[h]] : 0.f;
    }
    finish_sums<FORM>(e, (int)row, n, count, s, as, ws, bias, res);
}

}  // namespace

hipError_t launch_fused_join(const FusedArgs& a, int form, hipStream_t s) {
    const int gpr = (a.e.N + 31) / 32 * 8;
    const int64_t threads = (int64_t)a.e.M * gpr;
    if (threads >= (int64_t)1 << 32) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((threads + NT - 1) / NT));
    if (form == FUSED_ONE) hipLaunchKernelGGL((fused_join_kernel<FUSED_ONE>), grid, dim3(NT), 0, s, a, gpr);
    else if (form == FUSED_PAIR) hipLaunchKernelGGL((fused_join_kernel<FUSED_PAIR>), grid, dim3(NT), 0, s, a, gpr);
    else hipLaunchKernelGGL((fused_join_kernel<FUSED_GRAD>), grid, dim3(NT), 0, s, a, gpr);
    return hipGetLastError();
}

}  // namespace qg
