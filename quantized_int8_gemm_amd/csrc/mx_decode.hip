// MX product for very few rows and columns too few to give every CU a tile of the
// tiled kernels: W is streamed once.
//
// A workgroup of eight waves owns 16 output columns over all of K.  The waves
// take chunks of 512 values of K in turn, straight from memory to registers:
// per 128 values one 16-byte load of W and one (e2m1) or two (e4m3) of A per
// lane, and one 16x16x128 matrix instruction or two; two chunks' loads are in flight at
// once.  Scale bytes come four words at a time, and a lane shifts the byte of its
// block into place.  The waves' partial tiles are added through LDS in a fixed
// order.  Bound by latency: 1 x 2048 x 8192 MXFP4 5.6 us, where 32 x 32 tiles take 7.1 (64
// workgroups instead of 128); MXFP8 6.3 and 10.7.  Its loads of A, which fill 16 rows
// whatever there are, let the tiles win past 3584 columns (MXFP8: 4096), or with more than
// eight rows.
#include "mx_mfma.h"

namespace qg {
namespace {

constexpr int NW = 8, UNROLL = 2;
constexpr uint32_t OUTSIDE = 0xffffff00u;   // past every window

// S16: scale rows are whole 16-byte groups (K a multiple of 512), so four steps'
// scale words come in one load.
template <bool A8, bool S16, typename T>
__global__ __launch_bounds__(NW * 64) void mx_decode_kernel(MxMatmulArgs p) {
    constexpr int AV = A8 ? 2 : 1, ABLK = A8 ? 32 : 16;
    __shared__ float part[NW][4][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int rows_w = p.N - n0 < 16 ? p.N - n0 : 16;
    const int nblk = p.K / 32, lda = (int)p.lda, ldw = (int)p.ldw, ldas = (int)p.ldas, ldws = (int)p.ldws;
    const uint32_t s_span = (uint32_t)((nblk + 3) & ~3);
    const __amdgpu_buffer_rsrc_t w_rsrc = make_rsrc(p.W + (int64_t)n0 * p.ldw, (uint32_t)((rows_w - 1) * ldw + nblk * 16));
    const __amdgpu_buffer_rsrc_t ws_rsrc = make_rsrc(p.ws + (int64_t)n0 * p.ldws, (uint32_t)((rows_w - 1) * ldws) + s_span);
    const __amdgpu_buffer_rsrc_t a_rsrc = make_rsrc(p.A, (uint32_t)((p.M - 1) * lda + nblk * ABLK));
    const __amdgpu_buffer_rsrc_t as_rsrc = make_rsrc(p.as, (uint32_t)((p.M - 1) * ldas) + s_span);

    auto scales = [&](__amdgpu_buffer_rsrc_t rs, uint32_t row, int chunk, bool live, uint32_t* s) {
        if constexpr (S16) {
            const u32x4 v = buffer_load16(rs, live ? row + (uint32_t)chunk * 16u : OUTSIDE, 0);
            s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int b = chunk * 16 + 4 * q;
                s[q] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, (int)(b < nblk ? row + (uint32_t)b : OUTSIDE), 0, 0);
            }
        }
    };

    v4f acc = {0.f, 0.f, 0.f, 0.f};
    const int chunks = (nblk + 15) / 16;
    for (int c0 = wave; c0 < chunks; c0 += NW * UNROLL) {
        u32x4 w[UNROLL][4], a[UNROLL][4][AV];
        uint32_t ws[UNROLL][4], as[UNROLL][4];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int chunk = c0 + u * NW;
            scales(ws_rsrc, (uint32_t)(r * ldws), chunk, chunk < chunks, ws[u]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int b = chunk * 16 + 4 * q + g;   // this lane's block
                w[u][q] = buffer_load16_nt(w_rsrc, b < nblk ? (uint32_t)(r * ldw + b * 16) : OUTSIDE);
            }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int chunk = c0 + u * NW;
            scales(as_rsrc, (uint32_t)(r * ldas), chunk, chunk < chunks, as[u]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int b0 = chunk * 16 + 4 * q;
                const uint32_t row = (uint32_t)(r * lda);
                if constexpr (A8) {
                    // k = 16 g .. + 15 of the step's first two blocks, then of its last two
                    a[u][q][0] = buffer_load16(a_rsrc, b0 + g / 2 < nblk ? row + (uint32_t)(b0 * 32 + 16 * g) : OUTSIDE, 0);
                    a[u][q][1] = buffer_load16(a_rsrc, b0 + 2 + g / 2 < nblk ? row + (uint32_t)(b0 * 32 + 64 + 16 * g) : OUTSIDE, 0);
                } else {
                    a[u][q][0] = buffer_load16(a_rsrc, b0 + g < nblk ? row + (uint32_t)((b0 + g) * 16) : OUTSIDE, 0);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int chunk = c0 + u * NW;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // scale bytes past K may be anything: 0 times the zero codes there
                const bool live = S16 || chunk * 16 + 4 * q + g < nblk;
                const uint32_t sw = live ? ws[u][q] >> (8 * g) : 0u, sa = live ? as[u][q] >> (8 * g) : 0u;
                acc = mfma_mx16<A8>(words4(w[u][q]), sw, A8 ? words8(a[u][q][0], a[u][q][AV - 1]) : words4(a[u][q][0]), sa, acc);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][e][lane] = acc[e];
    __syncthreads();
    if (tid < 256) {   // one thread per element
        const int e = tid >> 6, l = tid & 63;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) s += part[k][e][l];
        const int m = l & 15, n = n0 + 4 * (l >> 4) + e;
        if (m < p.M && n < p.N) put<T>(p.out, (int64_t)m * p.ldo + n, p.act_scale != nullptr ? s * p.act_scale[m] : s);
    }
}

template <bool A8>
hipError_t by_out(const MxMatmulArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.N + 15) / 16)), block(NW * 64);
#define QG_DECODE(T)                                                                                       \
    do {                                                                                                   \
        if (a.K % 512 == 0) hipLaunchKernelGGL((mx_decode_kernel<A8, true, T>), grid, block, 0, s, a);     \
        else hipLaunchKernelGGL((mx_decode_kernel<A8, false, T>), grid, block, 0, s, a);                   \
    } while (0)
    if (a.out_type == QG_FP32) QG_DECODE(float);
    else if (a.out_type == QG_BF16) QG_DECODE(__bf16);
    else QG_DECODE(_Float16);
#undef QG_DECODE
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_decode(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    return a8 ? by_out<true>(a, s) : by_out<false>(a, s);
}

}  // namespace qg
