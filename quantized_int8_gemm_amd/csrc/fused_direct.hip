// Fused A8W8 products of few outputs, of weights whose rows lie along the sum: each
// workgroup owns TM x TN outputs over all of K, its eight waves take one range of K each and
// read their fragments straight from memory, and the waves' sums meet in LDS, where the
// epilogue takes them.  One launch, no stages, one barrier.
//
// A few rows are bound by streaming the weight: lane (g, i) reads 16 bytes of row i at k-bytes
// 64 kb + 16 g of a step, which is the matrix core's fragment as it lies in memory, NB steps
// in flight a wave.  Small products of more rows are bound by latency: the range of K that a
// wave walks is an eighth of what a tiled kernel's workgroup does.
//
// ANY: rows that are not whole 16-byte pieces, read at any alignment.
#include "fused_common.h"
#include "fused_load.h"
#include "fused_stage.h"

namespace qg {
namespace {

using fused::NOWHERE;
constexpr int WAVES = 8, NT = 64 * WAVES, STEP = 128, KB = STEP / 64;

// GRAD: A is the two planes of the factors, B the branches' weights one behind the other.
template <int FORM, int TM, int TN, int NB, bool ANY>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(2))) void fused_direct_kernel(FusedArgs p) {
    constexpr bool PAIR = FORM == FUSED_PAIR, GRAD = FORM == FUSED_GRAD;
    constexpr int H = FORM == FUSED_ONE ? 1 : 2, AH = GRAD ? 2 : 1, BH = PAIR ? 2 : 1, FM = TM / 16, FN = TN / 16;
    __shared__ __attribute__((aligned(16))) int red[WAVES][H][TM * TN];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int M = p.e.M, N = p.e.N, K = p.k_bytes;
    const int tiles_m = (M + TM - 1) / TM;
    const int tiles = tiles_m * ((N + TN - 1) / TN);
    if (GRAD && (int)blockIdx.x >= tiles) {
        fused::sum_bias<NT>(p, (int)blockIdx.x - tiles, reinterpret_cast<float*>(red));
        return;
    }
    const int tile = xcd_remap(blockIdx.x, tiles);   // an XCD's workgroups share weights
    const int m0 = tile % tiles_m * TM, n0 = tile / tiles_m * TN;
    const int rows = M - m0 < TM ? M - m0 : TM, cols = N - n0 < TN ? N - n0 : TN;
    const int lda = (int)p.lda;
    const int nkb = (p.K + STEP - 1) / STEP, steps = GRAD ? nkb * p.branches : nkb;
    const int a_row = GRAD ? steps * STEP : K;   // bytes of A's rows
    auto a_base = [&](int h) { return p.A[h] + (int64_t)m0 * p.lda; };
    const __amdgpu_buffer_rsrc_t a_rsrc = make_rsrc(a_base(0), (uint32_t)((rows - 1) * lda + a_row));
    const __amdgpu_buffer_rsrc_t a_rsrc2 = GRAD ? make_rsrc(a_base(1), (uint32_t)((rows - 1) * lda + a_row)) : a_rsrc;
    const __amdgpu_buffer_rsrc_t b_rsrc = make_rsrc(p.B[0] + (int64_t)n0 * p.ldb[0], (uint32_t)((cols - 1) * (int)p.ldb[0] + K));
    const __amdgpu_buffer_rsrc_t b_rsrc2 =
        PAIR || (GRAD && p.branches == 2) ? make_rsrc(p.B[1] + (int64_t)n0 * p.ldb[1], (uint32_t)((cols - 1) * (int)p.ldb[1] + K)) : b_rsrc;

    const int mine = (steps + WAVES - 1) / WAVES, first = wave * mine;
    u32x4 av[NB][KB][AH][FM], bv[NB][KB][BH][FN];
    auto fetch = [&](int i, int b) {
        const int step = first + i;
        const bool live = i < mine && step < steps;
        const int branch = GRAD && step >= nkb ? 1 : 0;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int k = step * STEP + 64 * kb + 16 * g, kw = k - branch * nkb * STEP;   // of A's row and the weight's
            if constexpr (ANY) {
#pragma unroll
                for (int h = 0; h < AH; ++h)
#pragma unroll
                    for (int a = 0; a < FM; ++a) {
                        const int r = 16 * a + i16;
                        av[b][kb][h][a] = load16_any(a_base(h) + (int64_t)(r < rows ? r : 0) * p.lda, k, live && r < rows ? a_row : 0);
                    }
#pragma unroll
                for (int h = 0; h < BH; ++h)
#pragma unroll
                    for (int c = 0; c < FN; ++c) {
                        const int r = 16 * c + i16, w = PAIR ? h : branch;
                        bv[b][kb][h][c] = load16_any(p.B[w] + (int64_t)(n0 + (r < cols ? r : 0)) * p.ldb[w], kw, live && r < cols ? K : 0);
                    }
            } else {
                // a piece of A past K gives zeros, and B's there then adds nothing
                const bool in = live && k < a_row;
#pragma unroll
                for (int h = 0; h < BH; ++h)
#pragma unroll
                    for (int c = 0; c < FN; ++c) {
                        const bool second = PAIR ? h == 1 : branch == 1;
                        bv[b][kb][h][c] = buffer_load16(second ? b_rsrc2 : b_rsrc,
                                                        in ? (uint32_t)((16 * c + i16) * (int)p.ldb[second ? 1 : 0] + kw) : NOWHERE, 0u);
                    }
#pragma unroll
                for (int h = 0; h < AH; ++h)
#pragma unroll
                    for (int a = 0; a < FM; ++a)
                        av[b][kb][h][a] = buffer_load16(h == 0 ? a_rsrc : a_rsrc2, in ? (uint32_t)((16 * a + i16) * lda + k) : NOWHERE, 0u);
            }
        }
    };
    v4i acc[H][FM][FN];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int c = 0; c < FN; ++c) acc[h][a][c] = v4i{0, 0, 0, 0};
    auto consume = [&](int b) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int c = 0; c < FN; ++c)
#pragma unroll
                    for (int a = 0; a < FM; ++a) acc[h][a][c] = mfma_i8_16x16x64(bv[b][kb][PAIR ? h : 0][c], av[b][kb][GRAD ? h : 0][a], acc[h][a][c]);
    };
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        fetch(b, b);
        __builtin_amdgcn_sched_barrier(0);
    }

    // The epilogue's own operands, on their way behind the first steps.  Four columns of a row
    // to a lane; a checkpoint's eight lanes of a block stay together (TN = 32 then).
    constexpr int GROUPS = TN / 4, ITEMS = TM * GROUPS;
    const int item = tid, row = item / GROUPS, c4 = item % GROUPS;
    const int m = m0 + row, n = n0 + 4 * c4, count = N - n;
    const bool has = ITEMS >= NT || wave < ITEMS / 64;
    v4f ws[H], bias = {0.f, 0.f, 0.f, 0.f};
    Raw4 res = {};
    float as = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) ws[h] = v4f{0.f, 0.f, 0.f, 0.f};
    if (has && m < M) {
        as = p.e.act_scale[(int64_t)m * p.e.as_stride];
#pragma unroll
        for (int h = 0; h < (GRAD ? 0 : H); ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < count) ws[h][i] = p.e.w_scale[h][(int64_t)(n + i) * p.e.ws_stride[h]];
        if (FORM == FUSED_ONE && p.e.bias != nullptr) bias = load4(p.e.bias + n, count);
        if (FORM == FUSED_ONE && p.e.res != nullptr) res = load_raw4((const char*)p.e.res + ((int64_t)m * p.e.ldr + n) * size_of(p.e.out_type), p.e.out_type, count);
    }

    int i = 0;
    for (; i + NB < mine; i += NB) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            consume(b);
            __builtin_amdgcn_sched_barrier(0);
            fetch(i + NB + b, b);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) consume(b);

    // Register r of block (a, c) in lane (g, i): row 16 a + i, column 16 c + 4 g + r.
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int c = 0; c < FN; ++c) *reinterpret_cast<v4i*>(&red[wave][h][sums_at<TN>(16 * a + i16, 4 * c + g)]) = acc[h][a][c];
    __syncthreads();
    static_assert(ITEMS <= NT && ITEMS % 64 == 0, "an item a lane");
    if (!has) return;
    v4i s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const v4i v = *reinterpret_cast<const v4i*>(&red[w][h][sums_at<TN>(row, c4)]);
#pragma unroll
            for (int q = 0; q < 4; ++q) s[h][q] = (int)((uint32_t)s[h][q] + (uint32_t)v[q]);
        }
    finish_sums<FORM>(p.e, m, n, m < M ? count : 0, s, as, ws, bias, res);
}

template <int FORM, int TM, int TN, int NB>
hipError_t launch_tile(const FusedArgs& a, bool any, hipStream_t s) {
    const int64_t tiles = (int64_t)((a.e.M + TM - 1) / TM) * ((a.e.N + TN - 1) / TN);
    const int64_t grid = tiles + (FORM == FUSED_GRAD && a.dbias != nullptr ? (a.bias_n + 31) / 32 : 0);
    if (grid * NT >= (int64_t)1 << 32) return hipErrorInvalidValue;
    // one step ahead where two would spill
    constexpr int ANY_NB = FORM != FUSED_ONE && TM * TN == 64 * 32 ? 1 : 2;
    if (any) hipLaunchKernelGGL((fused_direct_kernel<FORM, TM, TN, ANY_NB, true>), dim3((unsigned)grid), dim3(NT), 0, s, a);
    else hipLaunchKernelGGL((fused_direct_kernel<FORM, TM, TN, NB, false>), dim3((unsigned)grid), dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <int FORM>
hipError_t launch(const FusedArgs& a, int tm, int tn, bool any, hipStream_t s) {
    if (tn == 16) {
        if (tm == 16) return launch_tile<FORM, 16, 16, 4>(a, any, s);
        if (tm == 32) return launch_tile<FORM, 32, 16, 4>(a, any, s);
        return launch_tile<FORM, 64, 16, 2>(a, any, s);
    }
    if (tm == 16) return launch_tile<FORM, 16, 32, 4>(a, any, s);
    if (tm == 32) return launch_tile<FORM, 32, 32, 2>(a, any, s);
    return launch_tile<FORM, 64, 32, 2>(a, any, s);
}

}  // namespace

hipError_t launch_fused_direct(const FusedArgs& a, int form, int tm, int tn, bool any, hipStream_t s) {
    return form == FUSED_ONE ? launch<FUSED_ONE>(a, tm, tn, any, s)
           : form == FUSED_PAIR ? launch<FUSED_PAIR>(a, tm, tn, any, s) : launch<FUSED_GRAD>(a, tm, tn, any, s);
}

}  // namespace qg
