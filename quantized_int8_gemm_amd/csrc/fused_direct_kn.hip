// Fused A8W8 products of few outputs, of weights [K,N] (a gradient's of weights [N,K]): as the
// kernel that reads [N,K] weights directly, each workgroup owns TM rows by 64 columns of sums
// over all of K (32 columns of a pair), its eight waves one range of K each, and their sums
// meet in LDS.  A [K,N] weight's fragments are not as they lie in memory, so each wave stages
// 64 rows of K by 64 bytes in LDS of its own, by loads that go there directly, and reads them
// transposed; A's 64-byte pieces of rows go the same way.  A wave waits for its own loads only,
// without a barrier.  Rows that are not whole 16-byte pieces (ANY) come through registers, the
// next step's while one is multiplied: 130 x 1000 x 512 6 us, where laying the weight out again first
// takes 3 and the product 5.  One launch; a tiled kernel's workgroup walks eight times as much of K.
#include "fused_common.h"
#include "fused_load.h"
#include "fused_stage.h"

namespace qg {
namespace {

using fused::NOWHERE;
using fused::kn_slot_of;
constexpr int WAVES = 8, NT = 64 * WAVES, STEP = 64, COLS = 64;

template <int N>
__device__ __forceinline__ void wait_own_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int FORM, int TM, bool ANY>
__global__ __launch_bounds__(NT, 2) void fused_direct_kn_kernel(FusedArgs p) {
    constexpr bool PAIR = FORM == FUSED_PAIR, GRAD = FORM == FUSED_GRAD;
    constexpr int H = FORM == FUSED_ONE ? 1 : 2;
    constexpr int FA = TM / 16 * (GRAD ? 2 : 1), FB = COLS / 16;     // fragments; a gradient's alternate hi, lo
    constexpr int C = PAIR ? COLS / 2 : COLS, RB = C;                // columns of the output; bytes of a weight's staged row
    constexpr int B_LOADS = STEP * COLS / 1024, LOADS = FA + B_LOADS;
    constexpr int STAGE = LOADS * 1024;                              // of a wave
    constexpr int STAGES = ANY ? 1 : STAGE * WAVES * 3 <= 128 * 1024 ? 3 : 2;
    constexpr int RED = WAVES * H * TM * C * 4, LDS = STAGES * STAGE * WAVES > RED ? STAGES * STAGE * WAVES : RED;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int M = p.e.M, N = p.e.N;
    const int tiles_m = (M + TM - 1) / TM, tiles = tiles_m * ((N + C - 1) / C);
    if (GRAD && (int)blockIdx.x >= tiles) {
        fused::sum_bias<NT>(p, (int)blockIdx.x - tiles, reinterpret_cast<float*>(smem));
        return;
    }
    const int tile = xcd_remap(blockIdx.x, tiles);   // an XCD's workgroups share weights
    const int m0 = tile % tiles_m * TM, n0 = tile / tiles_m * C;
    const int rows = M - m0 < TM ? M - m0 : TM, lda = (int)p.lda;
    // whole chunks of 128 of a gradient's factors
    const int nkb = GRAD ? (p.K + 127) / 128 * 2 : (p.K + STEP - 1) / STEP, steps = GRAD ? nkb * p.branches : nkb;
    const int a_row = GRAD ? steps * STEP : p.k_bytes;
    auto a_words = [&](int h) { return rsrc_words(p.A[h] + (int64_t)m0 * p.lda, (uint32_t)((rows - 1) * lda + a_row)); };
    auto b_words = [&](int h) { return rsrc_words(p.B[h] + n0, (uint32_t)((p.K - 1) * (int)p.ldb[h] + (p.b_cols - n0))); };
    const v4i a_rsrc = a_words(0), a_rsrc2 = GRAD ? a_words(1) : a_rsrc;
    const v4i b_rsrc = b_words(0), b_rsrc2 = PAIR || (GRAD && p.branches == 2) ? b_words(1) : b_rsrc;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem + wave * (STAGES * STAGE);
    uint8_t* const own = smem + wave * (STAGES * STAGE);

    // A load moves 16 rows of A by 64 bytes, or 1024 / RB rows of a weight.
    const int ar = lane >> 2, a_col = 16 * dma::kc_slot<STEP>(ar, lane & 3);
    const int br = lane / (RB / 16);
    const int mine = (steps + WAVES - 1) / WAVES, first = wave * mine;
    auto issue = [&](int i, int stage) {
        const int step = first + i;
        const bool live = i < mine && step < steps;
        const bool second = GRAD && step >= nkb;
        const int k = step * STEP, kw = second ? k - nkb * STEP : k;
        const uint32_t to = lds0 + stage * STAGE;
        const bool in = live && k + a_col < a_row;
#pragma unroll
        for (int a = 0; a < FA; ++a) {
            const int r = (GRAD ? a >> 1 : a) * 16 + ar;
            dma16(GRAD && (a & 1) ? a_rsrc2 : a_rsrc, in ? (uint32_t)(r * lda + k + a_col) : NOWHERE, to + a * 1024);
        }
#pragma unroll
        for (int q = 0; q < B_LOADS; ++q) {
            const int half = PAIR ? q / (B_LOADS / 2) : 0, r = (PAIR ? q % (B_LOADS / 2) : q) * (1024 / RB) + br;
            const int ld = (int)p.ldb[PAIR ? half : second ? 1 : 0];
            const uint32_t from = live ? (uint32_t)(kw + r) * (uint32_t)ld + 16 * kn_slot_of<RB>(r, lane % (RB / 16)) : NOWHERE;
            if (PAIR ? half == 1 : second) dma16(b_rsrc2, from, to + (FA + q) * 1024);
            else dma16(b_rsrc, from, to + (FA + q) * 1024);
        }
    };

    v4i acc[FA][FB];
#pragma unroll
    for (int a = 0; a < FA; ++a)
#pragma unroll
        for (int b = 0; b < FB; ++b) acc[a][b] = v4i{0, 0, 0, 0};
    auto compute = [&](int stage) {
        const uint8_t* S = own + stage * STAGE;
        u32x4 af[FA], bf[FB];
#pragma unroll
        for (int a = 0; a < FA; ++a) af[a] = *reinterpret_cast<const u32x4*>(S + (16 * a + i16) * STEP + (dma::kc_slot<STEP>(i16, g) << 4));
#pragma unroll
        for (int j = 0; j < FB; ++j) {
            // lane (g, i) addresses rows 16 g + i / 2 (and + 8), bytes 8 (i & 1) .. of the fragment's 16 columns
            const int r = 16 * g + (i16 >> 1), seg = PAIR ? j & 1 : j;
            const uint8_t* base = S + FA * 1024 + (PAIR && j >= FB / 2 ? STEP * RB : 0) + 8 * (i16 & 1);
            const dma::v2i lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) dma::v2i*)(base + r * RB + (kn_slot_of<RB>(r, seg) << 4)));
            const dma::v2i hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) dma::v2i*)(base + (r + 8) * RB + (kn_slot_of<RB>(r + 8, seg) << 4)));
            bf[j] = u32x4{(uint32_t)lo.x, (uint32_t)lo.y, (uint32_t)hi.x, (uint32_t)hi.y};
        }
#pragma unroll
        for (int a = 0; a < FA; ++a)
#pragma unroll
            for (int b = 0; b < FB; ++b) acc[a][b] = mfma_i8_16x16x64(bf[b], af[a], acc[a][b]);
    };

    // The epilogue's own operands, ahead of the loop: four columns of a row to a lane; a
    // checkpoint's eight lanes of a block stay together.
    constexpr int GROUPS = C / 4, ITEMS = TM * GROUPS;
    static_assert(ITEMS <= NT && ITEMS % 64 == 0, "an item a lane");
    const int row = tid / GROUPS, c4 = tid % GROUPS;
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
        if (FORM == FUSED_ONE && p.e.res != nullptr)
            res = load_raw4((const char*)p.e.res + ((int64_t)m * p.e.ldr + n) * size_of(p.e.out_type), p.e.out_type, count);
    }

    if constexpr (ANY) {
        u32x4 ra[FA], rb[B_LOADS];
        auto fetch = [&](int i) {
            const int step = first + i;
            const bool live = i < mine && step < steps, second = GRAD && step >= nkb;
            const int k = step * STEP, kw = second ? k - nkb * STEP : k;
#pragma unroll
            for (int a = 0; a < FA; ++a) {
                const int r = (GRAD ? a >> 1 : a) * 16 + ar;
                const int8_t* base = p.A[GRAD ? a & 1 : 0] + (int64_t)(m0 + (r < rows ? r : 0)) * p.lda;
                ra[a] = load16_any(base, k + a_col, live && r < rows ? a_row : 0);
            }
#pragma unroll
            for (int q = 0; q < B_LOADS; ++q) {
                const int half = PAIR ? q / (B_LOADS / 2) : 0, r = (PAIR ? q % (B_LOADS / 2) : q) * (1024 / RB) + br, row = kw + r;
                const int w = PAIR ? half : second ? 1 : 0;
                rb[q] = load16_any(p.B[w] + (int64_t)(row < p.K ? row : 0) * p.ldb[w], n0 + 16 * kn_slot_of<RB>(r, lane % (RB / 16)),
                                   live && row < p.K ? N : 0);
            }
        };
        fetch(0);
        for (int i = 0; i < mine; ++i) {
            // a wave's LDS accesses are in order: these follow the last turn's reads
#pragma unroll
            for (int a = 0; a < FA; ++a) *reinterpret_cast<u32x4*>(own + a * 1024 + lane * 16) = ra[a];
#pragma unroll
            for (int q = 0; q < B_LOADS; ++q) *reinterpret_cast<u32x4*>(own + (FA + q) * 1024 + lane * 16) = rb[q];
            asm volatile("" ::: "memory");
            fetch(i + 1);
            compute(0);
            asm volatile("" ::: "memory");
        }
    } else {
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) issue(i, i);
        int at = 0;
        for (int i = 0; i < mine; ++i) {
            // the stage that is filled now was read in the last turn, and those reads are done
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            issue(i + STAGES - 1, at == 0 ? STAGES - 1 : at - 1);
            wait_own_loads<LOADS * (STAGES - 1)>();   // all but the later stages' are there
            compute(at);
            at = at + 1 == STAGES ? 0 : at + 1;
        }
        wait_own_loads<0>();
    }
    __syncthreads();   // every wave is done with its stages
    int* const red = reinterpret_cast<int*>(smem);
#pragma unroll
    for (int a = 0; a < FA; ++a)
#pragma unroll
        for (int b = 0; b < FB; ++b) {
            const int h = GRAD ? a & 1 : PAIR ? b / (FB / 2) : 0;
            const int rr = (GRAD ? a >> 1 : a) * 16 + i16, c = (PAIR ? b % (FB / 2) : b) * 4 + g;
            *reinterpret_cast<v4i*>(red + (wave * H + h) * TM * C + sums_at<C>(rr, c)) = acc[a][b];
        }
    __syncthreads();
    if (!has) return;
    v4i s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const v4i v = *reinterpret_cast<const v4i*>(red + (w * H + h) * TM * C + sums_at<C>(row, c4));
#pragma unroll
            for (int q = 0; q < 4; ++q) s[h][q] = (int)((uint32_t)s[h][q] + (uint32_t)v[q]);
        }
    finish_sums<FORM>(p.e, m, n, m < M ? count : 0, s, as, ws, bias, res);
}

template <int FORM, int TM, bool ANY>
hipError_t launch_tile(const FusedArgs& a, hipStream_t s) {
    constexpr int C = FORM == FUSED_PAIR ? COLS / 2 : COLS;
    const int64_t tiles = (int64_t)((a.e.M + TM - 1) / TM) * ((a.e.N + C - 1) / C);
    const int64_t grid = tiles + (FORM == FUSED_GRAD && a.dbias != nullptr ? (a.bias_n + 31) / 32 : 0);
    if (grid * NT >= (int64_t)1 << 32) return hipErrorInvalidValue;
    hipLaunchKernelGGL((fused_direct_kn_kernel<FORM, TM, ANY>), dim3((unsigned)grid), dim3(NT), 0, s, a);
    return hipGetLastError();
}

// A gradient's 32 rows, two fragments each, gained nothing over 16 or over tiles (500 and 1000 x 512 over 4000
// 29 and 39 us, tiles of 64 x 128 28 and 35).
template <int FORM, bool ANY>
hipError_t launch(const FusedArgs& a, int tm, hipStream_t s) {
    if (tm == 16) return launch_tile<FORM, 16, ANY>(a, s);
    if constexpr (FORM == FUSED_GRAD) return hipErrorInvalidValue;
    else return launch_tile<FORM, 32, ANY>(a, s);
}

template <int FORM>
hipError_t launch(const FusedArgs& a, int tm, bool any, hipStream_t s) {
    return any ? launch<FORM, true>(a, tm, s) : launch<FORM, false>(a, tm, s);
}

}  // namespace

hipError_t launch_fused_direct_kn(const FusedArgs& a, int form, int tm, bool any, hipStream_t s) {
    return form == FUSED_ONE ? launch<FUSED_ONE>(a, tm, any, s)
           : form == FUSED_PAIR ? launch<FUSED_PAIR>(a, tm, any, s) : launch<FUSED_GRAD>(a, tm, any, s);
}

}  // namespace qg
