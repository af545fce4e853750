// Tiled int8 matrix-core kernel of the fused A8W8 products and of their gradients;
// included by one translation unit per form:
//   ONE   one product;
//   PAIR  a gate's and an up projection's products of the same A;
//   GRAD  the product of a gradient's factors with the weight: the two int8 planes of
//         the factors (256 hi + lo) as A, the weights one behind the other along the sum.
//
// The two products of PAIR and GRAD meet in the registers of one lane: a tile's
// 16-column (PAIR) or 16-row (GRAD) fragments alternate between the two operands,
// so fragment 2 j and 2 j + 1 of a wave hold the same outputs of both.  Everything else
// is one int8 product, bound by the matrix cores where there are many rows.
//
// A workgroup computes a BM x BN tile of sums (BN / 2 columns of a pair, BM / 2 rows of
// a gradient), K in chunks of 128 bytes:
//  * DMA: chunks go global -> LDS directly (buffer_load ... lds), in a ring of RING
//    stages, the next ones in flight while one is multiplied.  Wants rows of whole
//    16-byte pieces.  A piece of A past K is asked for past the buffer's end, which
//    gives zeros; whatever B holds there then adds nothing.
//    Tiles of 64 and 128 rows are bound by these loads, 75 bytes a nanosecond to a CU and 14
//    TB/s to all (300 x 4096 x 14336 38 us): the next chunk's fragments read under this one's
//    products, and waves that share a tile by parts of K, so that half as much is read from LDS,
//    took the same time.
//  * RING 0: through registers with loads of any alignment, the next chunk's in flight
//    while this one is multiplied, and one stage.
//  * Fragments as in the int8 products: K-contiguous operands by ds_read_b128, [K,N]
//    weights by ds_read_b64_tr_b8; segments swizzled so that both are free of bank
//    conflicts.  Operands are swapped in v_mfma_i32_16x16x64_i8, so a lane's four
//    registers are four consecutive columns of a row.
//  * The int32 sums pass through LDS, so that each lane finishes four columns of a row
//    and whole rows leave together; the epilogue is the same code for every kernel.
//    With p.partial, K is divided among workgroups (blockIdx.y), each leaves its sums there
//    as they are, and a second kernel adds them and finishes.
#pragma once
#include "fused_common.h"
#include "fused_kernels.h"
#include "fused_load.h"
#include "fused_stage.h"
#include "int8_dma_impl.h"

namespace qg {
namespace fused {

constexpr int BK = 128;          // bytes of K per chunk
constexpr int KB = BK / 64;      // matrix instructions along it
constexpr int GROUP_M = 8;

// 128 x 128 tiles on two stages, two workgroups to a CU: four waves a SIMD asked for.
template <int MODE, int BM, int BN, int WM, int WN, bool B_KMAJOR, int RING>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, (BM == 128 && RING == 2 ? 4 : 2)) void fused_tiled_kernel(FusedArgs p) {
    constexpr bool PAIR = MODE == FUSED_PAIR, GRAD = MODE == FUSED_GRAD;
    constexpr int H = MODE == FUSED_ONE ? 1 : 2;
    constexpr int BMR = GRAD ? BM / 2 : BM, BNR = PAIR ? BN / 2 : BN;   // rows and columns of the output
    constexpr int NT = (BM / WM) * (BN / WN) * 64;
    constexpr int ROUND = NT * 16;                                     // bytes that one load round moves
    constexpr int WAVES_N = BN / WN, WAVES_M = BM / WM, FM = WM / 16, FN = WN / 16;
    constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
    constexpr int A_ROUNDS = A_BYTES / ROUND, B_ROUNDS = B_BYTES / ROUND;
    constexpr bool DMA = RING > 0;
    constexpr int STAGES = DMA ? RING : 1;
    constexpr int LOADS = A_ROUNDS + B_ROUNDS;                         // per lane and chunk
    constexpr int RB = PAIR ? BN / 2 : BN;                             // row bytes of a [K,N] tile (of each half)
    static_assert(NT == 512, "eight waves");
    static_assert(A_BYTES % ROUND == 0 && B_BYTES % ROUND == 0 && (BK * RB) % ROUND == 0, "whole load rounds");
    static_assert(LOADS * (STAGES - 2) < 64, "vmcnt range");
    static_assert((!GRAD || FM % 2 == 0) && (!PAIR || FN % 2 == 0), "fragments in pairs");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * STAGE];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int g = lane >> 4, i16 = lane & 15;

    const int M = p.e.M, N = p.e.N;
    const int tiles_m = (M + BMR - 1) / BMR, tiles_n = (N + BNR - 1) / BNR;
    int tm, tn;
    if constexpr (GRAD) {
        if ((int)blockIdx.x >= tiles_m * tiles_n) {
            if (blockIdx.y == 0) sum_bias<NT>(p, (int)blockIdx.x - tiles_m * tiles_n, reinterpret_cast<float*>(smem));
            return;
        }
    }
    tile_coords(xcd_remap(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, GROUP_M, tm, tn);
    const int m0 = tm * BMR, n0 = tn * BNR;
    const int rows_a = M - m0 < BMR ? M - m0 : BMR;
    const int cols_b = N - n0 < BNR ? N - n0 : BNR;
    const int lda = (int)p.lda;
    // K of one weight, and chunks of it; of GRAD's planes each weight's part is whole chunks
    const int K = p.K, nkb = (K + BK - 1) / BK, all = GRAD ? nkb * p.branches : nkb;
    // this workgroup's chunks: all, or one split's
    const int k0 = p.partial != nullptr ? (int)blockIdx.y * p.split_chunks : 0;
    const int nk = p.partial != nullptr && all - k0 > p.split_chunks ? k0 + p.split_chunks : all;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    // A wave's load instruction covers eight LDS rows of a K-contiguous tile, all of one
    // fragment, which is one of the even (first operand) or the odd ones in every round.
    const int half = (wave >> 1) & 1;
    const int8_t* const A = p.A[GRAD ? half : 0] + (int64_t)m0 * p.lda;
    auto b_base = [&](int h) {
        return B_KMAJOR ? p.B[h] + (int64_t)n0 * p.ldb[h] : p.B[h] + n0;
    };
    auto b_words = [&](int h) {
        const int ld = (int)p.ldb[h];
        return rsrc_words(b_base(h), (uint32_t)(B_KMAJOR ? (cols_b - 1) * ld + p.k_bytes : (K - 1) * ld + (p.b_cols - n0)));
    };
    v4i a_rsrc = {}, b_rsrc = {}, b_rsrc2 = {};   // b_rsrc2: the second half of a [K,N] pair, or GRAD's second weight
    if constexpr (DMA) {
        a_rsrc = rsrc_words(A, (uint32_t)((rows_a - 1) * lda + (GRAD ? all * BK : p.k_bytes)));
        b_rsrc = b_words(PAIR && B_KMAJOR ? half : 0);
        if ((PAIR && !B_KMAJOR) || (GRAD && p.branches == 2)) b_rsrc2 = b_words(1);
    }

    // Place of this lane's 16 bytes in each load round: LDS byte q * ROUND + wave * 1024 +
    // lane * 16, and what lies there.
    auto kc_row = [&](int q) { return (q * ROUND + wave * 1024 + lane * 16) / BK; };
    const int kc_col = 16 * dma::kc_slot<BK>(wave * 8 + (lane >> 3), lane & 7);   // rounds are multiples of 16 rows
    auto real = [](int r) { return (r >> 5) * 16 + (r & 15); };                    // of alternating fragments
    uint32_t a_off[A_ROUNDS], b_off[B_ROUNDS], b_off2[GRAD ? B_ROUNDS : 1];
#pragma unroll
    for (int q = 0; q < A_ROUNDS; ++q) a_off[q] = (uint32_t)((GRAD ? real(kc_row(q)) : kc_row(q)) * lda + kc_col);
    auto b_place = [&](int q, int ld) {
        if constexpr (B_KMAJOR) {
            return (uint32_t)((PAIR ? real(kc_row(q)) : kc_row(q)) * ld + kc_col);
        } else {
            const int o = (q * ROUND) % (BK * RB) + wave * 1024 + lane * 16;
            const int r = o / RB;
            return (uint32_t)(r * ld + 16 * kn_slot_of<RB>(r, (o % RB) / 16));
        }
    };
    auto half_of = [](int q) { return PAIR && !B_KMAJOR ? (q * ROUND) / (BK * RB) : 0; };
#pragma unroll
    for (int q = 0; q < B_ROUNDS; ++q) {
        b_off[q] = b_place(q, (int)p.ldb[PAIR ? (B_KMAJOR ? half : half_of(q)) : 0]);
        if constexpr (GRAD) b_off2[q] = b_place(q, (int)p.ldb[1]);
    }

    u32x4 ar[DMA ? 1 : A_ROUNDS], br[DMA ? 1 : B_ROUNDS];
    auto issue = [&](int kt, int stage) {
        const bool second = GRAD && kt >= nkb;           // of GRAD's weights
        const int kc = second ? kt - nkb : kt;           // chunk of this weight
        if constexpr (DMA) {
            const uint32_t sbase = lds0 + stage * STAGE + wave * 1024;
            const uint32_t ka = (uint32_t)(kt * BK);
            if (!GRAD && (kt + 1) * BK > p.k_bytes) {
                const bool in = kt * BK + kc_col < p.k_bytes;
#pragma unroll
                for (int q = 0; q < A_ROUNDS; ++q) dma16(a_rsrc, in ? a_off[q] + ka : NOWHERE, sbase + q * ROUND);
            } else {
#pragma unroll
                for (int q = 0; q < A_ROUNDS; ++q) dma16(a_rsrc, a_off[q] + ka, sbase + q * ROUND);
            }
            if (GRAD && second) {
                const uint32_t kb = B_KMAJOR ? (uint32_t)(kc * BK) : (uint32_t)(kc * BK) * (uint32_t)p.ldb[1];
#pragma unroll
                for (int q = 0; q < B_ROUNDS; ++q) dma16(b_rsrc2, b_off2[q] + kb, sbase + A_BYTES + q * ROUND);
            } else {
                const uint32_t kb = B_KMAJOR ? (uint32_t)(kc * BK) : (uint32_t)(kc * BK) * (uint32_t)p.ldb[0];
                const uint32_t kb2 = PAIR && !B_KMAJOR ? (uint32_t)(kc * BK) * (uint32_t)p.ldb[1] : 0u;
#pragma unroll
                for (int q = 0; q < B_ROUNDS; ++q) {
                    if (half_of(q) == 1) dma16(b_rsrc2, b_off[q] + kb2, sbase + A_BYTES + q * ROUND);
                    else dma16(b_rsrc, b_off[q] + kb, sbase + A_BYTES + q * ROUND);
                }
            }
        } else {
#pragma unroll
            for (int q = 0; q < A_ROUNDS; ++q) {
                const int r = GRAD ? real(kc_row(q)) : kc_row(q);
                ar[q] = load16_any(A + (int64_t)(r < rows_a ? r : 0) * p.lda, kt * BK + kc_col, r < rows_a ? (GRAD ? all * BK : K) : 0);
            }
#pragma unroll
            for (int q = 0; q < B_ROUNDS; ++q) {
                const int h = PAIR ? (B_KMAJOR ? half : half_of(q)) : second ? 1 : 0;
                if constexpr (B_KMAJOR) {
                    const int r = PAIR ? real(kc_row(q)) : kc_row(q);
                    br[q] = load16_any(b_base(h) + (int64_t)(r < cols_b ? r : 0) * p.ldb[h], kc * BK + kc_col, r < cols_b ? K : 0);
                } else {
                    const int o = (q * ROUND) % (BK * RB) + wave * 1024 + lane * 16;
                    const int r = o / RB, k = kc * BK + r;
                    br[q] = load16_any(p.B[h] + (int64_t)(k < K ? k : 0) * p.ldb[h], n0 + 16 * kn_slot_of<RB>(r, (o % RB) / 16),
                                       k < K ? N : 0);
                }
            }
        }
    };
    auto put = [&]() {   // what issue() read into registers, to LDS
        if constexpr (!DMA) {
#pragma unroll
            for (int q = 0; q < A_ROUNDS; ++q) *reinterpret_cast<u32x4*>(smem + q * ROUND + wave * 1024 + lane * 16) = ar[q];
#pragma unroll
            for (int q = 0; q < B_ROUNDS; ++q) *reinterpret_cast<u32x4*>(smem + A_BYTES + q * ROUND + wave * 1024 + lane * 16) = br[q];
        }
    };

    // The epilogue's own operands, on their way before everything else: the column scales of
    // this lane's four columns, and a row's scale for the others by LDS (a load between the
    // epilogue's stores would wait for those before it: 29 us of a 256 x 256 tile were that).
    // CPT lanes share a row; sums of row rr and columns c .. c + 3 of operand h lie at chunk
    // (c / 4) ^ (rr & 15) of row h * PR + rr.
    constexpr int PASSES = BM * BN * 4 <= STAGES * STAGE ? 1 : BM * BN * 2 <= STAGES * STAGE ? 2 : 4;
    static_assert(WAVES_M % PASSES == 0 && BM * BN * 4 / PASSES <= STAGES * STAGE, "passes of whole wave rows");
    constexpr int PW = WAVES_M / PASSES, PR = BMR / PASSES, CPT = BNR / 4, ROWS_AT_ONCE = NT / CPT;
    static_assert(CPT >= 16 && NT % CPT == 0 && PR % ROWS_AT_ONCE == 0 && BMR <= NT, "whole rounds of rows");
    __shared__ float as_rows[BMR];
    const int c4 = tid % CPT, n = n0 + 4 * c4, count = N - n;
    const bool whole = rows_a == BMR && cols_b == BNR;   // no row or column outside
    float as_mine = 0.f;
    v4f ws[H], bias = {0.f, 0.f, 0.f, 0.f};
    if (p.partial == nullptr) {
        if (tid < rows_a) as_mine = p.e.act_scale[(int64_t)(m0 + tid) * p.e.as_stride];
        if constexpr (!GRAD) {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) ws[h][i] = i < count ? p.e.w_scale[h][(int64_t)(n + i) * p.e.ws_stride[h]] : 0.f;
            if (!PAIR && p.e.bias != nullptr) bias = load4(p.e.bias + n, count);
        }
    }

    v4i acc[FM][FN];
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b) acc[a][b] = v4i{0, 0, 0, 0};

    auto a_rd_at = [&](int kb) { return (wm * WM + i16) * BK + (dma::kc_slot<BK>(i16, 4 * kb + g) << 4); };
    auto read_b = [&](const uint8_t* S, int kb, u32x4* bf) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if constexpr (B_KMAJOR) {
                bf[j] = *reinterpret_cast<const u32x4*>(S + A_BYTES + (wn * WN + j * 16 + i16) * BK +
                                                        (dma::kc_slot<BK>(i16, 4 * kb + g) << 4));
            } else {
                // lane (g, i) addresses k-rows 16 g + i / 2 (and + 8), bytes 8 (i & 1) .. of the
                // fragment's 16 columns, and receives column i of those eight rows
                const int r = 16 * g + (i16 >> 1);
                const int seg = PAIR ? wn * (WN / 32) + (j >> 1) : wn * (WN / 16) + j;
                const uint8_t* base = S + A_BYTES + (PAIR && (j & 1) ? BK * RB : 0) + kb * 64 * RB + 8 * (i16 & 1);
                const dma::v2i lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (__attribute__((address_space(3))) dma::v2i*)(base + r * RB + (kn_slot_of<RB>(r, seg) << 4)));
                const dma::v2i hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (__attribute__((address_space(3))) dma::v2i*)(base + (r + 8) * RB + (kn_slot_of<RB>(r + 8, seg) << 4)));
                bf[j] = u32x4{(uint32_t)lo.x, (uint32_t)lo.y, (uint32_t)hi.x, (uint32_t)hi.y};
            }
        }
    };

    // Every fragment of B is read at the start of a chunk, A's one ahead of its products; the
    // next chunk's loads are issued right after the first reads.
    auto compute = [&](int stage, int next, int next_stage) {
        const uint8_t* S = smem + stage * STAGE;
        u32x4 bfs[KB][FN];
        read_b(S, 0, bfs[0]);
        u32x4 af_next = *reinterpret_cast<const u32x4*>(S + a_rd_at(0));
#pragma unroll
        for (int kb = 1; kb < KB; ++kb) read_b(S, kb, bfs[kb]);
        __builtin_amdgcn_sched_barrier(0);
        if (next < nk) issue(next, next_stage);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int a_rd = a_rd_at(kb);
#pragma unroll
            for (int a = 0; a < FM; ++a) {
                const u32x4 af = af_next;
                if (a + 1 < FM) af_next = *reinterpret_cast<const u32x4*>(S + a_rd + (a + 1) * 16 * BK);
                else if (kb + 1 < KB) af_next = *reinterpret_cast<const u32x4*>(S + a_rd_at(kb + 1));
                __builtin_amdgcn_sched_barrier(0);   // the next read ahead of this block's products
#pragma unroll
                for (int b = 0; b < FN; ++b) acc[a][b] = mfma_i8_16x16x64(bfs[kb][b], af, acc[a][b]);
            }
        }
    };

    if constexpr (DMA) {
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i)
            if (k0 + i < nk) issue(k0 + i, i);
        int at = 0;
        for (int kt = k0; kt < nk; ++kt) {
            // chunk kt has landed once at most the later ones are on their way
            if (STAGES > 2 && kt + STAGES - 2 < nk) wait_vmcnt<LOADS * (STAGES - 2)>();
            else if (STAGES > 2 && kt + 1 < nk) wait_vmcnt<LOADS>();
            else wait_vmcnt<0>();
            __syncthreads();
            compute(at, kt + STAGES - 1, at == 0 ? STAGES - 1 : at - 1);
            at = at + 1 == STAGES ? 0 : at + 1;
        }
    } else {
        issue(k0, 0);
        for (int kt = k0; kt < nk; ++kt) {
            if (kt > k0) __syncthreads();   // every wave has read the last chunk
            put();
            __syncthreads();
            compute(0, kt + 1, 0);
        }
    }

    // Places of a lane's four columns, from the tile's corner (one address in scalar registers)
    // by 32 bits, which the host has checked, a row at a time.
    const int size = size_of(p.e.out_type);
    const int64_t corner = (int64_t)m0;
    char* const out0 = reinterpret_cast<char*>(p.e.out) + (corner * p.e.ldo + n0) * size;
    const char* const res0 = reinterpret_cast<const char*>(p.e.res) + (corner * p.e.ldr + n0) * size;
    // Residuals, U turns ahead: one read where it is used would cost a memory latency, and
    // each wait for them is also one for the stores before (8192 x 8192 x 8192, bf16: 547 us so).
    // Where registers are few, two.
    constexpr int TURNS = PR / ROWS_AT_ONCE, U = BM == 256 || RING == 2 ? 2 : TURNS < 4 ? TURNS : 4;
    Raw4 next[U];
    auto fetch = [&](int pass, int q0) {
        if (MODE != FUSED_ONE || p.e.res == nullptr) return;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int rr = pass * PR + (q0 + u) * ROWS_AT_ONCE + tid / CPT;
            next[u] = Raw4{};
            if (rr < rows_a) next[u] = load_raw4(res0 + ((uint32_t)rr * (uint32_t)p.e.ldr + 4 * c4) * size, p.e.out_type, count);
        }
    };
    if (p.partial == nullptr) {
        if (BMR == NT || tid < BMR) as_rows[tid] = as_mine;
        fetch(0, 0);
    }
    int* const stage = reinterpret_cast<int*>(smem);
    __syncthreads();   // every wave has read the last chunk
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
        if (pass > 0) __syncthreads();   // the previous pass has been read
        if (wm / PW == pass) {
#pragma unroll
            for (int a = 0; a < FM; ++a)
#pragma unroll
                for (int b = 0; b < FN; ++b) {
                    const int h = GRAD ? a & 1 : PAIR ? b & 1 : 0;
                    const int rr = (wm % PW) * (GRAD ? WM / 2 : WM) + (GRAD ? a >> 1 : a) * 16 + i16;
                    const int c = wn * (PAIR ? WN / 2 : WN) + (PAIR ? b >> 1 : b) * 16 + 4 * g;
                    *reinterpret_cast<v4i*>(stage + (h * PR + rr) * BNR + (((c >> 2) ^ (rr & 15)) << 2)) = acc[a][b];
                }
        }
        __syncthreads();
        // `full`: no lane has anything outside
        auto turns = [&](auto full) {
            constexpr bool FULL = decltype(full)::value;
            const uint32_t r0 = pass * PR + tid / CPT;
            uint32_t at_out = (r0 * (uint32_t)p.e.ldo + 4 * c4) * size;
            uint32_t at_code = r0 * (uint32_t)p.e.ld_ckpt + 4 * c4, at_block = (r0 * (uint32_t)p.e.ld_ckpt_scale + c4 / 8) * 4;
#pragma unroll 1
            for (int q0 = 0; q0 < TURNS; q0 += U) {
                Raw4 res[U];
#pragma unroll
                for (int u = 0; u < U; ++u) res[u] = next[u];
                if (q0 + U < TURNS) fetch(pass, q0 + U);
                else if (pass + 1 < PASSES) fetch(pass + 1, 0);
                v4f z0[U], z1[U];
                Goes to[U];
                int live[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int rr = (q0 + u) * ROWS_AT_ONCE + tid / CPT;
                    live[u] = FULL ? 4 : pass * PR + rr < rows_a ? count : 0;
                    const int at = rr * BNR + ((c4 ^ (rr & 15)) << 2);
                    const v4i s0 = *reinterpret_cast<const v4i*>(stage + at);
                    v4i s1 = {0, 0, 0, 0};
                    if constexpr (H == 2) s1 = *reinterpret_cast<const v4i*>(stage + PR * BNR + at);
                    const float as = as_rows[pass * PR + rr];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (GRAD) {
                            z0[u][i] = __builtin_fmaf((float)s0[i], 256.f, (float)s1[i]) * as;
                        } else {
                            z0[u][i] = (float)s0[i] * as * ws[0][i];
                            if constexpr (PAIR) z1[u][i] = (float)s1[i] * as * ws[1][i];
                        }
                    }
                    to[u].out = out0 + at_out;
                    to[u].starts = c4 % 8 == 0;
#pragma unroll
                    for (int h = 0; h < (GRAD ? 0 : H); ++h) {
                        to[u].code[h] = p.e.ckpt[h] + (corner * p.e.ld_ckpt + n0) + at_code;
                        to[u].scale[h] = reinterpret_cast<float*>(reinterpret_cast<char*>(p.e.ckpt_scale[h] + (corner * p.e.ld_ckpt_scale + n0 / INT8_BLOCK)) + at_block);
                    }
                    at_out += (uint32_t)(ROWS_AT_ONCE * p.e.ldo) * size;
                    at_code += (uint32_t)(ROWS_AT_ONCE * p.e.ld_ckpt);
                    at_block += (uint32_t)(ROWS_AT_ONCE * p.e.ld_ckpt_scale) * 4;
                }
                if constexpr (GRAD) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (live[u] > 0) store4(to[u].out, p.e.out_type, live[u], z0[u]);
                } else {
                    finish<PAIR, FULL, U>(p.e, to, live, z0, z1, bias, res);
                }
            }
        };
        if (p.partial != nullptr) {
            for (int q = 0; q < TURNS; ++q) {
                const int rr = q * ROWS_AT_ONCE + tid / CPT, m = pass * PR + rr;
                const int at = rr * BNR + ((c4 ^ (rr & 15)) << 2);
                if (m >= rows_a || count <= 0) continue;
                int* to = p.partial + ((int64_t)blockIdx.y * H * M + m0 + m) * p.ld_partial + n;
                *reinterpret_cast<v4i*>(to) = *reinterpret_cast<const v4i*>(stage + at);
                if constexpr (H == 2) *reinterpret_cast<v4i*>(to + (int64_t)M * p.ld_partial) = *reinterpret_cast<const v4i*>(stage + PR * BNR + at);
            }
        } else if (whole) {
            turns(std::integral_constant<bool, true>());
        } else {
            turns(std::integral_constant<bool, false>());
        }
    }
}

template <int MODE, int BM, int BN, int WM, int WN, int RING>
hipError_t launch_tile(const FusedArgs& a, bool kmajor, hipStream_t s) {
    constexpr int BMR = MODE == FUSED_GRAD ? BM / 2 : BM, BNR = MODE == FUSED_PAIR ? BN / 2 : BN;
    constexpr int NT = (BM / WM) * (BN / WN) * 64;
    const int64_t tiles = (int64_t)((a.e.M + BMR - 1) / BMR) * ((a.e.N + BNR - 1) / BNR);
    if (tiles * NT >= (int64_t)1 << 32) return hipErrorInvalidValue;
    const int behind = MODE == FUSED_GRAD && a.dbias != nullptr ? (a.bias_n + 31) / 32 : 0;
    const dim3 grid((unsigned)(tiles + behind), a.partial != nullptr ? a.splits : 1);
    if (kmajor) hipLaunchKernelGGL((fused_tiled_kernel<MODE, BM, BN, WM, WN, true, RING>), grid, dim3(NT), 0, s, a);
    else hipLaunchKernelGGL((fused_tiled_kernel<MODE, BM, BN, WM, WN, false, RING>), grid, dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_form(const FusedArgs& a, FusedTile tile, bool kmajor, hipStream_t s) {
    switch (tile) {
        case FUSED_256x256: return launch_tile<MODE, 256, 256, 128, 64, 2>(a, kmajor, s);
        case FUSED_128x128: return launch_tile<MODE, 128, 128, 32, 64, 2>(a, kmajor, s);
        case FUSED_128x128_DEEP: return launch_tile<MODE, 128, 128, 64, 32, 4>(a, kmajor, s);
        case FUSED_64x128_DEEP: return launch_tile<MODE, 64, 128, 32, 32, 6>(a, kmajor, s);
        default: return launch_tile<MODE, 64, 128, 32, 32, 0>(a, kmajor, s);
    }
}

}  // namespace fused
}  // namespace qg
