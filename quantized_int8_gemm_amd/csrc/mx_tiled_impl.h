// Tiled MX product on the scaled matrix cores, fed by direct global-to-LDS
// loads; included by one translation unit per tile shape.
//
// A workgroup computes a BM x BN tile of the output, K in stages of NB blocks
// (32 NB values) held in a ring of STAGES LDS stages:
//  * Code rows of A and W go global -> LDS in 16-byte segments.  Each lane's
//    bytes land at consecutive LDS addresses, so the lane picks the global
//    segment whose swizzled home is that address.  Rows past M or N, and
//    segments past K, lie outside the buffer windows and read as zero.
//  * Scale bytes come in groups of 16 a row (1, 2 or 4 stages' worth) into places
//    beside the ring, a part of a later group with every stage.  Fetched a stage's 8
//    bytes at a time they asked L2 for as many cache lines as the codes did: 8192^3
//    MXFP4 292 us so, 276 in groups.
//  * The contraction may visit blocks in any order, so that a lane's scales lie
//    side by side: the two lane groups of a 32x32x64 instruction take blocks s
//    and NB/2 + s of the stage in step s.  One read per fragment row then brings
//    the scales of all a wave's steps, and the instruction picks the byte.
//  * While a step's products run, the next step's fragments are read, across the
//    stages' border too: the barrier stands before the stage's last step, when
//    every wave holds the last fragments of the old stage, so its ring place is
//    free for the chunk STAGES on, whose loads are spread over that step and the
//    next (all at once they hold the matrix instructions up).  Against reading
//    after the barrier: 8192^3 MXFP4 303 -> 292 us.  The products of one row block may
//    mix with the next one's reads: 8192^3 with MXFP8 activations, when they were
//    multiplied once, 410 -> 400 us.
//  * KW waves share a wave tile, each with its part of every stage's steps; their
//    sums are added through LDS, in order, so results repeat bit for bit.  Small
//    tiles need it: with one wave a SIMD every step waits for its fragments.
//  * The finished wave tile goes through LDS, 32 rows and 64 columns at a time, and
//    leaves in whole rows of those.
// Two figures side by side are of one run; from one run to another the same kernel
// differs by 2 %.
// What bounds 8192^3 MXFP4 (264 us, 4.2 PFLOP/s): the instruction alone on register
// operands runs at 7.1 PFLOP/s on random data, the clock falling from 2.4 to 1.7 GHz
// (9.7 PFLOP/s on zeros), and on this product's fragments at 5.9; the kernel keeps
// the matrix cores busy 55 % of the cycles at 1.77 GHz.  With MXFP8 activations, whose
// products take two instructions at 4.3 PFLOP/s, 8192^3 takes 668 us and 4096^3 87, the
// matrix cores busy 62 % of the cycles at 2.13 GHz.  Taken at 276 us, it ran 223 us
// without its loads, 265 without its fragment reads, 226 without its products and 172
// with its loads alone: no stream stands out, and each costs clock.  A stage takes
// 2918 cycles of which 2048 are products; the first chunk's latency is 6500 cycles a
// tile and the output 5400, but one workgroup a CU that walks its tiles and fetches
// the next one's first chunk under the output ran at the same 272 us (the clock falls
// as the stalls go).  Four waves of 128 x 128 (a third fewer fragment reads, one wave
// per SIMD) measured 284 against 276 us, wave priorities the same, two steps' worth
// of loads at once 287.
#pragma once
#include "mx_mfma.h"

namespace qg {
namespace mx {

constexpr int GROUP_M = 4;   // tile rows walked together (8: 8192^3 MXFP4 261.3 against 258.9 us)

// Slot of 16-byte segment s in a row of WIDTH bytes: the 16 rows that a
// fragment read touches at one segment take 16 distinct 16-byte places of a
// 256-byte span.
template <int WIDTH>
__device__ __forceinline__ int slot(int r, int s) {
    if constexpr (WIDTH == 64) return s ^ ((((r >> 1) ^ (r >> 3)) & 1) | ((r >> 1) & 2));
    else if constexpr (WIDTH == 128) return s ^ ((r >> 1) & 7);
    else return s ^ (r & 15);
}

template <bool A8>
__device__ __forceinline__ v16f mfma_step(int s, v8i w, uint32_t ws, v8i a, uint32_t as, v16f c) {
    switch (s) {   // the byte is an immediate; s is a constant of the unrolled loop
        case 0: return mfma_mx32<A8, 0, 0>(w, ws, a, as, c);
        case 1: return mfma_mx32<A8, 1, 1>(w, ws, a, as, c);
        case 2: return mfma_mx32<A8, 2, 2>(w, ws, a, as, c);
        default: return mfma_mx32<A8, 3, 3>(w, ws, a, as, c);
    }
}

constexpr uint32_t OUTSIDE = 0xffffff00u;   // past every window

// A wave-uniform value that the compiler takes as it is: address sums stay one
// vector addition next to their use instead of a register each across the loop.
__device__ __forceinline__ uint32_t scalar(uint32_t v) {
    v = __builtin_amdgcn_readfirstlane(v);
    asm volatile("" : "+s"(v));
    return v;
}

template <int BM, int BN, int WM, int WN, int KW, int NB, int STAGES, bool A8, typename T>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * KW * 64) void mx_tiled_kernel(MxMatmulArgs p) {
    constexpr int NT = (BM / WM) * (BN / WN) * KW * 64, NW = NT / 64 / KW, WAVES_N = BN / WN;
    constexpr int FM = WM / 32, FN = WN / 32, NS = NB / 2, SPW = NS / KW;   // steps of a stage, of a wave
    constexpr int AW = NB * (A8 ? 32 : 16), WW = NB * 16;         // bytes of a stage's code rows
    constexpr int A_BYTES = BM * AW, W_BYTES = BN * WW;
    constexpr int STAGE = A_BYTES + W_BYTES;
    constexpr int A_ROUNDS = A_BYTES / (NT * 16), W_ROUNDS = W_BYTES / (NT * 16), LOADS = A_ROUNDS + W_ROUNDS;
    // Scales: groups of 16 bytes a row, Q stages' worth, in places of their own.
    // With the loads of a chunk goes one Qth of a group: with those that start in
    // stage kt's last step the part of the group after that of stage kt + 1 + D.
    // D is what the wait at a stage's end leaves time for, so the last part of a
    // group has landed when its first stage begins.
    constexpr int Q = 16 / NB;
    constexpr int S_ROUNDS = ((BM + BN) * 4 + NT * Q - 1) / (NT * Q);   // per stage; rows past BM + BN are unused
    constexpr int D = STAGES > 3 ? STAGES - 3 : 0, PLACES = (D + Q - 1) / Q + 2;
    constexpr int GROUP = S_ROUNDS * Q * NT * 4, SCALES = STAGES * STAGE;
    // loads newer than the next chunk's and than the last part of its scale group
    constexpr int AFTER = STAGES == 2 ? 0 : LOADS + D * (LOADS + S_ROUNDS);
    constexpr int OB = sizeof(T), AV = A8 ? 2 : 1;
    static_assert(SPW == 2 || SPW == 4, "an even number of steps alternates the fragments' buffers");
    static_assert(WN == 32 || WN % 64 == 0, "output staging");
    static_assert(A_BYTES % (NT * 16) == 0 && W_BYTES % (NT * 16) == 0, "whole load rounds");
    static_assert(BM % 16 == 0, "a wave's scale words are of one operand");
    static_assert((LOADS + S_ROUNDS) * (STAGES - 1) < 64, "vmcnt range");
    constexpr int SW = WN < 64 ? WN : 64;   // columns staged at a time
    static_assert(STAGES * STAGE >= NW * 32 * SW * OB, "output staging fits the stage ring");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * STAGE + PLACES * GROUP];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = wave / NW, wm = wave % NW / WAVES_N, wn = wave % WAVES_N;
    const int g = lane >> 5, r32 = lane & 31;

    const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
    int tm, tn;
    tile_coords(xcd_remap(blockIdx.x, gridDim.x), tiles_m, tiles_n, GROUP_M, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int rows_a = p.M - m0 < BM ? p.M - m0 : BM, rows_w = p.N - n0 < BN ? p.N - n0 : BN;
    const int lda = (int)p.lda, ldw = (int)p.ldw, ldas = (int)p.ldas, ldws = (int)p.ldws;
    const int nblk = p.K / 32;
    constexpr int ABLK = A8 ? 32 : 16;
    const v4i a_rsrc = rsrc_words(p.A + (int64_t)m0 * p.lda, (uint32_t)((rows_a - 1) * lda + nblk * ABLK));
    const v4i w_rsrc = rsrc_words(p.W + (int64_t)n0 * p.ldw, (uint32_t)((rows_w - 1) * ldw + nblk * 16));
    // scale rows are readable to the end of their last 4-byte word
    const uint32_t s_span = (uint32_t)((nblk + 3) & ~3);
    const v4i as_rsrc = rsrc_words(p.as + (int64_t)m0 * p.ldas, (uint32_t)((rows_a - 1) * ldas) + s_span);
    const v4i ws_rsrc = rsrc_words(p.ws + (int64_t)n0 * p.ldws, (uint32_t)((rows_w - 1) * ldws) + s_span);
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    // Global offset (stage 0) and block of this lane's segment in a load round.
    // A round covers a multiple of 16 rows, so all rounds of an operand take the
    // same segment, a fixed number of rows apart (or of 8: odd rounds of A take
    // the segment with bit 3 flipped).
    constexpr int A_ROWS = NT * 16 / AW, W_ROWS = NT * 16 / WW;
    static_assert(A_ROWS % 8 == 0 && W_ROWS % 16 == 0, "one swizzle for all rounds, or two in turn");
    const int a_seg = slot<AW>(tid * 16 / AW, tid * 16 % AW / 16), w_seg = slot<WW>(tid * 16 / WW, tid * 16 % WW / 16);
    const uint32_t a_off = (uint32_t)(tid * 16 / AW * lda + 16 * a_seg), w_off = (uint32_t)(tid * 16 / WW * ldw + 16 * w_seg);
    const uint32_t a_odd = (uint32_t)(tid * 16 / AW * lda + 16 * (a_seg ^ 8));
    const int nk = (nblk + NB - 1) / NB;

    // Part `part` of PARTS of the loads of chunk kt.  Blocks past K, whole chunks
    // too, are read from outside the windows: every chunk issues the same loads,
    // so the loop has no branches and its waits are constants.
    constexpr int PARTS = 2 * FM;
    auto issue = [&](int kt, int stage, int part) __attribute__((always_inline)) {
        const uint32_t base = lds0 + (uint32_t)stage * STAGE, codes = base + wave * 1024;
        const uint32_t ka = scalar(kt * AW), kw = scalar(kt * WW);
        const int rest = nblk - kt * NB;   // blocks from this chunk on
#pragma unroll
        for (int i = part * LOADS / PARTS; i < (part + 1) * LOADS / PARTS; ++i) {
            if (i < A_ROUNDS) {
                const int flip = i * A_ROWS & 8, seg = a_seg ^ flip;
                dma16(a_rsrc, 16 * seg / ABLK >= rest ? OUTSIDE : (flip ? a_odd : a_off) + ((uint32_t)(i * A_ROWS * lda) + ka), codes + i * NT * 16);
            } else {
                const int q = i - A_ROUNDS;
                dma16(w_rsrc, w_seg >= rest ? OUTSIDE : w_off + ((uint32_t)(q * W_ROWS * ldw) + kw), codes + A_BYTES + q * NT * 16);
            }
        }
    };
    // Part t % Q of scale group t / Q + ahead, in 4-byte words, four lanes to a row.
    auto issue_scales = [&](int t, int ahead) __attribute__((always_inline)) {
        const int j = t / Q + ahead, q0 = t % Q * S_ROUNDS;
        const uint32_t base = lds0 + SCALES + (uint32_t)(j % PLACES) * GROUP + wave * 256;
        const uint32_t blk = (uint32_t)(j * 16 + tid % 4 * 4);
#pragma unroll
        for (int i = 0; i < S_ROUNDS; ++i) {
            const int q = q0 + i, first = q * (NT / 4) + wave * 16, r = first + lane / 4;
            const bool of_a = first < BM;
            const bool none = first >= BM + BN || (int)blk >= nblk;
            const uint32_t at = (uint32_t)(of_a ? r * ldas : (r - BM) * ldws) + blk;
            dma4(of_a ? as_rsrc : ws_rsrc, none ? OUTSIDE : at, base + q * NT * 4);
        }
    };

    v16f acc[FM][FN];
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

    float row_scale[FM];
#pragma unroll
    for (int a = 0; a < FM; ++a) {
        const int m = m0 + wm * WM + a * 32 + r32;
        row_scale[a] = p.act_scale != nullptr && m < p.M ? p.act_scale[m] : 1.0f;
    }

    auto read16 = [&](const uint8_t* at) {   // as a vector type, which is 16-byte aligned
        const v4i v = *reinterpret_cast<const v4i*>(at);
        return u32x4{(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
    };
    // Where in a stage this lane's fragment of step s and row block 0 lies, and
    // its scales; e2m1 fragments are held in four registers and widened at the
    // instruction.
    uint32_t a_at[SPW][AV], w_at[SPW], as_at = SCALES + (wm * WM + r32) * 16 + g * NS + kw * SPW;
    uint32_t ws_at = SCALES + (BM + wn * WN + r32) * 16 + g * NS + kw * SPW;
#pragma unroll
    for (int s = 0; s < SPW; ++s) {
        const int q = kw * SPW + s;   // this wave's steps are q of the stage
        const uint32_t row = (wm * WM + r32) * AW;
        if constexpr (A8) {
            a_at[s][0] = row + 16 * slot<AW>(r32, 2 * q + g);
            a_at[s][AV - 1] = row + 16 * slot<AW>(r32, 2 * (NS + q) + g);
        } else {
            a_at[s][0] = row + 16 * slot<AW>(r32, g * NS + q);
        }
        w_at[s] = A_BYTES + (wn * WN + r32) * WW + 16 * slot<WW>(r32, g * NS + q);
    }
#pragma unroll
    for (int s = 0; s < SPW; ++s) {
#pragma unroll
        for (int v = 0; v < AV; ++v) asm volatile("" : "+v"(a_at[s][v]));
        asm volatile("" : "+v"(w_at[s]));
    }
    asm volatile("" : "+v"(as_at), "+v"(ws_at));
    auto read_scale = [&](const uint8_t* at) -> uint32_t {
        if constexpr (SPW == 4) return *reinterpret_cast<const uint32_t*>(at);
        else return *reinterpret_cast<const uint16_t*>(at);
    };

    // Fragments of the current step and the next; scales of the chunk, and of
    // the next one as read.
    u32x4 af[2][FM][AV], wf[2][FN];
    uint32_t as[FM], ws[FN], as_read[FM], ws_read[FN];
    auto read_scales = [&](int kt) {
        const uint8_t* S = smem + scalar((uint32_t)(kt / Q % PLACES) * GROUP + (uint32_t)(kt % Q) * NB);
#pragma unroll
        for (int b = 0; b < FN; ++b) ws_read[b] = read_scale(S + ws_at + b * 512);
#pragma unroll
        for (int a = 0; a < FM; ++a) as_read[a] = read_scale(S + as_at + a * 512);
    };
    auto read_w = [&](const uint8_t* S, int s, int buf) {
#pragma unroll
        for (int b = 0; b < FN; ++b) wf[buf][b] = read16(S + w_at[s] + b * 32 * WW);
    };
    auto read_a = [&](const uint8_t* S, int a, int s, int buf) {
#pragma unroll
        for (int v = 0; v < AV; ++v) af[buf][a][v] = read16(S + a_at[s][v] + a * 32 * AW);
    };
    // Step s of this wave's in chunk kt, which lies in ring place `stage`: the
    // products of the fragments at hand, in buffers cur, while those of the next
    // step (at the stage's end, of the next chunk) are read.
    auto step = [&](int kt, int stage, int s, int cur) __attribute__((always_inline)) {
        const bool last = s == SPW - 1;
        const int ns = last ? 0 : s + 1, nxt = cur ^ 1, after = stage + 1 == STAGES ? 0 : stage + 1;
        const uint8_t* S = smem + scalar((uint32_t)(last ? after : stage) * STAGE);
        if (s == 0) {
            // scale bytes past K may be anything: 0 (2^-127) times the zero codes there
            const int rest = nblk - kt * NB - g * NS - kw * SPW;
            const uint32_t mask = rest >= 4 ? ~0u : (rest <= 0 ? 0u : (1u << (8 * rest)) - 1u);
#pragma unroll
            for (int b = 0; b < FN; ++b) ws[b] = ws_read[b] & mask;
#pragma unroll
            for (int a = 0; a < FM; ++a) as[a] = as_read[a] & mask;
        }
#pragma unroll
        for (int a = 0; a < FM; ++a) {
            // W's fragments: first where A's are twice their size, else along with A's
            // (8192^3 MXFP4 261.5 against 259.7 us, MXFP8 669 against 674)
            if constexpr (A8) {
                if (a == 0) read_w(S, ns, nxt);
            } else {
#pragma unroll
                for (int b = a * FN / FM; b < (a + 1) * FN / FM; ++b) wf[nxt][b] = read16(S + w_at[ns] + b * 32 * WW);
            }
            read_a(S, a, ns, nxt);
            if (last && a == 0) {
                read_scales(kt + 1);
                issue_scales(kt + 1 + D, 1);
            }
            if (last) issue(kt + STAGES, stage, a);
            if (s == 0) issue(kt + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1, FM + a);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = 0; b < FN; ++b)
                acc[a][b] = mfma_step<A8>(s, words4(wf[cur][b]), ws[b], A8 ? words8(af[cur][a][0], af[cur][a][AV - 1]) : words4(af[cur][a][0]),
                                                 as[a], acc[a][b]);
        }
    };
#pragma unroll
    for (int t = 0; t < Q; ++t) issue_scales(t, 0);
#pragma unroll
    for (int c = 0; c < STAGES; ++c) {
        if (c >= STAGES - 1 - D) issue_scales(c - (STAGES - 1 - D), 1);
#pragma unroll
        for (int part = 0; part < (c < STAGES - 1 ? PARTS : FM); ++part) issue(c, c, part);
    }
    // chunk 0 and its scales have landed once at most the loads after them are outstanding
    wait_vmcnt<S_ROUNDS * (D + 1) + LOADS * (STAGES - 2) + FM * LOADS / PARTS>();
    __syncthreads();
    read_w(smem, 0, 0);
#pragma unroll
    for (int a = 0; a < FM; ++a) read_a(smem, a, 0, 0);
    read_scales(0);
    int stage = 0;
    auto chunk = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < SPW - 1; ++s) step(kt, stage, s, s & 1);
        // the next chunk and its scales are there, and every wave has read this
        // chunk's last fragments
        wait_vmcnt<AFTER>();
        __syncthreads();
        step(kt, stage, SPW - 1, 1);
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    };
    for (int kt = 0; kt < nk; ++kt) chunk(kt);
    wait_vmcnt<0>();   // loads past K write zeros
    __syncthreads();   // every wave is done with the stage ring

    const bool mine = KW == 1 || kw == 0;   // the waves that leave the results
    if constexpr (KW > 1) {
        // the other waves' sums over their steps join in order
        constexpr int WAVE = FM * FN * 4096;
        static_assert((KW - 1) * NW * WAVE <= STAGES * STAGE + PLACES * GROUP, "sums fit the ring");
        auto at = [&](int k, int a, int b, int q) {
            return reinterpret_cast<v4f*>(smem + ((k - 1) * NW + wave % NW) * WAVE + ((a * FN + b) * 4 + q) * 1024 + 16 * lane);
        };
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (!mine) *at(kw, a, b, q) = v4f{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
        __syncthreads();
        if (mine) {
#pragma unroll
            for (int k = 1; k < KW; ++k)
#pragma unroll
                for (int a = 0; a < FM; ++a)
#pragma unroll
                    for (int b = 0; b < FN; ++b)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const v4f v = *at(k, a, b, q);
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[a][b][4 * q + i] += v[i];
                        }
        }
        __syncthreads();
    }

    // 32 rows and SW columns of the wave's tile at a time through the wave's own piece of LDS:
    // register 4 q + i of a lane is row r32, column 8 q + 4 g + i.  Chunk c (16
    // bytes) of a staged row lies at c ^ swizzle, so neither side collides.
    constexpr int PITCH = SW * OB, CPR = PITCH / 16, PER = 16 / OB, RPI = 64 / CPR;   // rows per store instruction
    if (!mine) return;
    uint8_t* own = smem + wave * 32 * PITCH;
    T* out = reinterpret_cast<T*>(p.out);
    auto swiz = [](int row, int c) { return CPR == 16 ? c ^ (row & 15) : CPR == 8 ? c ^ ((row >> 1) & 7) : c ^ ((row >> 2) & 3); };
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int h = 0; h < FN; h += SW / 32) {
#pragma unroll
            for (int b = 0; b < SW / 32; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    T t[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[i] = (T)(acc[a][h + b][4 * q + i] * row_scale[a]);
                    const int byte = (b * 32 + 8 * q + 4 * g) * OB;
                    __builtin_memcpy(__builtin_assume_aligned(own + r32 * PITCH + 16 * swiz(r32, byte / 16) + byte % 16, 4 * OB), t, 4 * OB);
                }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int k = 0; k < 32 / RPI; ++k) {
                const int row = k * RPI + lane / CPR, c = lane % CPR;
                const u32x4 v = read16(own + row * PITCH + 16 * swiz(row, c));
                const int m = m0 + wm * WM + a * 32 + row, n = n0 + wn * WN + h * 32 + c * PER;
                if (m < p.M && n < p.N) {
                    T* dst = out + (int64_t)m * p.ldo + n;
                    if (n + PER <= p.N) {   // at any alignment
                        *reinterpret_cast<v4i_any*>(dst) = v4i_any{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
                    } else {
                        T e[PER];
                        __builtin_memcpy(e, &v, 16);
#pragma unroll
                        for (int i = 0; i < PER; ++i)
                            if (n + i < p.N) dst[i] = e[i];
                    }
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
}

template <int BM, int BN, int WM, int WN, int KW, int NB, int STAGES, bool A8, typename T>
hipError_t launch_one(const MxMatmulArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN)));
    hipLaunchKernelGGL((mx_tiled_kernel<BM, BN, WM, WN, KW, NB, STAGES, A8, T>), grid, dim3((BM / WM) * (BN / WN) * KW * 64), 0, s, a);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int KW, int NB, int STAGES, bool A8>
hipError_t launch_out(const MxMatmulArgs& a, hipStream_t s) {
    if (a.out_type == QG_FP32) return launch_one<BM, BN, WM, WN, KW, NB, STAGES, A8, float>(a, s);
    if (a.out_type == QG_BF16) return launch_one<BM, BN, WM, WN, KW, NB, STAGES, A8, __bf16>(a, s);
    return launch_one<BM, BN, WM, WN, KW, NB, STAGES, A8, _Float16>(a, s);
}

}  // namespace mx
}  // namespace qg
