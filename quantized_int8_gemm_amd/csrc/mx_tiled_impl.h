// Tiled MX product on the scaled matrix cores, fed by direct global-to-LDS
// loads; included by one translation unit per tile shape.
//
// A workgroup computes a BM x BN tile of the output, K in stages of NB blocks
// (32 NB values) held in a ring of STAGES LDS stages:
//  * Code rows of A and W go global -> LDS in 16-byte segments, scale bytes in
//    4-byte words, STAGES - 1 stages ahead of the one being multiplied.  Each
//    lane's bytes land at consecutive LDS addresses, so the lane picks the
//    global segment whose swizzled home is that address.  Rows past M or N, and
//    segments past K, lie outside the buffer windows and read as zero.
//  * The contraction may visit blocks in any order, so that a lane's scales lie
//    side by side: the two lane groups of a 32x32x64 instruction take blocks s
//    and NB/2 + s of the stage in step s.  One NB/2-byte read per fragment row
//    then brings the scales of the whole stage, and the instruction picks the
//    byte.
//  * The finished wave tile goes through LDS, 32 rows at a time, and leaves in
//    whole rows of 64 columns.
// SK: blockIdx.y divides K into ranges of split_k values; each range leaves its
// fp32 tile in the workspace and the one that takes the tile's last ticket adds
// them all in order (so results repeat bit for bit) and writes the output.
#pragma once
#include "mx_mfma.h"
#include "kernels.h"

namespace qg {
namespace mx {

constexpr int GROUP_M = 8;

__device__ __forceinline__ v4i rsrc_words(const void* base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    v4i r;
    r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu));
    r.z = __builtin_amdgcn_readfirstlane((int)bytes);
    r.w = 0x00020000;
    return r;
}

// 16 (4) bytes per lane from buffer offset `voff` into LDS at lds_base + 16
// (4) * lane.  Inline assembly, so that the compiler does not wait for these
// loads before every LDS read; the kernel waits for them explicitly.  M0 (the
// LDS destination) is set inside the block and declared clobbered; nothing else
// in these kernels uses it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(v4i rsrc, uint32_t voff, uint32_t lds_base) {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_base);
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :: "v"(voff), "s"(rsrc), "s"(m0) : "memory", "m0");
}
__device__ __forceinline__ void dma4(v4i rsrc, uint32_t voff, uint32_t lds_base) {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_base);
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :: "v"(voff), "s"(rsrc), "s"(m0) : "memory", "m0");
}
#pragma clang diagnostic pop

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Slot of 16-byte segment s in a row of WIDTH bytes: the 16 rows that a
// fragment read touches at one segment take 16 distinct 16-byte places of a
// 256-byte span.
template <int WIDTH>
__device__ __forceinline__ int slot(int r, int s) {
    if constexpr (WIDTH == 64) return s ^ ((((r >> 1) ^ (r >> 3)) & 1) | ((r >> 1) & 2));
    else if constexpr (WIDTH == 128) return s ^ ((r >> 1) & 7);
    else return s ^ (r & 15);
}

template <bool A8, bool EXACT>
__device__ __forceinline__ v16f mfma_step(int s, v8i w, uint32_t ws, v8i a, uint32_t as, v16f c) {
    switch (s) {   // the byte is an immediate; s is a constant of the unrolled loop
        case 0: return mfma_mx32<A8, EXACT, 0, 0>(w, ws, a, as, c);
        case 1: return mfma_mx32<A8, EXACT, 1, 1>(w, ws, a, as, c);
        case 2: return mfma_mx32<A8, EXACT, 2, 2>(w, ws, a, as, c);
        default: return mfma_mx32<A8, EXACT, 3, 3>(w, ws, a, as, c);
    }
}

constexpr uint32_t OUTSIDE = 0xffffff00u;   // past every window

template <int BM, int BN, int WM, int WN, int NB, int STAGES, bool A8, typename T, bool SK>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void mx_tiled_kernel(MxMatmulArgs p) {
    constexpr bool EXACT = A8 && sizeof(T) == 4;
    constexpr int NT = (BM / WM) * (BN / WN) * 64, NW = NT / 64, WAVES_N = BN / WN;
    constexpr int FM = WM / 32, FN = WN / 32, NS = NB / 2;
    constexpr int AW = NB * (A8 ? 32 : 16), WW = NB * 16;         // bytes of a stage's code rows
    constexpr int A_BYTES = BM * AW, W_BYTES = BN * WW;
    constexpr int S_BYTES = ((BM + BN) * NB + NT * 4 - 1) / (NT * 4) * (NT * 4);   // whole load rounds, the excess unused
    constexpr int STAGE = A_BYTES + W_BYTES + S_BYTES;
    constexpr int A_ROUNDS = A_BYTES / (NT * 16), W_ROUNDS = W_BYTES / (NT * 16), S_ROUNDS = S_BYTES / (NT * 4);
    constexpr int LOADS = A_ROUNDS + W_ROUNDS + S_ROUNDS;
    constexpr int OB = sizeof(T);
    static_assert(WN == 64, "output staging");
    static_assert(A_BYTES % (NT * 16) == 0 && W_BYTES % (NT * 16) == 0, "whole load rounds");
    static_assert((BM * NB) % 256 == 0, "a wave's scale words are of one operand");
    static_assert(LOADS * (STAGES - 2) < 64, "vmcnt range");
    static_assert(STAGES * STAGE >= NW * 32 * WN * OB, "output staging fits the stage ring");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * STAGE];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int g = lane >> 5, r32 = lane & 31;

    const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
    int tm, tn;
    tile_coords(xcd_remap(blockIdx.x, gridDim.x), tiles_m, tiles_n, GROUP_M, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int rows_a = p.M - m0 < BM ? p.M - m0 : BM, rows_w = p.N - n0 < BN ? p.N - n0 : BN;
    const int lda = (int)p.lda, ldw = (int)p.ldw, ldas = (int)p.ldas, ldws = (int)p.ldws;
    // this workgroup's blocks of K: kb0 .. kb0 + nblk
    const int kb0 = SK ? (int)blockIdx.y * (p.split_k / 32) : 0;
    const int left = p.K / 32 - kb0;
    const int nblk = SK && left > p.split_k / 32 ? p.split_k / 32 : left;
    constexpr int ABLK = A8 ? 32 : 16;
    const v4i a_rsrc = rsrc_words(p.A + (int64_t)m0 * p.lda + kb0 * ABLK, (uint32_t)((rows_a - 1) * lda + nblk * ABLK));
    const v4i w_rsrc = rsrc_words(p.W + (int64_t)n0 * p.ldw + kb0 * 16, (uint32_t)((rows_w - 1) * ldw + nblk * 16));
    // scale rows are readable to the end of their last 4-byte word
    const uint32_t s_span = (uint32_t)((nblk + 3) & ~3);
    const v4i as_rsrc = rsrc_words(p.as + (int64_t)m0 * p.ldas + kb0, (uint32_t)((rows_a - 1) * ldas) + s_span);
    const v4i ws_rsrc = rsrc_words(p.ws + (int64_t)n0 * p.ldws + kb0, (uint32_t)((rows_w - 1) * ldws) + s_span);
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    // Global offset (stage 0) and block of each load round's segment.
    uint32_t a_off[A_ROUNDS], w_off[W_ROUNDS], s_off[S_ROUNDS];
    int a_blk[A_ROUNDS], w_blk[W_ROUNDS], s_blk[S_ROUNDS];
#pragma unroll
    for (int q = 0; q < A_ROUNDS; ++q) {
        const int o = (q * NT + tid) * 16, r = o / AW, s = slot<AW>(r, (o % AW) / 16);
        a_off[q] = (uint32_t)(r * lda + 16 * s);
        a_blk[q] = 16 * s / ABLK;
    }
#pragma unroll
    for (int q = 0; q < W_ROUNDS; ++q) {
        const int o = (q * NT + tid) * 16, r = o / WW, s = slot<WW>(r, (o % WW) / 16);
        w_off[q] = (uint32_t)(r * ldw + 16 * s);
        w_blk[q] = s;
    }
#pragma unroll
    for (int q = 0; q < S_ROUNDS; ++q) {
        const int o = (q * NT + tid) * 4, r = o / NB;
        s_blk[q] = o % NB;
        s_off[q] = (uint32_t)((r < BM ? r * ldas : (r - BM) * ldws) + s_blk[q]);
    }
    const int nk = (nblk + NB - 1) / NB;
    const bool ragged = nblk % NB != 0;

    auto issue = [&](int kt, int stage) {
        const uint32_t base = lds0 + stage * STAGE, codes = base + wave * 1024;
        const bool tail = ragged && kt == nk - 1;
        const int rest = nblk - kt * NB;
#pragma unroll
        for (int q = 0; q < A_ROUNDS; ++q)
            dma16(a_rsrc, tail && a_blk[q] >= rest ? OUTSIDE : a_off[q] + (uint32_t)(kt * AW), codes + q * NT * 16);
#pragma unroll
        for (int q = 0; q < W_ROUNDS; ++q)
            dma16(w_rsrc, tail && w_blk[q] >= rest ? OUTSIDE : w_off[q] + (uint32_t)(kt * WW), codes + A_BYTES + q * NT * 16);
#pragma unroll
        for (int q = 0; q < S_ROUNDS; ++q) {
            const bool of_a = __builtin_amdgcn_readfirstlane((q * NT + wave * 64) * 4 < BM * NB ? 1 : 0);
            const bool none = ((q * NT + tid) * 4 >= (BM + BN) * NB) || (tail && s_blk[q] >= rest);
            dma4(of_a ? as_rsrc : ws_rsrc, none ? OUTSIDE : s_off[q] + (uint32_t)(kt * NB),
                 base + A_BYTES + W_BYTES + wave * 256 + q * NT * 4);
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

    auto read16 = [&](const uint8_t* at) { return *reinterpret_cast<const u32x4*>(at); };
    auto read_a = [&](const uint8_t* S, int a, int s) -> v8i {
        const uint8_t* row = S + (wm * WM + a * 32 + r32) * AW;
        if constexpr (A8)
            return words8(read16(row + 16 * slot<AW>(r32, 2 * s + g)), read16(row + 16 * slot<AW>(r32, 2 * (NS + s) + g)));
        else
            return words4(read16(row + 16 * slot<AW>(r32, g * NS + s)));
    };
    auto read_w = [&](const uint8_t* S, int b, int s) -> v8i {
        return words4(read16(S + A_BYTES + (wn * WN + b * 32 + r32) * WW + 16 * slot<WW>(r32, g * NS + s)));
    };
    auto read_scale = [&](const uint8_t* S, int row) -> uint32_t {
        const uint8_t* at = S + A_BYTES + W_BYTES + row * NB + g * NS;
        if constexpr (NS == 4) return *reinterpret_cast<const uint32_t*>(at);
        else return *reinterpret_cast<const uint16_t*>(at);
    };

    auto compute = [&](int stage, int next_kt, int kt) {
        const uint8_t* S = smem + stage * STAGE;
        uint32_t as[FM], ws[FN];
#pragma unroll
        for (int b = 0; b < FN; ++b) ws[b] = read_scale(S, BM + wn * WN + b * 32 + r32);
#pragma unroll
        for (int a = 0; a < FM; ++a) as[a] = read_scale(S, wm * WM + a * 32 + r32);
        v8i wf[NS][FN];
#pragma unroll
        for (int b = 0; b < FN; ++b) wf[0][b] = read_w(S, b, 0);
        v8i a_next = read_a(S, 0, 0);
#pragma unroll
        for (int s = 1; s < NS; ++s)
#pragma unroll
            for (int b = 0; b < FN; ++b) wf[s][b] = read_w(S, b, s);
        __builtin_amdgcn_sched_barrier(0);
        if (next_kt >= 0) issue(next_kt, next_kt % STAGES);
        __builtin_amdgcn_sched_barrier(0);
        if (ragged && kt == nk - 1) {
            // scale bytes past K may be anything: 0 (2^-127) times the zero codes there
            const int rest = nblk - kt * NB - g * NS;
            const uint32_t mask = rest >= 4 ? ~0u : (rest <= 0 ? 0u : (1u << (8 * rest)) - 1u);
#pragma unroll
            for (int b = 0; b < FN; ++b) ws[b] &= mask;
#pragma unroll
            for (int a = 0; a < FM; ++a) as[a] &= mask;
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
            for (int a = 0; a < FM; ++a) {
                const v8i af = a_next;
                if (a + 1 < FM) a_next = read_a(S, a + 1, s);
                else if (s + 1 < NS) a_next = read_a(S, 0, s + 1);
                __builtin_amdgcn_sched_barrier(0);   // the next read goes ahead of these products
#pragma unroll
                for (int b = 0; b < FN; ++b) acc[a][b] = mfma_step<A8, EXACT>(s, wf[s][b], ws[b], af, as[a], acc[a][b]);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < nk) issue(s, s);
    for (int kt = 0; kt < nk; ++kt) {
        if (kt + STAGES - 2 < nk) wait_vmcnt<LOADS * (STAGES - 2)>();
        else wait_vmcnt<0>();
        __syncthreads();
        compute(kt % STAGES, kt + STAGES - 1 < nk ? kt + STAGES - 1 : -1, kt);
    }
    __syncthreads();   // every wave is done with the stage ring

    if constexpr (SK) {
        const int S = (int)gridDim.y, sk = (int)blockIdx.y;
        if (S > 1) {
            constexpr int COHERENT = 16;   // sc1: device scope
            constexpr int TILE_BYTES = BM * BN * 4;
            const int tile = tm * tiles_n + tn;   // < SKINNY_MAX_TICKETS (host plan)
            int* tickets = reinterpret_cast<int*>(p.workspace);
            char* part = reinterpret_cast<char*>(p.workspace) + SKINNY_TICKET_BYTES + (size_t)tile * S * TILE_BYTES;
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(part, (uint32_t)(S * TILE_BYTES));
            auto at = [&](int s2, int a, int b, int q) {
                return (int)(s2 * TILE_BYTES + (((wave * FM + a) * FN + b) * 4 + q) * 1024 + 16 * lane);
            };
#pragma unroll
            for (int a = 0; a < FM; ++a)
#pragma unroll
                for (int b = 0; b < FN; ++b)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const v4f v = {acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v), rs, at(sk, a, b, q), 0, COHERENT);
                    }
            __builtin_amdgcn_s_waitcnt(0);
            __shared__ int ticket;
            __syncthreads();
            if (tid == 0) ticket = __hip_atomic_fetch_add(&tickets[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (ticket != S - 1) return;
            // every range's tile, the own one too, in order
#pragma unroll
            for (int a = 0; a < FM; ++a)
#pragma unroll
                for (int b = 0; b < FN; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
            for (int s2 = 0; s2 < S; ++s2) {
                v4f v[FM][FN][4];
#pragma unroll
                for (int a = 0; a < FM; ++a)
#pragma unroll
                    for (int b = 0; b < FN; ++b)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            v[a][b][q] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, at(s2, a, b, q), 0, COHERENT));
#pragma unroll
                for (int a = 0; a < FM; ++a)
#pragma unroll
                    for (int b = 0; b < FN; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[a][b][i] += v[a][b][i / 4][i % 4];
            }
            if (tid == 0) __hip_atomic_store(&tickets[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }

    // 32 rows of the wave's tile at a time through the wave's own piece of LDS:
    // register 4 q + i of a lane is row r32, column 8 q + 4 g + i.  Chunk c (16
    // bytes) of a staged row lies at c ^ swizzle, so neither side collides.
    constexpr int PITCH = WN * OB, CPR = PITCH / 16, PER = 16 / OB, RPI = 64 / CPR;   // rows per store instruction
    uint8_t* stage = smem + wave * 32 * PITCH;
    T* out = reinterpret_cast<T*>(p.out);
    const bool vec = (p.ldo * OB) % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    auto swiz = [](int row, int c) { return OB == 2 ? c ^ ((row >> 1) & 7) : c ^ (row & 15); };
#pragma unroll
    for (int a = 0; a < FM; ++a) {
#pragma unroll
        for (int b = 0; b < FN; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                T t[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = (T)(acc[a][b][4 * q + i] * row_scale[a]);
                const int byte = (b * 32 + 8 * q + 4 * g) * OB;
                __builtin_memcpy(__builtin_assume_aligned(stage + r32 * PITCH + 16 * swiz(r32, byte / 16) + byte % 16, 4 * OB), t, 4 * OB);
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 32 / RPI; ++k) {
            const int row = k * RPI + lane / CPR, c = lane % CPR;
            const u32x4 v = read16(stage + row * PITCH + 16 * swiz(row, c));
            const int m = m0 + wm * WM + a * 32 + row, n = n0 + wn * WN + c * PER;
            if (m < p.M && n < p.N) {
                T* dst = out + (int64_t)m * p.ldo + n;
                if (vec && n + PER <= p.N) {
                    *reinterpret_cast<u32x4*>(dst) = v;
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

template <int BM, int BN, int WM, int WN, int NB, int STAGES, bool A8, bool SK>
hipError_t launch_out(const MxMatmulArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN)), SK ? (unsigned)a.splits : 1);
    const dim3 block((BM / WM) * (BN / WN) * 64);
    if (a.out_type == QG_FP32)
        hipLaunchKernelGGL((mx_tiled_kernel<BM, BN, WM, WN, NB, STAGES, A8, float, SK>), grid, block, 0, s, a);
    else if (a.out_type == QG_BF16)
        hipLaunchKernelGGL((mx_tiled_kernel<BM, BN, WM, WN, NB, STAGES, A8, __bf16, SK>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((mx_tiled_kernel<BM, BN, WM, WN, NB, STAGES, A8, _Float16, SK>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace mx
}  // namespace qg
