// What the fused kernels that stage operands in LDS share.
#pragma once
#include "fused_common.h"
#include "int8_dma_impl.h"

namespace qg {
namespace fused {

constexpr uint32_t NOWHERE = 0x80000000u;   // past every buffer's end

// Slot of segment s of k-row r of a [K,N] tile whose rows are RB bytes.  A transposed read
// touches 16 rows, 8 of two groups 16 rows apart.  For RB = 64 they lie four to 256 bytes, and
// bits 2 and 4 of r tell those that would share a slot apart; for 32 eight to 256, and bit 4 does.
template <int RB>
__device__ __forceinline__ int kn_slot_of(int r, int s) {
    if constexpr (RB == 32) return s ^ ((r >> 4) & 1);
    else if constexpr (RB == 64) return s ^ (((r >> 2) & 1) | ((r >> 3) & 2));
    else return dma::kn_slot<RB>(r, s);
}

// dbias[n] = sum of the partial rows, for 32 columns a workgroup: NT / 32 lanes a column, joined
// in a fixed order.  Behind the tiles in one launch: on their own they took 3 us more.
template <int NT>
__device__ __forceinline__ void sum_bias(const FusedArgs& p, int block, float* red) {
    constexpr int ROWS = NT / 32;
    const int cl = threadIdx.x & 31, q = threadIdx.x >> 5, c = block * 32 + cl;
    float s = 0.f;
    if (c < p.bias_n) {
#pragma unroll 8
        for (int i = q; i < p.parts; i += ROWS) s += p.part[(int64_t)i * p.bias_n + c];
    }
    red[q * 33 + cl] = s;
    __syncthreads();
    if (q == 0 && c < p.bias_n) {
#pragma unroll
        for (int i = 1; i < ROWS; ++i) s += red[i * 33 + cl];
        p.dbias[c] = s;
    }
}

}  // namespace fused
}  // namespace qg
