// Loads of 16 bytes at any alignment.
#pragma once
#include "mx_common.h"

namespace qg {

// 16 bytes from column c of a row of `limit` on, zeros past its end (limit 0: no load).
// Where they would pass the end, the row's last 16 are read and moved down.
__device__ __forceinline__ u32x4 load16_any(const int8_t* row, int c, int limit) {
    const int past = c + 16 - limit;
    if (past >= 16) return u32x4{0u, 0u, 0u, 0u};
    if (limit >= 16) {
        const v4i_any v = *reinterpret_cast<const v4i_any*>(row + (past > 0 ? limit - 16 : c));
        uint32_t w[5] = {(uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3], 0u};
        if (past > 0) {
#pragma unroll
            for (int d = 2; d >= 1; d /= 2)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = past & 4 * d ? (i + d < 4 ? w[i + d] : 0u) : w[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], (uint32_t)past & 3u);
        }
        return u32x4{w[0], w[1], w[2], w[3]};
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (int i = 0; c + i < limit; ++i) {
        const uint32_t b = (uint32_t)(uint8_t)row[c + i] << (8 * (i & 3));
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] |= i / 4 == q ? b : 0u;
    }
    return u32x4{w[0], w[1], w[2], w[3]};
}

}  // namespace qg
