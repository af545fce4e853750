// 128 x 128 tiles of the MX product, wave tiles of 64 x 64 (MXFP4) or 32 x 128 (MXFP8
// activations, whose fragments are split: half as many as in 64 x 64 ones, 2048 x 2048 x
// 4096 with fp32 output 33.3 -> 29.3 us).  Where every CU has at most one of them, eight
// waves (two to a wave tile) and a deep ring: four stages of 256 values of K (MXFP4, 140
// KiB) or three (MXFP8 activations, 152 KiB): 2048 x 2048 x 4096 MXFP4 17.4 us, with two
// stages and four waves 24.4.  For more, four waves and two stages of 256 values (72 KiB,
// two workgroups a CU) or three of 128 (MXFP8 activations, 80 KiB).
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_128x128(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    const bool one_round = (int64_t)((a.M + 127) / 128) * ((a.N + 127) / 128) <= MX_ROUND;
    if (!a8)
        return one_round ? mx::launch_out<128, 128, 64, 64, 2, 8, 4, false>(a, s)
                         : mx::launch_out<128, 128, 64, 64, 1, 8, 2, false>(a, s);
    return one_round ? mx::launch_out<128, 128, 32, 128, 2, 8, 3, true>(a, s)
                     : mx::launch_out<128, 128, 32, 128, 1, 4, 3, true>(a, s);
}
}  // namespace qg
