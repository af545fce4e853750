// 64 x 128 tiles of the MX product: wave tiles of 32 x 64, two waves each, stages of
// 256 values of K, five of them (MXFP4, 132 KiB) or four (MXFP8 activations, 140
// KiB): a CU has one such workgroup, which has to cover the memory's latency by
// itself.  512 x 4096 x 4096 12.6 us MXFP4, 19 to 20 MXFP8; 300 x 5001 x 4096 MXFP8
// with fp32 output 17.4 a call.  The second wave of a wave tile and the deeper ring
// brought the first from 15.2 to 13.1, the last, before other steps, from 23.8 to 22.2.
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_64x128(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    return a8 ? mx::launch_out<64, 128, 32, 64, 2, 8, 4, true>(a, s) : mx::launch_out<64, 128, 32, 64, 2, 8, 5, false>(a, s);
}
}  // namespace qg
