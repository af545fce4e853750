// 64 x 128 tiles of the MX product: wave tiles of 32 x 64, two waves each, stages of
// 256 values of K, five of them (MXFP4, 126 KiB) or four (MXFP8 activations, 134
// KiB): a CU has one such workgroup, which has to cover the memory's latency by
// itself.  512 x 4096 x 4096 MXFP4 13.1 us, with two stages and one wave a wave tile
// 15.2; 300 x 5001 x 4096 fp32 22.2 us, one wave a wave tile 23.8 (19.8 since rows that
// start at any byte are written in 16-byte pieces too).
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_64x128(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    return a8 ? mx::launch_out<64, 128, 32, 64, 2, 8, 4, true>(a, s) : mx::launch_out<64, 128, 32, 64, 2, 8, 5, false>(a, s);
}
}  // namespace qg
