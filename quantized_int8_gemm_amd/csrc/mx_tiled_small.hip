// The small tiles of the MX product, for outputs that would leave CUs idle under
// larger ones; wave tiles of 32 x 32, stages of 512 values of K.  At N = K = 8192
// (36 MB of weights, from memory) with MXFP4 / MXFP8 activations: 32 x 32 tiles, four
// waves, M = 1 10.9 / 13.2 us, M = 16 11.3 / 14.2 (weights in the Infinity Cache: M = 1
// 8.8 / 11.7, M = 16 9.3 / 12.4); 64 x 32, four waves a wave tile, M = 64 15.6 / 18.9; 64 x
// 64, two waves a wave tile, M = 128 17.2 / 25.5.  When each was chosen, stages of 256
// values were 4 to 10 % slower, two waves fewer 15 to 30 %.
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_32x32(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    return a8 ? mx::launch_out<32, 32, 32, 32, 4, 16, 5, true>(a, s) : mx::launch_out<32, 32, 32, 32, 4, 16, 7, false>(a, s);
}
hipError_t launch_mx_64x32(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    return a8 ? mx::launch_out<64, 32, 32, 32, 4, 16, 3, true>(a, s) : mx::launch_out<64, 32, 32, 32, 4, 16, 5, false>(a, s);
}
hipError_t launch_mx_64x64(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    return a8 ? mx::launch_out<64, 64, 32, 32, 2, 16, 3, true>(a, s) : mx::launch_out<64, 64, 32, 32, 2, 16, 4, false>(a, s);
}
}  // namespace qg
