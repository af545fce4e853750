// 64 x 128 tiles of the MX product: four waves of 32 x 64, stages of 256 values
// of K, two of them (MXFP4 56 KiB, MXFP8 activations 72 KiB).
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_64x128(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    if (a.splits > 1)
        return a8 ? mx::launch_out<64, 128, 32, 64, 8, 2, true, true>(a, s)
                  : mx::launch_out<64, 128, 32, 64, 8, 2, false, true>(a, s);
    return a8 ? mx::launch_out<64, 128, 32, 64, 8, 2, true, false>(a, s)
              : mx::launch_out<64, 128, 32, 64, 8, 2, false, false>(a, s);
}
}  // namespace qg
