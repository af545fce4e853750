// 128 x 128 tiles of the MX product: four waves of 64 x 64.  MXFP4: stages of
// 256 values of K, two of them (72 KiB, two workgroups per CU); MXFP8
// activations: 128 values, three (80 KiB).
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_128x128(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    if (a.splits > 1)
        return a8 ? mx::launch_out<128, 128, 64, 64, 4, 3, true, true>(a, s)
                  : mx::launch_out<128, 128, 64, 64, 8, 2, false, true>(a, s);
    return a8 ? mx::launch_out<128, 128, 64, 64, 4, 3, true, false>(a, s)
              : mx::launch_out<128, 128, 64, 64, 8, 2, false, false>(a, s);
}
}  // namespace qg
