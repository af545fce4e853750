// 64 x 128 tiles of the MX product: four waves of 32 x 64, stages of 256 values
// of K.  Five of them (MXFP4, 132 KiB) or four (MXFP8 activations, 140 KiB): one
// workgroup a CU has to keep its share of the memory's latency covered by itself.
// With two stages and twice the workgroups 512 x 4096 x 4096 took 25.3 us (and 15.2
// with one workgroup a CU) against 12.7.
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_64x128(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    if (a.splits > 1)
        return a8 ? mx::launch_out<64, 128, 32, 64, 8, 4, true, true>(a, s)
                  : mx::launch_out<64, 128, 32, 64, 8, 5, false, true>(a, s);
    return a8 ? mx::launch_out<64, 128, 32, 64, 8, 4, true, false>(a, s)
              : mx::launch_out<64, 128, 32, 64, 8, 5, false, false>(a, s);
}
}  // namespace qg
