// 128 x 128 tiles of the MX product: four waves of 64 x 64.
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_128x128(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    if (a.splits > 1)
        return a8 ? mx::launch_out<128, 128, 64, 64, 8, 3, true, true>(a, s)
                  : mx::launch_out<128, 128, 64, 64, 8, 4, false, true>(a, s);
    if (mx::one_round<128, 128>(a))
        return a8 ? mx::launch_out<128, 128, 64, 64, 8, 3, true, false>(a, s)
                  : mx::launch_out<128, 128, 64, 64, 8, 4, false, false>(a, s);
    return a8 ? mx::launch_out<128, 128, 64, 64, 4, 3, true, false>(a, s)
              : mx::launch_out<128, 128, 64, 64, 8, 2, false, false>(a, s);
}
}  // namespace qg
