// 256 x 256 tiles of the MX product: eight waves of 128 x 64.  MXFP4: stages of
// 256 values of K, two of them (144 KiB with the scales); MXFP8 activations: 128
// values, three (160 KiB).
// An fp32 output of MXFP8 activations splits every A fragment (mx_mfma.h): waves of 64 x
// 128 split half as many for the same products, 8192^3 769 -> 688 us.
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_256x256(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    if (!a8) return mx::launch_out<256, 256, 128, 64, 1, 8, 2, false>(a, s);
    if (a.out_type == QG_FP32) return mx::launch_one<256, 256, 64, 128, 1, 4, 3, true, float>(a, s);
    return mx::launch_half<256, 256, 128, 64, 1, 4, 3, true>(a, s);
}
}  // namespace qg
