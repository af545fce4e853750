// 256 x 256 tiles of the MX product: eight waves.  MXFP4: wave tiles of 128 x 64,
// stages of 256 values of K, two of them (144 KiB with the scales); MXFP8 activations:
// 128 values, three (160 KiB), and wave tiles of 64 x 128, since every A fragment is
// split (mx_mfma.h) and these split half as many for the same products, 8192^3 with
// fp32 output 769 -> 688 us (bf16 668).
#include "mx_tiled_impl.h"

namespace qg {
hipError_t launch_mx_256x256(const MxMatmulArgs& a, bool a8, hipStream_t s) {
    return a8 ? mx::launch_out<256, 256, 64, 128, 1, 4, 3, true>(a, s) : mx::launch_out<256, 256, 128, 64, 1, 8, 2, false>(a, s);
}
}  // namespace qg
