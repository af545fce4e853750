// Tiled kernels of the fused A8W8 products, form GRAD.
#include "fused_tiled_impl.h"

namespace qg {

hipError_t launch_fused_grad(const FusedArgs& a, FusedTile tile, bool kmajor, hipStream_t s) {
    return fused::launch_form<FUSED_GRAD>(a, tile, kmajor, s);
}

}  // namespace qg
