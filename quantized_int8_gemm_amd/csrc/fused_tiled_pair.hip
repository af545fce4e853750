// Tiled kernels of the fused A8W8 products, form PAIR.
#include "fused_tiled_impl.h"

namespace qg {

hipError_t launch_fused_pair(const FusedArgs& a, FusedTile tile, bool kmajor, hipStream_t s) {
    return fused::launch_form<FUSED_PAIR>(a, tile, kmajor, s);
}

}  // namespace qg
