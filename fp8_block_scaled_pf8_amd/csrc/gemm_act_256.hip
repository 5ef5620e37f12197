// Tile shapes of the product with its epilogue, apart from the rest so that they compile side by side (gfx950).
#include "gemm_act_tile.h"

namespace pf8 {

template hipError_t launch_fprop_act_tiles<256, 256>(const FpropActArgs& a, hipStream_t stream);

}  // namespace pf8
