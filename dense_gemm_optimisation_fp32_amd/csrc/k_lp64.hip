// Kernel translation unit: grouped bfloat16 and 4-bit products, 64 x 128 tiles.
#include "lp_launch.hpp"

namespace gemmf32 {

using Tile = LpTile<64, 128, 2, 2>;

void launch_lp64(const GroupedArgs &a, const LpCall &c, hipStream_t s) { launch_lp<Tile>(a, c, s); }

}  // namespace gemmf32
