// Kernel translation unit: grouped bfloat16 and 4-bit products, 256 x 256 tiles.
#include "lp_launch.hpp"

namespace gemmf32 {

using Tile = LpTile<256, 256, 2, 4, 2>;

void launch_lp256(const GroupedArgs &a, const LpCall &c, hipStream_t s) { launch_lp<Tile>(a, c, s); }

}  // namespace gemmf32
