// Kernel translation unit: grouped bfloat16 and 4-bit products, 128 x 128 tiles.
#include "lp_launch.hpp"

namespace gemmf32 {

using Tile = LpTile<128, 128, 2, 2, 2>;

int launch_lp128(const GroupedArgs &a, const LpCall &c, hipStream_t s)
{
    return c.weight_grad ? launch_lp_grad<Tile>(a, c, s) : launch_lp<Tile>(a, c, s);
}
int launch_lp128_unaligned(const GroupedArgs &a, const LpCall &c, hipStream_t s) { return launch_lp_unaligned<Tile>(a, c, s); }

}  // namespace gemmf32
