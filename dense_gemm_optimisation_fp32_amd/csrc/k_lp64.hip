// Kernel translation unit: grouped bfloat16 and 4-bit products, 64 x 128 tiles
// and, for few of them, longer rings of slabs.
#include "lp_launch.hpp"

namespace gemmf32 {

int launch_lp64(const GroupedArgs &a, const LpCall &c, hipStream_t s) { return launch_lp<LpTile<64, 128, 2, 2, 2>>(a, c, s); }
int launch_lp64_ring(const GroupedArgs &a, const LpCall &c, hipStream_t s) { return launch_lp<LpTile<64, 128, 2, 2, 3>>(a, c, s); }
int launch_lp64_square(const GroupedArgs &a, const LpCall &c, hipStream_t s) { return launch_lp<LpTile<64, 64, 2, 2, 4>>(a, c, s); }

int launch_lp64_square_grad(const GroupedArgs &a, const LpCall &c, hipStream_t s)
{
    return launch_lp_grad<LpTile<64, 64, 2, 2, 4>>(a, c, s);
}

}  // namespace gemmf32
