// Kernel translation unit: orthogonalising, a workgroup a small tile.
#include "ortho_launch.hpp"

namespace gemmf32 {

int launch_ortho_64_square(const OrthoArgs &a, const OrthoCall &c, hipStream_t s)
{
    return launch_ortho_tiles<LpTile<64, 64, 2, 2, 4>, 1>(a, c, s);
}
int launch_ortho_64_parts(const OrthoArgs &a, const OrthoCall &c, hipStream_t s)
{
    return launch_ortho_tiles<LpTile<64, 64, 2, 2, 4>, 2>(a, c, s);
}
int launch_ortho_64(const OrthoArgs &a, const OrthoCall &c, hipStream_t s)
{
    return launch_ortho_tiles<LpTile<64, 128, 2, 2, 3>, 1>(a, c, s);
}

}  // namespace gemmf32
