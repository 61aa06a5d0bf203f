// Kernel translation unit: orthogonalising, 256 x 256 tiles.
#include "ortho_launch.hpp"

namespace gemmf32 {

int launch_ortho_256(const OrthoArgs &a, const OrthoCall &c, long long wgs, hipStream_t s)
{
    return launch_ortho_pipe<LpTile<256, 256, 2, 4, 2>>(a, c, wgs, s);
}

}  // namespace gemmf32
