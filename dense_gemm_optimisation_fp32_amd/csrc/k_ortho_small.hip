// Kernel translation unit: orthogonalising matrices of few rows.
#include "expert_launch.hpp"
#include "ortho_small.hpp"

namespace gemmf32 {

namespace {

template <class E, int S, int WAVES, bool SHARED, bool FIRST>
int launch_strip(const OrthoStripArgs &a, int batch, hipStream_t s)
{
    return launch(ortho_strip_kernel<E, S, WAVES, SHARED, FIRST>, (long long)batch * a.strips, WAVES * 64, 0, s, a);
}

template <class E>
int launch_type(const OrthoStripArgs &a, int blocks, bool first, int batch, hipStream_t s)
{
    if (a.strips == 1) {
        if (blocks == 1) return launch_strip<E, 1, 8, false, false>(a, batch, s);
        if (blocks == 2) return launch_strip<E, 2, 16, false, false>(a, batch, s);
        if (blocks == 3) return launch_strip<E, 3, 16, false, false>(a, batch, s);
        return launch_strip<E, 4, 16, false, false>(a, batch, s);
    }
    if (blocks == 1) return first ? launch_strip<E, 1, 8, true, true>(a, batch, s) : launch_strip<E, 1, 8, true, false>(a, batch, s);
    if (blocks == 2) return first ? launch_strip<E, 2, 8, true, true>(a, batch, s) : launch_strip<E, 2, 8, true, false>(a, batch, s);
    return first ? launch_strip<E, 4, 16, true, true>(a, batch, s) : launch_strip<E, 4, 16, true, false>(a, batch, s);
}

}  // namespace

int launch_ortho_strips(const OrthoStripArgs &a, int blocks, bool bf16, bool first, int batch, hipStream_t s)
{
    return bf16 ? launch_type<__bf16>(a, blocks, first, batch, s) : launch_type<float>(a, blocks, first, batch, s);
}

}  // namespace gemmf32
