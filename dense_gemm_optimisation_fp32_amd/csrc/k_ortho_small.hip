// Kernel translation unit: orthogonalising matrices of few rows.
#include "expert_launch.hpp"
#include "ortho_small.hpp"

namespace gemmf32 {

namespace {

template <class E, int ROWS, int S, int WAVES, bool SHARED, bool FIRST>
int launch_strip(const OrthoStripArgs &a, int batch, hipStream_t s)
{
    return launch(ortho_strip_kernel<E, ROWS, S, WAVES, SHARED, FIRST>, (long long)batch * a.strips, WAVES * 64, 0, s, a);
}

// A strip of several: X / |X| and its share, or a step.
template <class E, int ROWS, int S, int WAVES>
int launch_shared(const OrthoStripArgs &a, bool first, int batch, hipStream_t s)
{
    return first ? launch_strip<E, ROWS, S, WAVES, true, true>(a, batch, s) : launch_strip<E, ROWS, S, WAVES, true, false>(a, batch, s);
}

template <class E>
int launch_type(const OrthoStripArgs &a, int blocks, bool first, int batch, hipStream_t s)
{
    if (a.start.m_pad > 64) {
        if (a.strips == 1)
            return blocks == 1 ? launch_strip<E, 128, 1, 16, false, false>(a, batch, s)
                               : launch_strip<E, 128, 2, 16, false, false>(a, batch, s);
        return blocks == 1 ? launch_shared<E, 128, 1, 16>(a, first, batch, s) : launch_shared<E, 128, 2, 16>(a, first, batch, s);
    }
    if (a.strips == 1) {
        if (blocks == 1) return launch_strip<E, 64, 1, 8, false, false>(a, batch, s);
        if (blocks == 2) return launch_strip<E, 64, 2, 16, false, false>(a, batch, s);
        if (blocks == 3) return launch_strip<E, 64, 3, 16, false, false>(a, batch, s);
        return launch_strip<E, 64, 4, 16, false, false>(a, batch, s);
    }
    if (blocks == 1) return launch_shared<E, 64, 1, 8>(a, first, batch, s);
    if (blocks == 2) return launch_shared<E, 64, 2, 8>(a, first, batch, s);
    return launch_shared<E, 64, 4, 16>(a, first, batch, s);
}

}  // namespace

int launch_ortho_strips(const OrthoStripArgs &a, int blocks, bool bf16, bool first, int batch, hipStream_t s)
{
    return bf16 ? launch_type<__bf16>(a, blocks, first, batch, s) : launch_type<float>(a, blocks, first, batch, s);
}

}  // namespace gemmf32
