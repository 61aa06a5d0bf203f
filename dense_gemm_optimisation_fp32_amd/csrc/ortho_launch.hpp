// Launches of the orthogonalising products for one tile shape (each shape's
// translation unit instantiates it).
#pragma once

#include "expert_launch.hpp"
#include "orthogonal.hpp"

namespace gemmf32 {

template <class T, bool A_KS, bool B_KS, class E, bool WIDE>
int launch_ortho_kernel(const OrthoArgs &a, hipStream_t s)
{
    return launch(ortho_kernel<T, A_KS, B_KS, E, WIDE>, (long long)a.tiles_m * a.tiles_n * a.batch, T::THREADS, 0, s, a);
}

template <class T>
int launch_ortho_tiles(OrthoArgs a, const OrthoCall &c, hipStream_t s)
{
    a.tiles_m = (a.rows + T::BM - 1) / T::BM;
    a.tiles_n = (a.cols + T::BN - 1) / T::BN;
    switch (c.what) {
    case kOrthoGram: return launch_ortho_kernel<T, false, false, _Float16, true>(a, s);
    case kOrthoStep: return launch_ortho_kernel<T, false, true, _Float16, true>(a, s);
    case kOrthoLast:
        if (c.bf16)
            return c.wide ? launch_ortho_kernel<T, false, true, __bf16, true>(a, s)
                          : launch_ortho_kernel<T, false, true, __bf16, false>(a, s);
        return c.wide ? launch_ortho_kernel<T, false, true, float, true>(a, s)
                      : launch_ortho_kernel<T, false, true, float, false>(a, s);
    default:
        if (c.bf16)
            return c.wide ? launch_ortho_kernel<T, true, false, __bf16, true>(a, s)
                          : launch_ortho_kernel<T, true, false, __bf16, false>(a, s);
        return c.wide ? launch_ortho_kernel<T, true, false, float, true>(a, s)
                      : launch_ortho_kernel<T, true, false, float, false>(a, s);
    }
}

}  // namespace gemmf32
