// Launches of the orthogonalising products for one tile shape (each shape's
// translation unit instantiates it).
#pragma once

#include "expert_launch.hpp"
#include "ortho_pipe.hpp"

namespace gemmf32 {

// KERNEL<..., A_KS, B_KS, E, WIDE> for what a call asks for.
#define ORTHO_KERNELS(c, KERNEL, ...)                                                                              \
    ((c).what == kOrthoGram   ? KERNEL<__VA_ARGS__, false, false, _Float16, true>                                          \
     : (c).what == kOrthoStep ? KERNEL<__VA_ARGS__, false, true, _Float16, true>                                           \
     : (c).what == kOrthoLast                                                                                    \
         ? ((c).bf16 ? ((c).wide ? KERNEL<__VA_ARGS__, false, true, __bf16, true> : KERNEL<__VA_ARGS__, false, true, __bf16, false>) \
                     : ((c).wide ? KERNEL<__VA_ARGS__, false, true, float, true> : KERNEL<__VA_ARGS__, false, true, float, false>))  \
         : ((c).bf16 ? ((c).wide ? KERNEL<__VA_ARGS__, true, false, __bf16, true> : KERNEL<__VA_ARGS__, true, false, __bf16, false>) \
                     : ((c).wide ? KERNEL<__VA_ARGS__, true, false, float, true> : KERNEL<__VA_ARGS__, true, false, float, false>)))

template <class T>
void ortho_count_tiles(OrthoArgs &a)
{
    a.tiles_m = (a.rows + T::BM - 1) / T::BM;
    a.tiles_n = (a.cols + T::BN - 1) / T::BN;
}

// A workgroup a tile, in K parts.
template <class T, int K>
int launch_ortho_tiles(OrthoArgs a, const OrthoCall &c, hipStream_t s)
{
    ortho_count_tiles<T>(a);
    return launch(ORTHO_KERNELS(c, ortho_kernel, T, K), (long long)ortho_tiles(a) * a.batch, T::THREADS * K, 0, s, a);
}

// The pipeline on `wgs` workgroups (a multiple of the XCDs), with tiles from
// a.whole on shared, and those tiles' sums.
template <class T>
int launch_ortho_pipe(OrthoArgs a, const OrthoCall &c, long long wgs, hipStream_t s)
{
    ortho_count_tiles<T>(a);
    const int st = launch(ORTHO_KERNELS(c, ortho_pipe_kernel, T), wgs, T::THREADS, 0, s, a);
    const long long shared = (long long)ortho_tiles(a) * a.batch - a.whole;
    if (st != GEMM_F32_SUCCESS || shared == 0) return st;
    return launch(ortho_join_kernel<T>, shared * (T::BM / 32) * (T::BN / 32) / 4, 256, 0, s, a);
}

}  // namespace gemmf32
