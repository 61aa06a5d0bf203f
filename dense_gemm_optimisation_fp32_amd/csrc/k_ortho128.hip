// Kernel translation unit: orthogonalising, 128 x 128 tiles, and the planes of X.
#include "ortho_launch.hpp"

namespace gemmf32 {

int launch_ortho_128(const OrthoArgs &a, const OrthoCall &c, long long wgs, hipStream_t s)
{
    return launch_ortho_pipe<LpTile<128, 128, 2, 2, 2>>(a, c, wgs, s);
}

int launch_ortho_squares(const OrthoStartArgs &a, bool bf16, int batch, hipStream_t s)
{
    return launch(bf16 ? ortho_squares_kernel<__bf16> : ortho_squares_kernel<float>, (long long)a.parts * batch, 256, 0, s, a);
}

int launch_ortho_start(const OrthoStartArgs &a, bool bf16, int batch, hipStream_t s)
{
    const int st = launch_ortho_squares(a, bf16, batch, s);
    if (st != GEMM_F32_SUCCESS) return st;
    return launch(bf16 ? ortho_start_kernel<__bf16> : ortho_start_kernel<float>,
                  (long long)(a.m_pad / 64) * (a.n_pad / 64) * batch, 256, 0, s, a);
}

}  // namespace gemmf32
