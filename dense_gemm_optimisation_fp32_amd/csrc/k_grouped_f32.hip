// Kernel translation unit: products grouped by expert in 32 bits.
#include "expert_launch.hpp"
#include "grouped_f32.hpp"

namespace gemmf32 {

namespace {
using Tile128 = DmaTile<128, 128, 16, 2, 2, 3, false>;
}

void launch_f32_grouped(GroupedArgs a, bool b_contiguous, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, Tile128::BM);
    a.tiles_n = (a.n + Tile128::BN - 1) / Tile128::BN;
    const unsigned grid = (unsigned)a.tiles_m * a.tiles_n;
    if (b_contiguous) f32_grouped_kernel<Tile128, true><<<grid, Tile128::THREADS, 0, s>>>(a);
    else f32_grouped_kernel<Tile128, false><<<grid, Tile128::THREADS, 0, s>>>(a);
}

void launch_f32_weight_grad(GroupedArgs a, hipStream_t s)
{
    a.tiles_m = (a.k + Tile128::BM - 1) / Tile128::BM;
    a.tiles_n = (a.n + Tile128::BN - 1) / Tile128::BN;
    f32_weight_grad_kernel<Tile128><<<(unsigned)a.tiles_m * a.tiles_n * a.groups, Tile128::THREADS, 0, s>>>(a);
}

}  // namespace gemmf32
