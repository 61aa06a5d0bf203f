// Kernel translation unit: grouped bfloat16 and 4-bit products, 256 x 256 tiles.
#include "expert_launch.hpp"
#include "lp_pipe.hpp"

namespace gemmf32 {

namespace {

using Tile = LpTile<256, 256, 2, 4, 2>;

template <int KIND, bool GRAD, bool B_KS, class E>
int launch_pipe(const GroupedArgs &a, bool wide, long long grid, hipStream_t s)
{
    return launch(wide ? lp_pipe_kernel<Tile, KIND, GRAD, B_KS, E, true> : lp_pipe_kernel<Tile, KIND, GRAD, B_KS, E, false>,
                  grid, Tile::THREADS, 0, s, a);
}

}  // namespace

int launch_lp256(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = c.weight_grad ? (a.k + Tile::BM - 1) / Tile::BM : grouped_row_tiles(a, Tile::BM);
    a.tiles_n = (a.n + Tile::BN - 1) / Tile::BN;
    // A workgroup a CU, as many on each XCD.
    const long long tiles = c.weight_grad ? grad_workgroups(a) : (long long)a.tiles_m * a.tiles_n;
    const long long most = c.cu_count / a.num_xcd * a.num_xcd;
    const long long grid = tiles < most ? (tiles + a.num_xcd - 1) / a.num_xcd * a.num_xcd : most;
    if (c.weight_grad) return launch_pipe<kBf16, true, true, __bf16>(a, c.wide, grid, s);
    if (c.fp4)
        return c.bf16 ? launch_pipe<kFp4, false, false, __bf16>(a, c.wide, grid, s)
                      : launch_pipe<kFp4, false, false, float>(a, c.wide, grid, s);
    return c.b_contiguous ? launch_pipe<kBf16, false, false, __bf16>(a, c.wide, grid, s)
                          : launch_pipe<kBf16, false, true, __bf16>(a, c.wide, grid, s);
}

}  // namespace gemmf32
