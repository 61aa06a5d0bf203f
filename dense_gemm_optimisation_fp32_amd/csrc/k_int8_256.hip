// Kernel translation unit: 8-bit products, 256 x 256 tiles.
#include "expert_launch.hpp"
#include "lp_pipe.hpp"

namespace gemmf32 {

namespace {

using Tile = LpTile<256, 256, 2, 4, 2>;

template <class E>
int launch_pipe(const GroupedArgs &a, bool wide, long long grid, hipStream_t s)
{
    return launch(wide ? lp_pipe_kernel<Tile, kInt8, false, false, E, true> : lp_pipe_kernel<Tile, kInt8, false, false, E, false>,
                  grid, Tile::THREADS, 0, s, a);
}

}  // namespace

int launch_int8_256(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, Tile::BM);
    a.tiles_n = (a.n + Tile::BN - 1) / Tile::BN;
    // A workgroup a CU, as many on each XCD.
    const long long tiles = (long long)a.tiles_m * a.tiles_n, most = c.cu_count / a.num_xcd * a.num_xcd;
    const long long grid = tiles < most ? (tiles + a.num_xcd - 1) / a.num_xcd * a.num_xcd : most;
    return c.bf16 ? launch_pipe<__bf16>(a, c.wide, grid, s) : launch_pipe<float>(a, c.wide, grid, s);
}

}  // namespace gemmf32
