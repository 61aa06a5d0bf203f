// Kernel translation unit: 8-bit products, 128 x 128 tiles and smaller.
#include "lp_launch.hpp"

namespace gemmf32 {

namespace {

template <class T>
int launch_int8(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    return c.bf16 ? launch_lp_grouped<T, kInt8, false, __bf16>(a, c.wide, s)
                  : launch_lp_grouped<T, kInt8, false, float>(a, c.wide, s);
}

}  // namespace

int launch_int8_128(const GroupedArgs &a, const LpCall &c, hipStream_t s) { return launch_int8<LpTile<128, 128, 2, 2, 2>>(a, c, s); }
int launch_int8_64(const GroupedArgs &a, const LpCall &c, hipStream_t s) { return launch_int8<LpTile<64, 128, 2, 2, 2>>(a, c, s); }
int launch_int8_64_ring(const GroupedArgs &a, const LpCall &c, hipStream_t s) { return launch_int8<LpTile<64, 128, 2, 2, 3>>(a, c, s); }
int launch_int8_64_square(const GroupedArgs &a, const LpCall &c, hipStream_t s) { return launch_int8<LpTile<64, 64, 2, 2, 4>>(a, c, s); }

}  // namespace gemmf32
