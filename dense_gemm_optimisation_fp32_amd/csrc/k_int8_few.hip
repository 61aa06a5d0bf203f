// Kernel translation unit: 8-bit products, few rows an expert.
#include "expert_launch.hpp"
#include "int8_few.hpp"

namespace gemmf32 {

namespace {

template <class T, bool QUANTISE>
int launch_tile(GroupedArgs a, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    const int rows = a.m < T::BM ? a.m : T::BM;          // most of a tile
    const size_t lds = QUANTISE ? (size_t)rows * int8_few_row(a.a_kblocks * 128) : 0;
    return launch(int8_few_kernel<T, QUANTISE>, (long long)a.tiles_m * a.tiles_n, T::THREADS, lds, s, a);
}

template <class X, bool QUANTISE>
int launch_kind(const GroupedArgs &a, int cu_count, hipStream_t s)
{
    using Large = Int8FewTile<X, 4, 2>;
    using Small = Int8FewTile<X, 8, 1>;
    // Strips of the larger kind that there are about: fewer than one a CU take the
    // smaller.  Measured, us, larger / smaller: 4 rows, 14336 columns, k = 4096 15.1 / 16.3;
    // 4096 columns, k = 14336 23.4 / 17.7; 16 rows over 8 experts of 14336 x 4096 77 / 87
    // (16 wavefronts or strips of 64 columns no faster in any).
    const long long rows = (a.m + 15) / 16, used = rows > a.groups ? rows : a.m < a.groups ? a.m : a.groups;
    return used * ((a.n + Large::BN - 1) / Large::BN) < cu_count ? launch_tile<Small, QUANTISE>(a, s)
                                                                       : launch_tile<Large, QUANTISE>(a, s);
}

}  // namespace

int launch_int8_few(const GroupedArgs &a, bool bf16, bool quantise, int cu_count, hipStream_t s)
{
    if (quantise) return bf16 ? launch_kind<__bf16, true>(a, cu_count, s) : launch_kind<float, true>(a, cu_count, s);
    return bf16 ? launch_kind<__bf16, false>(a, cu_count, s) : launch_kind<float, false>(a, cu_count, s);
}

}  // namespace gemmf32
