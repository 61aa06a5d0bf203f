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
    using Large = Int8FewTile<X, 4, 1, 2>;
    using Small = Int8FewTile<X, 8, 1, 1>;
    using Short = Int8FewTile<X, 2, 2, 2>;
    // Strips of the larger kind that there are about: fewer than one a CU take the
    // smaller.  Measured, us, larger / smaller: 4 rows, 14336 columns, k = 4096 15.1 / 16.3;
    // 4096 columns, k = 14336 23.4 / 17.7; 16 rows over 8 experts of 14336 x 4096 77 / 87
    // (16 wavefronts or strips of 64 columns no faster in any).
    const long long rows = (a.m + 15) / 16, used = rows > a.groups ? rows : a.m < a.groups ? a.m : a.groups;
    const long long strips = used * ((a.n + Large::BN - 1) / Large::BN);
    // Many strips of short k share out columns instead (us, larger / so): 479 rows over 42
    // experts, 2752 columns, k = 256 20.2 / 15.7, 1024 37.9 / 35.6, 2048 60.1 / 60.0; 16 rows over 8
    // of 14336 columns, k = 1024 29.7 / 24.5, 4096 69.5 / 74.5; four rows, one matrix, 14336
    // columns, k = 1024 8.1 / 8.3.
    if (a.k <= 1024 && strips >= 4ll * cu_count) return launch_tile<Short, QUANTISE>(a, s);
    return strips < cu_count ? launch_tile<Small, QUANTISE>(a, s) : launch_tile<Large, QUANTISE>(a, s);
}

}  // namespace

int launch_int8_few(const GroupedArgs &a, bool bf16, bool quantise, int cu_count, hipStream_t s)
{
    if (quantise) return bf16 ? launch_kind<__bf16, true>(a, cu_count, s) : launch_kind<float, true>(a, cu_count, s);
    return bf16 ? launch_kind<__bf16, false>(a, cu_count, s) : launch_kind<float, false>(a, cu_count, s);
}

}  // namespace gemmf32
