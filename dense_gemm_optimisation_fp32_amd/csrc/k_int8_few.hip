// Kernel translation unit: 8-bit products, few rows an expert.
#include "expert_launch.hpp"
#include "int8_few.hpp"

namespace gemmf32 {

namespace {

template <class T>
int launch_tile(GroupedArgs a, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    return launch(int8_few_kernel<T>, (long long)a.tiles_m * a.tiles_n, T::THREADS, 0, s, a);
}

template <class X>
int launch_kind(const GroupedArgs &a, int cu_count, hipStream_t s)
{
    using Large = Int8FewTile<X, 4, 2>;
    using Small = Int8FewTile<X, 8, 1>;
    const long long rows = (a.m + 15) / 16, used = rows > a.groups ? rows : a.m < a.groups ? a.m : a.groups;
    return used * ((a.n + Large::BN - 1) / Large::BN) < 4ll * cu_count ? launch_tile<Small>(a, s) : launch_tile<Large>(a, s);
}

}  // namespace

int launch_int8_few(const GroupedArgs &a, bool bf16, int cu_count, hipStream_t s)
{
    return bf16 ? launch_kind<__bf16>(a, cu_count, s) : launch_kind<float>(a, cu_count, s);
}

}  // namespace gemmf32
