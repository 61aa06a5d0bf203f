// Kernel translation unit: products grouped by expert, few rows an expert.
#include "expert_launch.hpp"
#include "grouped_few.hpp"

namespace gemmf32 {

namespace {

template <int KIND, bool B_KS, class T>
int launch_tile(GroupedArgs a, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    return launch(few_grouped_kernel<KIND, B_KS, T>, (long long)a.tiles_m * a.tiles_n, T::THREADS, 0, s, a);
}

template <int KIND, bool B_KS, class X>
int launch_kind(const GroupedArgs &a, int cu_count, hipStream_t s)
{
    using Large = FewTile<KIND, B_KS, X, 4, 2>;
    using Small = FewTile<KIND, B_KS, X, 8, 1>;
    // Strips of the larger kind that there are about.  Few of them are bound by
    // latency, many by bandwidth (16 rows over 8 experts, 14336 columns, k =
    // 4096, bfloat16: 137 to 157 us from card to card, 5.3 to 6.1 TB/s): fewer
    // than four a CU take the smaller strips (2 of 8 experts, 4096 columns, k =
    // 1024, 32 bits: 12.0 us with the larger, 8.9 so).  In 4 bits, where a strip also quantises its rows, fewer
    // than one a CU (4 rows, 4096 columns, k = 14336: 16.5 / 10.2 us; 14336
    // columns, k = 4096: 10.4 / 12.0).
    constexpr long long least = KIND == kFewFp4 ? 1 : 4;
    const long long rows = (a.m + 15) / 16, used = rows > a.groups ? rows : a.m < a.groups ? a.m : a.groups;
    return used * ((a.n + Large::BN - 1) / Large::BN) < least * cu_count ? launch_tile<KIND, B_KS, Small>(a, s)
                                                                         : launch_tile<KIND, B_KS, Large>(a, s);
}

}  // namespace

int launch_few(const GroupedArgs &a, bool bf16, bool fp4, bool b_contiguous, int cu_count, hipStream_t s)
{
    if (fp4)
        return bf16 ? launch_kind<kFewFp4, false, __bf16>(a, cu_count, s)
                    : launch_kind<kFewFp4, false, float>(a, cu_count, s);
    if (b_contiguous)
        return bf16 ? launch_kind<kFewBf16, false, __bf16>(a, cu_count, s)
                    : launch_kind<kFewF32, false, float>(a, cu_count, s);
    return bf16 ? launch_kind<kFewBf16, true, __bf16>(a, cu_count, s)
                : launch_kind<kFewF32, true, float>(a, cu_count, s);
}

}  // namespace gemmf32
