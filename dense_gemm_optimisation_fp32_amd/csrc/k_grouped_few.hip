// Kernel translation unit: products grouped by expert, few rows an expert.
#include "expert_launch.hpp"
#include "grouped_few.hpp"

namespace gemmf32 {

namespace {

template <int KIND, bool B_KS, class X, int MT>
void launch_mt(GroupedArgs a, hipStream_t s)
{
    using T = FewTile<KIND, B_KS, X>;
    a.tiles_m = grouped_row_tiles(a, 16 * MT);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    few_grouped_kernel<KIND, B_KS, X, MT><<<(unsigned)a.tiles_m * a.tiles_n, T::THREADS, 0, s>>>(a);
}

template <int KIND, bool B_KS, class X>
void launch_kind(const GroupedArgs &a, int row_tiles, hipStream_t s)
{
    if (row_tiles <= 1) launch_mt<KIND, B_KS, X, 1>(a, s);
    else launch_mt<KIND, B_KS, X, 2>(a, s);
}

}  // namespace

void launch_few(const GroupedArgs &a, bool bf16, bool fp4, bool b_contiguous, int row_tiles, hipStream_t s)
{
    if (fp4) {
        if (bf16) launch_kind<kFewFp4, false, __bf16>(a, row_tiles, s);
        else launch_kind<kFewFp4, false, float>(a, row_tiles, s);
    } else if (b_contiguous) {
        if (bf16) launch_kind<kFewBf16, false, __bf16>(a, row_tiles, s);
        else launch_kind<kFewF32, false, float>(a, row_tiles, s);
    } else {
        if (bf16) launch_kind<kFewBf16, true, __bf16>(a, row_tiles, s);
        else launch_kind<kFewF32, true, float>(a, row_tiles, s);
    }
}

}  // namespace gemmf32
