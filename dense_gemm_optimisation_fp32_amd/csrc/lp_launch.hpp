// Launches of the low-precision tile kernels for one tile shape (each
// shape's translation unit instantiates it).  Operands whose rows are not
// 4-byte aligned take the 128 x 128 tile's kernels with register copies, whatever
// their size: the three products of 8192 rows over 16 experts take 1310 us at
// k = 2049, n = 4099 (410 + 357 + 543), 544 at 2048 x 4096 (178 + 173 + 193).  Of that,
// C's stores of single elements cost where its rows are not whole 16 bytes: 955
// at 2048 x 4098, where all copies are direct.
#pragma once

#include "expert_launch.hpp"
#include "lp_gemm.hpp"

namespace gemmf32 {

template <class T, int KIND, bool B_KS, class E>
int launch_lp_grouped(const GroupedArgs &a, bool wide, hipStream_t s)
{
    return launch(wide ? lp_grouped_kernel<T, KIND, B_KS, E, true> : lp_grouped_kernel<T, KIND, B_KS, E, false>,
                  (long long)a.tiles_m * a.tiles_n, T::THREADS, 0, s, a);
}

template <class T>
int launch_lp(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    if (c.fp4)
        return c.bf16 ? launch_lp_grouped<T, kFp4, false, __bf16>(a, c.wide, s)
                      : launch_lp_grouped<T, kFp4, false, float>(a, c.wide, s);
    return c.b_contiguous ? launch_lp_grouped<T, kBf16, false, __bf16>(a, c.wide, s)
                          : launch_lp_grouped<T, kBf16, true, __bf16>(a, c.wide, s);
}

template <class T>
int launch_lp_grad(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = (a.k + T::BM - 1) / T::BM;
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    return launch(c.wide ? lp_weight_grad_kernel<T, true> : lp_weight_grad_kernel<T, false>, grad_workgroups(a),
                  T::THREADS, 0, s, a);
}

template <class T>
int launch_lp_unaligned(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = c.weight_grad ? (a.k + T::BM - 1) / T::BM : grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    if (c.weight_grad)
        return launch(lp_weight_grad_kernel<T, false, true>, grad_workgroups(a), T::THREADS, 0, s, a);
    return launch(c.b_contiguous ? lp_grouped_kernel<T, kBf16, false, __bf16, false, true>
                                 : lp_grouped_kernel<T, kBf16, true, __bf16, false, true>,
                  (long long)a.tiles_m * a.tiles_n, T::THREADS, 0, s, a);
}

}  // namespace gemmf32
