// Launches of the low-precision tile kernels for one tile shape (each
// shape's translation unit instantiates it).  Operands whose rows are not
// 4-byte aligned take the 128 x 128 tile's kernels with register copies.
#pragma once

#include "expert_launch.hpp"
#include "lp_gemm.hpp"

namespace gemmf32 {

template <class T, int KIND, bool B_KS, class E>
void launch_lp_grouped(const GroupedArgs &a, bool wide, hipStream_t s)
{
    const unsigned grid = (unsigned)a.tiles_m * a.tiles_n;
    if (wide) lp_grouped_kernel<T, KIND, B_KS, E, true><<<grid, T::THREADS, 0, s>>>(a);
    else lp_grouped_kernel<T, KIND, B_KS, E, false><<<grid, T::THREADS, 0, s>>>(a);
}

template <class T>
void launch_lp(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    if (c.fp4) {
        if (c.bf16) launch_lp_grouped<T, kFp4, false, __bf16>(a, c.wide, s);
        else launch_lp_grouped<T, kFp4, false, float>(a, c.wide, s);
    } else if (c.b_contiguous) {
        launch_lp_grouped<T, kBf16, false, __bf16>(a, c.wide, s);
    } else {
        launch_lp_grouped<T, kBf16, true, __bf16>(a, c.wide, s);
    }
}

template <class T>
void launch_lp_grad(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = (a.k + T::BM - 1) / T::BM;
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    const unsigned grid = (unsigned)grad_workgroups(a);
    if (c.wide) lp_weight_grad_kernel<T, true><<<grid, T::THREADS, 0, s>>>(a);
    else lp_weight_grad_kernel<T, false><<<grid, T::THREADS, 0, s>>>(a);
}

template <class T>
void launch_lp_unaligned(GroupedArgs a, const LpCall &c, hipStream_t s)
{
    a.tiles_m = c.weight_grad ? (a.k + T::BM - 1) / T::BM : grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    const unsigned grid = (unsigned)a.tiles_m * a.tiles_n;
    if (c.weight_grad) lp_weight_grad_kernel<T, false, true><<<(unsigned)grad_workgroups(a), T::THREADS, 0, s>>>(a);
    else if (c.b_contiguous) lp_grouped_kernel<T, kBf16, false, __bf16, false, true><<<grid, T::THREADS, 0, s>>>(a);
    else lp_grouped_kernel<T, kBf16, true, __bf16, false, true><<<grid, T::THREADS, 0, s>>>(a);
}

}  // namespace gemmf32
