// Launches of the expert-layer kernels, defined in their translation units
// and called by the C entry points in expert_ops.hip.  They return a
// gemm_f32_status.
#pragma once

#include "expert_common.hpp"
#include "launch.hpp"

namespace gemmf32 {

struct Mx4Args;
struct RouteArgs;

// Bound on the row tiles of bm rows: each run of rows (the experts' and the
// two of no expert) has at most one tile that is not full.
inline int grouped_row_tiles(const GroupedArgs &a, int bm)
{
    const long long tiles = (long long)a.m / bm + (a.offsets ? a.groups + 2 : 1);
    return (int)(tiles < a.m ? tiles : a.m);
}

// Workgroups of a weight gradient with a tile each: every XCD's share of every
// expert's tiles.
inline long long grad_workgroups(const GroupedArgs &a)
{
    return ((long long)a.tiles_m * a.tiles_n + a.num_xcd - 1) / a.num_xcd * a.num_xcd * a.groups;
}

// Which of a tile shape's kernels a call takes.
struct LpCall {
    bool fp4, bf16;         // 4-bit operands; 16-bit results
    bool b_contiguous;      // B's columns contiguous along k
    bool weight_grad;
    bool wide;              // 16-byte stores of C
    int cu_count;
};

// Status of the current device (a gemm_f32_status) and its facts.  In
// gemm_f32.hip.
int current_device(int *cu_count, int *num_xcd);

int launch_mx4_quantize(const Mx4Args &a, bool bf16, bool columns, hipStream_t s);
int launch_mx4_dequantize(const Mx4Args &a, bool bf16, hipStream_t s);
int launch_f32_grouped(const GroupedArgs &a, bool b_contiguous, int cu_count, hipStream_t s);
int launch_f32_weight_grad(const GroupedArgs &a, int cu_count, hipStream_t s);
int launch_lp256(GroupedArgs a, const LpCall &c, hipStream_t s);
// 64 x 128 tiles in two stages or three, 64 x 64 in four.
int launch_lp64(const GroupedArgs &a, const LpCall &c, hipStream_t s);
int launch_lp64_ring(const GroupedArgs &a, const LpCall &c, hipStream_t s);
int launch_lp64_square(const GroupedArgs &a, const LpCall &c, hipStream_t s);
int launch_lp64_square_grad(const GroupedArgs &a, const LpCall &c, hipStream_t s);
int launch_lp128(const GroupedArgs &a, const LpCall &c, hipStream_t s);
int launch_lp128_unaligned(const GroupedArgs &a, const LpCall &c, hipStream_t s);
// Few rows an expert: tiles of 16 rows.
int launch_few(const GroupedArgs &a, bool bf16, bool fp4, bool b_contiguous, int cu_count, hipStream_t s);
int launch_route(const RouteArgs &a, bool bf16, bool grad, hipStream_t s);

}  // namespace gemmf32
