// Launches of the expert-layer kernels, defined in their translation units
// and called by the C entry points in expert_ops.hip.  They return a
// gemm_f32_status.
#pragma once

#include "expert_common.hpp"
#include "launch.hpp"

namespace gemmf32 {

struct BalanceArgs;
struct Int8Args;
struct Mx4Args;
struct OrthoArgs;
struct OrthoStartArgs;
struct OrthoStripArgs;
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

// Which of a tile shape's orthogonalising products a call takes: X X^T and A A,
// B X, the last B X, or its transposed.
enum OrthoProduct { kOrthoGram, kOrthoStep, kOrthoLast, kOrthoTurned };
struct OrthoCall {
    OrthoProduct what;
    bool bf16, wide;        // of the result
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
int launch_balance(const BalanceArgs &b, bool bf16, bool grad, hipStream_t s);
int launch_int8_quantize(const Int8Args &a, bool bf16, bool columns, hipStream_t s);
int launch_int8_dequantize(const Int8Args &a, bool bf16, hipStream_t s);
// 8-bit products, by tile as above.
int launch_int8_256(GroupedArgs a, const LpCall &c, hipStream_t s);
int launch_int8_128(const GroupedArgs &a, const LpCall &c, hipStream_t s);
int launch_int8_64(const GroupedArgs &a, const LpCall &c, hipStream_t s);
int launch_int8_64_ring(const GroupedArgs &a, const LpCall &c, hipStream_t s);
int launch_int8_64_square(const GroupedArgs &a, const LpCall &c, hipStream_t s);
// quantise: A holds the rows of X, which every workgroup quantises for itself.
int launch_int8_few(const GroupedArgs &a, bool bf16, bool quantise, int cu_count, hipStream_t s);
// Matrices of few rows: strips of `blocks` x 64 columns (1, 2 or 4; one strip: 1 to 4; of
// more than 64 rows 1 or 2).
int launch_ortho_strips(const OrthoStripArgs &a, int blocks, bool bf16, bool first, int batch, hipStream_t s);
int launch_ortho_squares(const OrthoStartArgs &a, bool bf16, int batch, hipStream_t s);
int launch_ortho_start(const OrthoStartArgs &a, bool bf16, int batch, hipStream_t s);
int launch_ortho_64_square(const OrthoArgs &a, const OrthoCall &c, hipStream_t s);
int launch_ortho_64_parts(const OrthoArgs &a, const OrthoCall &c, hipStream_t s);     // two parts of a workgroup share the slabs
int launch_ortho_64(const OrthoArgs &a, const OrthoCall &c, hipStream_t s);
int launch_ortho_128(const OrthoArgs &a, const OrthoCall &c, long long wgs, hipStream_t s);
int launch_ortho_256(const OrthoArgs &a, const OrthoCall &c, long long wgs, hipStream_t s);

}  // namespace gemmf32
