// Device helpers shared by the expert-layer kernels (products grouped by
// expert, 4-bit products, routing): the launch arguments, the search for the
// rows that a workgroup's tile covers, and 16-bit conversions.
#pragma once

#include "device_common.hpp"

namespace gemmf32 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned char u8;
typedef int i32x4 __attribute__((ext_vector_type(4)));

// Launch arguments of the grouped kernels.  Strides and extents in bytes.
struct GroupedArgs {
    const char *A;             // rows of A, sorted by expert
    const char *B;             // the experts' matrices (weight gradient: the rows of G)
    char *C;                   // rows of C (weight gradient: the experts' matrices)
    const u8 *a_scales;        // 4-bit products: scales of A and B, (k / 128, rows, 4)
    const u8 *b_scales;
    const float *bias;         // (groups, n) or NULL
    const int *offsets;        // groups + 1 row offsets, or NULL: one expert with every row
    int m, n, k;               // rows of A, columns of C, contraction (weight gradient: rows of dB)
    int groups;
    long long lda, ldb, ldc;   // bytes from row to row (B: from k-row to k-row, or column to column)
    long long expert_stride;   // bytes from expert to expert (B; weight gradient: C)
    long long bias_stride;     // floats from expert to expert
    int tiles_m, tiles_n;      // tiles_m: bound on the row tiles of all experts
    int group_m;               // row tiles per rasterisation group
    int num_xcd;
    int act;                   // 0 none, 1 ReLU, 2 GELU
    int a_kblocks;             // 4-bit products: 128-column blocks of a row
};

// The rows of one tile: expert (-1: rows of no expert, which become zero),
// its first row, and the expert's rows from there on.
struct RowTile {
    int expert, row, rows;
};

// Rows of entry e: an expert, or (the two entries after the experts) the rows
// after the last expert's and before the first's.  Offsets are read from
// device memory that the host has not seen, so they are clamped to the rows
// there are: a wrong list gives wrong rows, never an access outside A and C.
struct Rows {
    int lo, hi;
};

__device__ __forceinline__ Rows entry_rows(const GroupedArgs &g, int e)
{
    if (!g.offsets) return Rows{0, e == 0 ? g.m : 0};
    // Entry groups + 1 (before the first expert) and those past it begin at 0
    // and end at offsets[0], or at 0.
    const int first = g.offsets[max(0, min(e, g.groups))], next = g.offsets[e < g.groups ? e + 1 : 0];
    int lo = e <= g.groups ? first : 0;
    int hi = e == g.groups ? g.m : e <= g.groups + 1 ? next : 0;
    lo = min(max(lo, 0), g.m);
    hi = min(max(hi, lo), g.m);
    return Rows{lo, hi};
}

// Sum over the lanes up to and with this one: within rows of 16 lanes, then
// the rows' last lanes on to the rows after them.
__device__ __forceinline__ int wave_inclusive_sum(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);    // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);    // row_bcast:15 into rows 1 and 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);    // row_bcast:31 into rows 2 and 3
    return x;
}

// Workgroup id -> (row tile, column tile), and the rows of that row tile.
// Every wavefront does it for itself, 64 experts at a time: the experts' row
// tiles are counted and summed over the lanes (the number of row tiles is
// only known on the device), the workgroup's place is taken from the actual
// number of tiles, so that the XCDs share the real work evenly, and the
// expert is found by ballot.  False: the workgroup is past the last tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const GroupedArgs &g, int wg, int lane, RowTile &rt, int &tn)
{
    const int entries = g.offsets ? g.groups + 2 : 1;
    int total = 0, base = (entries - 1) / 64 * 64, sum = 0;
    Rows rows{0, 0};
    for (int b = 0; b <= base; b += 64) {
        rows = entry_rows(g, b + lane);
        sum = wave_inclusive_sum((rows.hi - rows.lo + BM - 1) / BM);
        total += __builtin_amdgcn_readlane(sum, 63);
    }
    const int all = min(total, g.tiles_m);
    if (wg >= all * g.tiles_n) return false;
    const int logical = xcd_contiguous(wg, all * g.tiles_n, g.num_xcd);
    const int width = g.group_m * g.tiles_n;
    const int first = logical / width * g.group_m;
    const int size = min(all - first, g.group_m);
    const int r = logical % width;
    const int tm = first + r % size;
    tn = r / size;
    // Back from the last 64 entries to those that hold row tile tm.
    int before = total - __builtin_amdgcn_readlane(sum, 63);
    while (before > tm) {
        base -= 64;
        rows = entry_rows(g, base + lane);
        sum = wave_inclusive_sum((rows.hi - rows.lo + BM - 1) / BM);
        before -= __builtin_amdgcn_readlane(sum, 63);
    }
    // The first lane whose running sum passes tm.
    const int at = __builtin_ctzll(__ballot(before + sum > tm));
    const int lo = __builtin_amdgcn_readlane(rows.lo, at), hi = __builtin_amdgcn_readlane(rows.hi, at);
    const int inside = tm - before - (__builtin_amdgcn_readlane(sum, at) - (hi - lo + BM - 1) / BM);
    rt.row = lo + inside * BM;
    rt.rows = hi - rt.row;
    rt.expert = base + at < g.groups ? base + at : -1;
    return true;
}

// Tiles of the weight gradients.  The contraction is an expert's rows, so the
// experts' tiles differ in work: every XCD takes an equal share of every
// expert's tiles (with whole experts to an XCD, the XCD with the most rows
// decided: 5003 rows over 16 uneven experts 365 us against 240 over even ones).
// Tile number q of XCD x; false: the XCD's last share of the expert is short.
__device__ __forceinline__ int grad_share(const GroupedArgs &g)
{
    return (g.tiles_m * g.tiles_n + g.num_xcd - 1) / g.num_xcd;
}

struct GradTile {
    int expert, tm, tn;
};

__device__ __forceinline__ bool grad_tile(const GroupedArgs &g, int x, int q, GradTile &t)
{
    const int share = grad_share(g);
    t.expert = q / share;
    const int r = x * share + q % share;
    const int width = g.group_m * g.tiles_n, first = r / width * g.group_m;
    const int size = min(g.tiles_m - first, g.group_m);
    if (r >= g.tiles_m * g.tiles_n) return false;
    t.tm = first + r % width % size;
    t.tn = r % width / size;
    return true;
}

// LDS written by a lane is read by another one of the same wavefront.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 16 bytes of a row at p, elements at or past `left` zero.  Any alignment that
// the elements have: unaligned wide loads are in order on this target.
template <class E>
__device__ __forceinline__ i32x4 load_chunk(const E *p, int left)
{
    constexpr int N = 16 / sizeof(E);
    struct __attribute__((packed, aligned(sizeof(E)))) Chunk {
        i32x4 v;
    };
    if (left >= N) return reinterpret_cast<const Chunk *>(p)->v;
    i32x4 r = {};
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left) {
            if constexpr (sizeof(E) == 4) r[i] = reinterpret_cast<const int *>(p)[i];
            else r[i / 2] |= (int)reinterpret_cast<const unsigned short *>(p)[i] << (16 * (i & 1));
        }
    return r;
}

// GELU as in gelu_erf (x Phi(x), erf by Abramowitz and Stegun 7.1.26,
// |error| <= 1.5e-7), with the reciprocal instruction (one unit in the last
// place) in place of the divide: 16 instructions instead of 26, in an epilogue
// that the matrix cores wait for.
__device__ __forceinline__ float gelu_rcp(float x)
{
    const float z = fabsf(x) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * z);
    const float poly =
        t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    // e^(-z^2) = 2^(-x^2 log2(e) / 2)
    const float y = poly * __builtin_amdgcn_exp2f(x * x * -0.72134752044448170f);
    return 0.5f * x * (x >= 0.0f ? 2.0f - y : y);
}

// (Compared so that a NaN stays one.)
__device__ __forceinline__ float activate(float x, int act)
{
    if (act == 1) x = x < 0.0f ? 0.0f : x;
    return act == 2 ? gelu_rcp(x) : x;
}

}  // namespace gemmf32
