// C entry points of include/expert_ops.h: argument checks, the choice of a
// kernel, and its launch.  No kernel is compiled in this unit.
#include "expert_ops.h"

#include <cmath>

#include "balance.hpp"
#include "expert_launch.hpp"
#include "int8.hpp"
#include "mx4.hpp"
#include "ortho_small.hpp"
#include "route.hpp"

using namespace gemmf32;

namespace {

constexpr int64_t kMaxInt = 0x7fffffff;
constexpr int64_t kMaxRowBytes = (int64_t)8 << 20;

bool size_ok(int64_t v, int64_t least) { return v >= least && v <= kMaxInt; }
bool dtype_ok(int d) { return d == EXPERT_F32 || d == EXPERT_BF16; }
bool layout_ok(int l) { return l == GEMM_F32_ROW_MAJOR || l == GEMM_F32_COL_MAJOR; }
int64_t elem(int dtype) { return dtype == EXPERT_BF16 ? 2 : 4; }
bool aligned(const void *p, int64_t to) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)to == 0; }
bool here(const void *p, int64_t to) { return p && aligned(p, to); }
int64_t padded(int64_t k) { return (k + 127) / 128 * 128; }

hipStream_t stream_of(void *s) { return reinterpret_cast<hipStream_t>(s); }

// Whether rows of C can be stored 16 bytes at a time.
bool wide_rows(const void *c, int64_t row_bytes, int64_t n, int64_t size)
{
    return aligned(c, 16) && row_bytes % 16 == 0 && n * size % 16 == 0;
}

// The tiles' workgroups are counted in 32 bits.
bool grid_ok(int64_t rows, int64_t cols, int64_t row_tile, int64_t col_tile, int64_t more)
{
    return (rows / row_tile + more) <= kMaxInt / ((cols + col_tile - 1) / col_tile);
}

// So are those of a weight gradient: every XCD (eight at most) takes an equal
// share of every expert's tiles, rounded up.
bool grad_ok(int64_t n, int64_t k, int64_t groups)
{
    const int64_t tiles = (k + 63) / 64 * ((n + 63) / 64);
    return (tiles + 7) / 8 * 8 <= kMaxInt / groups;
}

// Whether the experts' k x n matrices share no element: one after the other,
// or the experts' rows in turn.  (The workgroups of two experts would write to
// the same place.)
bool apart(int64_t n, int64_t k, int64_t groups, int64_t ld, int64_t stride)
{
    return groups == 1 || stride >= (k - 1) * ld + n || (stride >= n && ld >= (groups - 1) * stride + n);
}

// A workgroup of the routing kernels steps its slot counters by up to 1024 past
// the last slot: more slots than this could wrap them.
constexpr int64_t kMaxSlots = kMaxInt - 2047;

// Rows an expert has on average.
int64_t mean_rows(int64_t m, int64_t groups) { return (m + groups - 1) / groups; }

// Most experts of the 256 x 256 tiles' kernels.
constexpr int64_t kPipeGroups = 1022;

// Whether the products of `rows` rows an expert take 256 x 256 tiles (one
// workgroup a CU) rather than 128 x 128 (two): where a tile is mostly full and
// there is a tile for every CU.  Measured, us, 16 experts, k = 2048, n = 4096,
// 256 / 128: 128 rows 59 / 53, 160 rows 67 / 89, 192 rows 66 / 92, 256 rows 70 /
// 97, 1024 rows 259 / 334; rows uneven by a deviation of 0.3 in their logarithm:
// 160 rows 62 / 85, 176 rows 92 / 90, 192 rows 92 / 109; 512 rows, k = n = 1024 (160
// tiles) 32 / 24.
bool large_tiles(int64_t rows, int64_t m, int64_t n, int64_t groups, int cus)
{
    return rows >= 192 && groups <= kPipeGroups && (m / 256 + groups / 2 + 1) * ((n + 255) / 256) >= cus;
}

// Up to this many rows an expert on average, 64 x 128 tiles (three workgroups a
// CU): such a product is bound by the experts' matrices, and by how many of
// their bytes are under way.  Measured, us, 128 / 64 rows a tile: bfloat16, 16
// experts, k = 2048, n = 4096, 64 rows each 47 / 44, 64 on average of uneven
// ones 79 / 58, 96 rows each 51 / 81 (their matrices are read twice); 4 bits, 32
// experts, 32 rows each 43 / 39, 64 45 / 44, 96 47 / 55.
constexpr int64_t kSmallTileRows = 64;

// Tiles of bm x bn that there are about: every expert's last is not full.
int64_t tiles_of(const GroupedArgs &a, int64_t rows, int bm, int bn)
{
    return a.groups * ((rows + bm - 1) / bm) * ((a.n + bn - 1) / bn);
}

// The bfloat16 and 4-bit tiles of `rows` rows an expert.  Few tiles are bound by
// the latency of one slab after the other: tiles small enough to give every CU
// one, and rings of as many slabs as LDS holds.  Measured, us, 128 x 128 tiles
// (64 x 128 up to 64 rows) in two stages / 64 x 128 in three, two workgroups a
// CU / 64 x 64 in four: bfloat16, one expert, k = n = 4096, 64 rows 54 / 33 /
// 24, 256 rows 58 / 33 / 25, 512 rows 57 / 34 / 37; k = 2048, n = 1024, 16
// experts, 64 rows each 31 / 21 / 18, 256 rows 34 / 32 / 40, 512 rows 42 / 57 /
// 72; 4 bits, k = n = 4096, 192 rows 17 / 15 / 13.
int launch_tiles(const GroupedArgs &a, const LpCall &c, int64_t rows, hipStream_t s)
{
    if (tiles_of(a, rows, 64, 64) <= c.cu_count) return launch_lp64_square(a, c, s);
    if (tiles_of(a, rows, 64, 128) <= 2 * c.cu_count) return launch_lp64_ring(a, c, s);
    if (rows <= kSmallTileRows) return launch_lp64(a, c, s);
    if (large_tiles(rows, a.m, a.n, a.groups, c.cu_count)) return launch_lp256(a, c, s);
    return launch_lp128(a, c, s);
}

// Up to this many rows an expert on average, the few-row kernels: one tile of
// theirs holds all rows of such an expert, so its matrix is read once; of more
// rows, every 16 read it again.
constexpr int64_t kFewRows = 16;

// Whether a product takes the few-row kernels: also with more rows where C has
// few 16 x 16 blocks, whose k those split over wavefronts while a tile takes
// slab after slab.  Measured, us, tiles / few rows: 32 bits, up to four blocks a
// CU: 3 experts, k = 6544, n = 1216, 18 rows 128 / 61 (B contiguous 115 / 44),
// 128 rows, seven a CU, 128 / 131 (118 / 164); one expert, k = n = 4096, 64 rows
// 81 / 40 (74 / 61), 128 rows 81 / 81 (76 / 98).  bfloat16 and 4 bits with B
// contiguous, up to two: one expert, k = n = 4096, 32 rows 24 / 17 (4 bits 12.0 /
// 9.6), 48 rows, three a CU, 24 / 24 (12.0 / 12.9); k = n = 1024, 128 rows 8.7 /
// 6.1 (8.0 / 5.6).
bool few_rows(bool f32, bool b_contiguous, int64_t rows, int64_t n, int64_t groups, int cus)
{
    if (rows <= kFewRows) return true;
    const int64_t blocks = groups * ((rows + 15) / 16) * ((n + 15) / 16);
    return blocks <= (f32 ? 4 : b_contiguous ? 2 : 0) * cus;
}

// The row tiles are counted on the device in 32 bits, also those of offsets
// that are not sorted, where every expert may seem to own nearly all rows.
bool counts_ok(int64_t m, int64_t groups)
{
    const int64_t least = mean_rows(m, groups) <= kFewRows ? 16 : 64;      // rows of a tile
    return m / least + 1 <= kMaxInt / (groups + 2);
}

// Longest contraction of 8-bit products: 127 * 127 * k stays below 2^31.
constexpr int64_t kInt8MaxK = 131072;

// Up to two rows and this many values of X an expert, and so many bytes of LDS for
// a tile's codes, the few-row kernel quantises them in every workgroup.  Measured, us, so / by
// a launch of their own: 1 row of 4096, 4096 columns 7.2 / 8.0, 14336 columns 13.9 / 14.5;
// 2 rows of 1024 over 8 experts 5.2 / 7.4; 4 rows of 4096 16.2 / 14.8, 16 of 1024 14 / 7.7, 11 of
// 256 for each of 42 experts 79 / 20.
constexpr int64_t kInt8FewValues = 4096, kInt8FewBytes = 66 * 1024;

// Most columns to quantise: counted in 32 bits up to the end of a piece of 2048.
constexpr int64_t kInt8MaxColumns = kMaxInt - 2048;

int64_t padded16(int64_t k) { return (k + 15) / 16 * 16; }

// The 8-bit tiles of `rows` rows an expert, by launch_tiles' rules (an
// instruction takes as long, and a slab has as many bytes), but for 64 x 128 tiles
// up to 72 rows: 32 experts of 65 rows, 32-bit results, 128 / 64, us: 4096 x 2048 85 / 89,
// 4099 x 2048 95 / 87, 4099 x 2049 118 / 110.
int launch_int8_tiles(const GroupedArgs &a, const LpCall &c, int64_t rows, hipStream_t s)
{
    if (tiles_of(a, rows, 64, 64) <= c.cu_count) return launch_int8_64_square(a, c, s);
    if (tiles_of(a, rows, 64, 128) <= 2 * c.cu_count) return launch_int8_64_ring(a, c, s);
    if (rows <= kSmallTileRows + 8) return launch_int8_64(a, c, s);
    if (large_tiles(rows, a.m, a.n, a.groups, c.cu_count)) return launch_int8_256(a, c, s);
    return launch_int8_128(a, c, s);
}

// --- orthogonalising -----------------------------------------------------------

int64_t padded64(int64_t k) { return (k + 63) / 64 * 64; }

constexpr int kOrthoParts = 512;           // workgroups that sum a matrix's squares, at most
constexpr int64_t kOrthoSpace = (int64_t)2 << 30;
constexpr int64_t kOrthoShares = (int64_t)512 * 256 * 256 * 4;      // bytes for shared tiles' sums
constexpr int64_t kOrthoOneStrip = (1 << 22) - 1;       // matrices of one strip a launch (1024 threads each)
constexpr double kOrthoMost = 31.0;        // of a plane's entries

// How a batch is worked on: its planes, and as many matrices at a time as 2 GiB
// hold (one at least), or a launch.
struct OrthoPlan {
    int64_t m, n, m_pad, n_pad;            // m <= n
    int64_t x_plane, g_plane;              // bytes
    int64_t blocks, strips;                // few rows: 64-column blocks of a strip, strips (else 0)
    int64_t matrix;                        // bytes of workspace a matrix
    int64_t chunk;
    int64_t shares;                        // bytes for shared tiles' sums

    OrthoPlan(int64_t batch, int64_t rows, int64_t cols)
    {
        m = rows < cols ? rows : cols;
        n = rows < cols ? cols : rows;
        m_pad = padded64(m);
        n_pad = padded64(n);
        x_plane = m_pad * n_pad * 2;
        g_plane = m_pad * m_pad * 2;
        matrix = 4 * x_plane + 4 * g_plane + kOrthoParts * 8 + 8;
        // Few rows: one strip (up to 256 columns, of 128 rows 128), else sixteen at most
        // up to 4096 columns, of 128 rows eight.  Measured, us: four of 64 x 192 25, by the
        // tiles 82; 64 x 384 in one strip 40.4, in six, a launch a step, 40; 128 x 128 56, by the
        // tiles 102, 128 x 512 86 / about 120, 128 x 1024 106 (bfloat16 107), 128 x 1088 by the
        // tiles 152 (143).  Longer ones of 64 rows stay in strips of 256 columns, each of which
        // adds up the shares of all in every step: 64 x 4096 69, 16384 107, 65536 263, 131072 843;
        // the tiles have not been measured there.
        const int64_t all = n_pad / 64;
        blocks = strips = 0;
        if (m <= 64) blocks = all <= 4 ? all : all <= 16 ? 1 : all <= 32 ? 2 : 4;
        else if (m <= 128 && all <= 16) blocks = all <= 2 ? all : all <= 8 ? 1 : 2;
        if (blocks) {
            strips = (all + blocks - 1) / blocks;
            matrix = strips == 1 ? 0 : 2 * x_plane + 2 * strips * m_pad * m_pad * 4 + kOrthoParts * 8;
        }
        chunk = matrix ? kOrthoSpace / matrix : kOrthoOneStrip;
        chunk = chunk < 1 ? 1 : chunk > batch ? batch : chunk;
        // (Small tiles are a workgroup's each where they are few, whatever their length.  From
        // 4096 columns on sharing them would be faster, 32 bits, us, so / shared: 1024 x 1024 262 / 263,
        // 1024 x 4096 547 / 525, 768 x 4096 482 / 434, 768 x 16384 1330 / 892, 512 x 32768 2192 / 869.)
        const int64_t side = m_pad / 64;
        shares = !strips && chunk * (side * (side + 1) / 2) > 256 ? kOrthoShares : 0;
    }
};

bool ortho_sizes_ok(int dtype, int64_t batch, int64_t rows, int64_t cols)
{
    const int64_t most = rows < cols ? cols : rows;
    return dtype_ok(dtype) && size_ok(batch, 0) && size_ok(rows, 1) && size_ok(cols, 1) && padded64(most) * 2 < kMaxRowBytes;
}

// Whether what the steps make of singular values of 0 .. 1 keeps the entries that
// planes hold, of X, A and B, below kOrthoMost (an entry is at most the largest singular value).
bool ortho_bounded(const float *coefficients, int steps)
{
    double top = 1.0;
    for (int i = 0; i < steps; ++i) {
        const double a = coefficients[3 * i], b = coefficients[3 * i + 1], c = coefficients[3 * i + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
        const double end = top * top;
        const auto q = [&](double u) { return std::fabs(a + b * u + c * u * u); };
        // B: a + b u + c u^2, largest at an end or where b + 2 c u = 0.
        double most = std::fmax(q(0.0), q(end));
        const double turn = c != 0.0 ? -b / (2.0 * c) : -1.0;
        if (turn > 0.0 && turn < end) most = std::fmax(most, q(turn));
        // X: sqrt(u) (a + b u + c u^2), largest at the end or where a + 3 b u + 5 c u^2 = 0.
        // (Each root in the form that takes no difference of near numbers, which a small c leaves.)
        double next = top * q(end);
        const double root = 9.0 * b * b - 20.0 * a * c;
        if (root >= 0.0) {
            const double half = -0.5 * (3.0 * b + std::copysign(std::sqrt(root), b));
            for (const double u : {half / (5.0 * c), a / half})
                if (u > 0.0 && u < end) next = std::fmax(next, std::sqrt(u) * q(u));
        }
        // (The last step's X is the result, in its own type.)
        if (!(end < kOrthoMost && most < kOrthoMost && (next < kOrthoMost || i + 1 == steps))) return false;
        top = next * 1.001;                // (rounding)
    }
    return true;
}

// `batch` matrices of few rows; o: x and the planes at the workspace's start.
int ortho_few_rows(const OrthoPlan &p, OrthoStartArgs o, int steps, const float *coefficients, float scale, bool bf16,
                   int batch, char *y, int64_t ldy, int64_t stride_y, hipStream_t s)
{
    OrthoStripArgs a{};
    a.strips = (int)p.strips;
    a.steps = steps;
    a.order = (int)p.m;
    a.width = (int)p.n;
    a.scale = scale;
    a.ldy = ldy;
    a.stride_y = stride_y;
    if (p.strips == 1) {
        a.start = o;
        a.y = y;
        for (int i = 0; i < 3 * steps; ++i) a.f[i] = coefficients[i];
        return launch_ortho_strips(a, (int)p.blocks, bf16, false, batch, s);
    }
    const int64_t shares = p.strips * p.m_pad * p.m_pad;             // floats a matrix
    float *const g0 = reinterpret_cast<float *>(o.planes + p.chunk * 2 * p.x_plane), *const g1 = g0 + p.chunk * shares;
    o.sums = reinterpret_cast<double *>(g1 + p.chunk * shares);
    int status = launch_ortho_squares(o, bf16, batch, s);
    if (status != GEMM_F32_SUCCESS) return status;
    a.start = o;
    a.planes_out = o.planes;
    a.shares_out = g0;
    status = launch_ortho_strips(a, (int)p.blocks, bf16, true, batch, s);
    for (int i = 0; i < steps && status == GEMM_F32_SUCCESS; ++i) {
        a.shares = i % 2 ? g1 : g0;
        a.shares_out = i % 2 ? g0 : g1;
        for (int j = 0; j < 3; ++j) a.f[j] = coefficients[3 * i + j];
        a.y = i + 1 == steps ? y : nullptr;
        status = launch_ortho_strips(a, (int)p.blocks, bf16, false, batch, s);
    }
    return status;
}

// How a product runs: tiles and workgroups, and what that takes, about, in us.
struct OrthoChoice {
    // 64 x 64 (in two parts, in one) and 64 x 128 a workgroup each; 128 and 256 in the pipeline.
    enum Kind { PARTS, SMALL, WIDE, MIDDLE, LARGE } kind;
    double us;
    int64_t wgs, whole;                                // tiles [0, whole) a workgroup's each, the others shared
};

// The fastest by a model of what was measured on one MI355X (us; slabs of 64 in the
// contraction; "shared" with the launch that joins):
//   product             tiles of 64, in parts / 64 x 128 / 128, shared / 256, shared
//   1024^2, 48          22 17   -   49 24   79 33   (symmetric)
//                       23 18  30   52 26   66 34
//   1536^2, 72          40 45   -   70 38  109 42   (symmetric)
//   2048^2, 96          83  -   -   90 61  132 57   (symmetric)
//                      101  -  77   93 86  123 73
//   4096^2, 192        488  -   -  379 284 272 256  (symmetric)
//                      705  - 560  475  -  330  -
//   16 x 2048^2, 64    580  -   -  380 376 328 320  (symmetric)
//   1088 x 5056, 34     60  -  52   47 58   56 56
//   1088^2, 79          32 25   -   72 30  103 39   (symmetric)
// A slab costs more the more CUs are at work (the clock falls); a tile of 256 has 6 us
// besides, 13 where it is stored on both sides of the diagonal; shares are written and
// read.
OrthoChoice ortho_choose(const OrthoArgs &a, int cus, bool may_share)
{
    const int64_t slabs = (int64_t)a.segments * (a.k / 64);
    const auto tiles = [&](int64_t bm, int64_t bn) {
        const int64_t tm = (a.rows + bm - 1) / bm, tn = (a.cols + bn - 1) / bn;
        return a.batch * (a.symmetric ? tm * (tm + 1) / 2 : tm * tn);
    };
    const auto rounds = [](int64_t n, int64_t slots) { return (double)((n + slots - 1) / slots); };
    const auto busy = [](int64_t n, int64_t slots) { return n < slots ? (double)n / slots : 1.0; };
    const int64_t n64 = tiles(64, 64);
    OrthoChoice best{n64 <= cus ? OrthoChoice::PARTS : OrthoChoice::SMALL,
                     2.0 + slabs * (n64 <= cus ? 0.33 : rounds(n64, 2 * cus) * 0.52), 0, 0};
    const auto take = [&](OrthoChoice::Kind kind, double us, int64_t wgs, int64_t whole) {
        if (us < best.us) best = OrthoChoice{kind, us, wgs, whole};
    };
    if (!a.symmetric) {
        const int64_t n = tiles(64, 128);
        take(OrthoChoice::WIDE, 2.0 + slabs * (n <= cus ? 0.62 : rounds(n, 2 * cus) * 0.75), 0, 0);
    }
    for (const int64_t side : {128, 256}) {
        const bool large = side == 256;
        const OrthoChoice::Kind kind = large ? OrthoChoice::LARGE : OrthoChoice::MIDDLE;
        const int64_t n = tiles(side, side), slots = cus / a.num_xcd * a.num_xcd * (large ? 1 : 2), left = n % slots;
        const double more = (a.symmetric ? 13.0 : 6.0) * (large ? 1.0 : 0.5);
        const double slab = large ? 1.15 + 0.55 * busy(n, slots) : 0.75 + 0.5 * busy(n, slots);
        take(kind, rounds(n, slots) * (slabs * slab + more), n < slots ? (n + a.num_xcd - 1) / a.num_xcd * a.num_xcd : slots, n);
        // (A part of fewer than four slabs is all start and end.)
        if (!may_share || left == 0 || (slots + left) * side * side * 4 > kOrthoShares || left * slabs < 4 * slots) continue;
        const double full = large ? 1.7 : 1.25, share_mb = (slots + left) * side * side * 4 * 1e-6;
        const double result_mb = left * side * side * 4e-6 * (a.symmetric ? 2 : 1);
        take(kind, n / slots * (slabs * full + more) + (double)(left * slabs) / slots * full + 8.0 + share_mb / 5.0 + 7.0 +
                       share_mb / 7.0 + result_mb / 5.0, slots, n - left);
    }
    return best;
}

int launch_ortho(OrthoArgs a, const OrthoCall &c, int cus, hipStream_t s)
{
    const OrthoChoice o = ortho_choose(a, cus, a.shares && (c.what == kOrthoGram || c.what == kOrthoStep));
    a.whole = (int)o.whole;
    a.shared_wgs = (int)o.wgs;
    switch (o.kind) {
    case OrthoChoice::PARTS: return launch_ortho_64_parts(a, c, s);
    case OrthoChoice::SMALL: return launch_ortho_64_square(a, c, s);
    case OrthoChoice::WIDE: return launch_ortho_64(a, c, s);
    case OrthoChoice::MIDDLE: return launch_ortho_128(a, c, o.wgs, s);
    default: return launch_ortho_256(a, c, o.wgs, s);
    }
}

}  // namespace

extern "C" {

int expert_grouped_linear(int dtype, int64_t m, int64_t n, int64_t k, int64_t groups, const void *A, int64_t lda,
                          const void *B, int layout_b, int64_t ldb, int64_t expert_stride, const int *offsets,
                          const float *bias, int activation, void *C, int64_t ldc, void *stream)
{
    const bool col = layout_b == GEMM_F32_COL_MAJOR;
    if (!dtype_ok(dtype) || !layout_ok(layout_b) || !size_ok(m, 0) || !size_ok(n, 1) || !size_ok(k, 1) ||
        !size_ok(groups, 1) || lda < k || ldb < (col ? k : n) || ldc < n || expert_stride < 0 || activation < 0 ||
        activation > 2)
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t size = elem(dtype);
    if (lda * size >= kMaxRowBytes || ldb * size >= kMaxRowBytes || ldc * size >= kMaxRowBytes)
        return GEMM_F32_ERR_INVALID_VALUE;
    if (!here(offsets, 4) || !here(B, size) || (bias && !aligned(bias, 4)) || (m > 0 && (!here(A, size) || !here(C, size))))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (dtype == EXPERT_F32 && (col ? (n - 1) * ldb + k : (k - 1) * ldb + n) * size > kMaxInt - 3)
        return GEMM_F32_ERR_INVALID_VALUE;
    if (!grid_ok(m, n, 16, 32, groups + 2) || !counts_ok(m, groups)) return GEMM_F32_ERR_INVALID_VALUE;
    GroupedArgs a{};
    int cus = 0;
    const int st = current_device(&cus, &a.num_xcd);
    if (st != GEMM_F32_SUCCESS) return st;
    if (m == 0) return GEMM_F32_SUCCESS;
    a.A = static_cast<const char *>(A);
    a.B = static_cast<const char *>(B);
    a.C = static_cast<char *>(C);
    a.bias = bias;
    a.offsets = offsets;
    a.m = (int)m;
    a.n = (int)n;
    a.k = (int)k;
    a.groups = (int)groups;
    a.lda = lda * size;
    a.ldb = ldb * size;
    a.ldc = ldc * size;
    a.expert_stride = expert_stride * size;
    a.bias_stride = n;
    a.group_m = 8;
    a.act = activation;
    const hipStream_t s = stream_of(stream);
    const int64_t rows = mean_rows(m, groups);
    // The copies of the bfloat16 tiles need 4-byte aligned rows.
    const bool copies = dtype == EXPERT_F32 || (aligned(A, 4) && aligned(B, 4) && a.lda % 4 == 0 && a.ldb % 4 == 0 &&
                                                a.expert_stride % 4 == 0);
    if (few_rows(dtype == EXPERT_F32, col, rows, n, groups, cus))
        return launch_few(a, dtype == EXPERT_BF16, false, col, cus, s);
    if (dtype == EXPERT_F32) return launch_f32_grouped(a, col, cus, s);
    const LpCall c{false, true, col, false, wide_rows(C, a.ldc, n, size), cus};
    return copies ? launch_tiles(a, c, rows, s) : launch_lp128_unaligned(a, c, s);
}

int expert_grouped_weight_grad(int dtype, int64_t m, int64_t n, int64_t k, int64_t groups, const void *A, int64_t lda,
                               const void *G, int64_t ldg, const int *offsets, void *dB, int64_t ldd,
                               int64_t expert_stride, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(m, 0) || !size_ok(n, 1) || !size_ok(k, 1) || !size_ok(groups, 1) || lda < k ||
        ldg < n || ldd < n || expert_stride < 0)
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t size = elem(dtype);
    if (lda * size >= kMaxRowBytes || ldg * size >= kMaxRowBytes || ldd * size >= kMaxRowBytes)
        return GEMM_F32_ERR_INVALID_VALUE;
    if (!here(offsets, 4) || !here(dB, size) || (m > 0 && (!here(A, size) || !here(G, size))))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (dtype == EXPERT_F32 && ((k - 1) * ldd + n) * size > kMaxInt - 3) return GEMM_F32_ERR_INVALID_VALUE;
    if (!apart(n, k, groups, ldd, expert_stride) || !grad_ok(n, k, groups)) return GEMM_F32_ERR_INVALID_VALUE;
    GroupedArgs a{};
    int cus = 0;
    const int st = current_device(&cus, &a.num_xcd);
    if (st != GEMM_F32_SUCCESS) return st;
    a.A = static_cast<const char *>(A);
    a.B = static_cast<const char *>(G);
    a.C = static_cast<char *>(dB);
    a.offsets = offsets;
    a.m = (int)m;
    a.n = (int)n;
    a.k = (int)k;
    a.groups = (int)groups;
    a.lda = lda * size;
    a.ldb = ldg * size;
    a.ldc = ldd * size;
    a.expert_stride = expert_stride * size;
    a.group_m = 8;
    const hipStream_t s = stream_of(stream);
    if (dtype == EXPERT_F32) return launch_f32_weight_grad(a, cus, s);
    const LpCall c{false, true, false, true, wide_rows(dB, a.ldc, n, size) && a.expert_stride % 16 == 0, cus};
    const bool copies = aligned(A, 4) && aligned(G, 4) && a.lda % 4 == 0 && a.ldb % 4 == 0;
    if (!copies) return launch_lp128_unaligned(a, c, s);
    // Few tiles: 64 x 64 in four stages (one expert, k = n = 1024, 128 x 128 / 64 x
    // 64: 64 rows 4.5 / 3.9 us, 1024 rows 12.4 / 9.0, 4096 rows 43 / 26; at 2 to 4
    // such tiles a CU, 64 x 128 in three stages gave nothing: k = n = 2048, 1024 rows
    // 14.8 / 17.3).
    if (groups * ((k + 63) / 64) * ((n + 63) / 64) <= cus) return launch_lp64_square_grad(a, c, s);
    // The larger tiles from 384 rows on, the length of the contraction, where there
    // is one for every CU (k = 2048, n = 4096, 256 / 128, us: 256 rows 137 / 135, 352 rows
    // 159 / 159, 384 rows 163 / 155, 416 rows 171 / 186, 512 rows 186 / 216, 1024 rows 287 /
    // 346; uneven ones 384 rows 173 / 159, 416 rows 177 / 186: the two meet near 400).
    if (mean_rows(m, groups) >= 384 && groups * ((k + 255) / 256) * ((n + 255) / 256) >= cus)
        return launch_lp256(a, c, s);
    return launch_lp128(a, c, s);
}

int expert_mx4_quantize(int dtype, int64_t rows, int64_t k, const void *X, int layout, int64_t ld, void *codes,
                        void *scales, void *stream)
{
    if (!dtype_ok(dtype) || !layout_ok(layout) || !size_ok(rows, 0) || !size_ok(k, 1) || k > kMaxInt - 1024 ||
        ld < (layout == GEMM_F32_COL_MAJOR ? rows : k))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (rows > 0 && (!here(X, elem(dtype)) || !here(codes, 16) || !here(scales, 4))) return GEMM_F32_ERR_INVALID_VALUE;
    if (rows > (kMaxInt - 3) / ((k + 31) / 32)) return GEMM_F32_ERR_INVALID_VALUE;
    const int st = current_device(nullptr, nullptr);
    if (st != GEMM_F32_SUCCESS) return st;
    if (rows == 0) return GEMM_F32_SUCCESS;
    const Mx4Args a{static_cast<const char *>(X), static_cast<u8 *>(codes), static_cast<u8 *>(scales), ld, (int)rows,
                    (int)k, (int)padded(k)};
    return launch_mx4_quantize(a, dtype == EXPERT_BF16, layout == GEMM_F32_COL_MAJOR, stream_of(stream));
}

int expert_mx4_dequantize(int dtype, int64_t rows, int64_t k, const void *codes, const void *scales, void *X,
                          int64_t ld, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(rows, 0) || !size_ok(k, 1) || k > kMaxInt - 1024 || ld < k)
        return GEMM_F32_ERR_INVALID_VALUE;
    if (rows > 0 && (!here(X, elem(dtype)) || !here(codes, 16) || !here(scales, 4))) return GEMM_F32_ERR_INVALID_VALUE;
    if (rows > (kMaxInt - 3) / ((k + 31) / 32)) return GEMM_F32_ERR_INVALID_VALUE;
    const int st = current_device(nullptr, nullptr);
    if (st != GEMM_F32_SUCCESS) return st;
    if (rows == 0) return GEMM_F32_SUCCESS;
    const Mx4Args a{static_cast<const char *>(X), static_cast<u8 *>(const_cast<void *>(codes)),
                    static_cast<u8 *>(const_cast<void *>(scales)), ld, (int)rows, (int)k, (int)padded(k)};
    return launch_mx4_dequantize(a, dtype == EXPERT_BF16, stream_of(stream));
}

int64_t expert_mx4_workspace(int64_t m, int64_t n, int64_t k, int64_t groups)
{
    if (!size_ok(m, 1) || !size_ok(n, 1) || !size_ok(k, 1) || !size_ok(groups, 1)) return 0;
    if (mean_rows(m, groups) <= kFewRows) return 0;
    // X's codes and scales.
    return m * (padded(k) / 2 + padded(k) / 32);
}

int expert_mx4_linear(int dtype, int64_t m, int64_t n, int64_t k, int64_t groups, const void *X, int64_t ldx,
                      const void *codes, const void *scales, const int *offsets, const float *bias, int activation,
                      void *Y, int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(m, 0) || !size_ok(n, 1) || !size_ok(k, 1) || !size_ok(groups, 1) || ldx < k ||
        ldy < n || activation < 0 || activation > 2 || (!offsets && groups != 1))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t size = elem(dtype), kp = padded(k);
    if (ldx * size >= kMaxRowBytes || ldy * size >= kMaxRowBytes || kp > kMaxRowBytes) return GEMM_F32_ERR_INVALID_VALUE;
    if ((offsets && !aligned(offsets, 4)) || !here(codes, 16) || !here(scales, 4) || (bias && !aligned(bias, 4)) ||
        (m > 0 && (!here(X, size) || !here(Y, size))))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (!grid_ok(m, n, 16, 32, groups + 2) || !counts_ok(m, groups) || m > (kMaxInt - 3) / ((k + 31) / 32))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t need = expert_mx4_workspace(m, n, k, groups);
    if (need > 0 && !here(workspace, 16)) return GEMM_F32_ERR_INVALID_VALUE;
    if (workspace_bytes < need) return GEMM_F32_ERR_SCRATCH_TOO_SMALL;
    GroupedArgs a{};
    int cus = 0;
    const int st = current_device(&cus, &a.num_xcd);
    if (st != GEMM_F32_SUCCESS) return st;
    if (m == 0) return GEMM_F32_SUCCESS;
    a.A = static_cast<const char *>(X);
    a.B = static_cast<const char *>(codes);
    a.C = static_cast<char *>(Y);
    a.b_scales = static_cast<const u8 *>(scales);
    a.bias = bias;
    a.offsets = offsets;
    a.m = (int)m;
    a.n = (int)n;
    a.k = (int)k;
    a.groups = (int)groups;
    a.lda = ldx * size;
    a.ldb = kp / 2;
    a.ldc = ldy * size;
    a.expert_stride = n * (kp / 2);
    a.bias_stride = n;
    a.group_m = 8;
    a.act = activation;
    a.a_kblocks = (int)(kp / 128);
    const hipStream_t s = stream_of(stream);
    const bool bf16 = dtype == EXPERT_BF16;
    const int64_t rows = mean_rows(m, groups);
    if (few_rows(false, true, rows, n, groups, cus)) return launch_few(a, bf16, true, true, cus, s);
    u8 *const xc = static_cast<u8 *>(workspace), *const xs = xc + m * (kp / 2);
    const int quantised =
        launch_mx4_quantize(Mx4Args{static_cast<const char *>(X), xc, xs, ldx, (int)m, (int)k, (int)kp}, bf16, false, s);
    if (quantised != GEMM_F32_SUCCESS) return quantised;
    a.A = reinterpret_cast<const char *>(xc);
    a.a_scales = xs;
    a.lda = kp / 2;
    const LpCall c{true, bf16, true, false, wide_rows(Y, a.ldc, n, size), cus};
    return launch_tiles(a, c, rows, s);
}

int64_t expert_route_workspace(int64_t tokens, int64_t groups)
{
    if (!size_ok(tokens, 1) || !size_ok(groups, 1) || tokens <= kRouteTokens) return 0;
    return (tokens + kRouteTokens - 1) / kRouteTokens * groups * 4;
}

int expert_route(int dtype, int64_t tokens, int64_t groups, int64_t choices, int normalize, const void *logits,
                 int64_t ld, float *weights, int *experts, int *offsets, int *order, void *workspace,
                 int64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(tokens, 0) || groups < 1 || groups > kRouteMaxExperts || choices < 1 ||
        choices > groups || choices > kRouteMaxChoices || tokens * choices > kMaxSlots || ld < groups ||
        (normalize != 0 && normalize != 1) || !here(offsets, 4))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (tokens > 0 && (!here(logits, elem(dtype)) || !here(weights, 4) || !here(experts, 4) || !here(order, 4)))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t need = expert_route_workspace(tokens, groups);
    if (need > 0 && !here(workspace, 4)) return GEMM_F32_ERR_INVALID_VALUE;
    if (workspace_bytes < need) return GEMM_F32_ERR_SCRATCH_TOO_SMALL;
    const int st = current_device(nullptr, nullptr);
    if (st != GEMM_F32_SUCCESS) return st;
    RouteArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.weights = weights;
    a.experts = experts;
    a.offsets = offsets;
    a.order = order;
    a.counts = static_cast<int *>(workspace);
    a.tokens = (int)tokens;
    a.groups = (int)groups;
    a.choices = (int)choices;
    a.normalize = normalize;
    return launch_route(a, dtype == EXPERT_BF16, false, stream_of(stream));
}

int expert_route_grad(int dtype, int64_t tokens, int64_t groups, int64_t choices, int normalize, const void *logits,
                      int64_t ld, const float *weights, const int *experts, const float *grad, void *dlogits,
                      int64_t ldd, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(tokens, 0) || groups < 1 || groups > kRouteMaxExperts || choices < 1 ||
        choices > groups || choices > kRouteMaxChoices || tokens * choices > kMaxInt || ld < groups || ldd < groups ||
        (normalize != 0 && normalize != 1))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (tokens > 0 && (!here(logits, elem(dtype)) || !here(weights, 4) || !here(experts, 4) || !here(grad, 4) ||
                       !here(dlogits, elem(dtype))))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int st = current_device(nullptr, nullptr);
    if (st != GEMM_F32_SUCCESS) return st;
    if (tokens == 0) return GEMM_F32_SUCCESS;
    RouteArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.weights = const_cast<float *>(weights);
    a.experts = const_cast<int *>(experts);
    a.tokens = (int)tokens;
    a.groups = (int)groups;
    a.choices = (int)choices;
    a.normalize = normalize;
    a.grad = grad;
    a.dlogits = dlogits;
    a.ldd = ldd;
    return launch_route(a, dtype == EXPERT_BF16, true, stream_of(stream));
}

int64_t expert_route_balanced_workspace(int64_t tokens, int64_t groups)
{
    if (!size_ok(tokens, 1) || !size_ok(groups, 1) || (tokens <= kRouteTokens && groups <= 512)) return 0;
    const int64_t part = tokens <= kBalanceFewTokens ? kBalancePart : kRouteTokens;
    return (tokens + part - 1) / part * groups * 4;
}

int expert_route_balanced(int dtype, int64_t tokens, int64_t groups, int64_t choices, int scores, int64_t sets,
                          int64_t kept_sets, int normalize, float scale, const void *logits, int64_t ld,
                          const float *bias, float *weights, int *experts, int *offsets, int *order, void *workspace,
                          int64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(tokens, 0) || groups < 1 || groups > kRouteMaxExperts || sets < 1 ||
        sets > kBalanceMaxSets || groups % sets != 0 || kept_sets < 1 || kept_sets > sets || choices < 1 ||
        choices > groups / sets * kept_sets || choices > kRouteMaxChoices || tokens * choices > kMaxSlots || ld < groups ||
        (scores != EXPERT_SIGMOID && scores != EXPERT_SOFTMAX) || (normalize != 0 && normalize != 1) ||
        !(scale > 0.0f && std::isfinite(scale)) || !here(offsets, 4) || (bias && !aligned(bias, 4)))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (tokens > 0 && (!here(logits, elem(dtype)) || !here(weights, 4) || !here(experts, 4) || !here(order, 4)))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t need = expert_route_balanced_workspace(tokens, groups);
    if (need > 0 && !here(workspace, 4)) return GEMM_F32_ERR_INVALID_VALUE;
    if (workspace_bytes < need) return GEMM_F32_ERR_SCRATCH_TOO_SMALL;
    const int st = current_device(nullptr, nullptr);
    if (st != GEMM_F32_SUCCESS) return st;
    BalanceArgs b{};
    b.route.logits = logits;
    b.route.ld = ld;
    b.route.weights = weights;
    b.route.experts = experts;
    b.route.offsets = offsets;
    b.route.order = order;
    b.route.counts = static_cast<int *>(workspace);
    b.route.tokens = (int)tokens;
    b.route.groups = (int)groups;
    b.route.choices = (int)choices;
    b.route.normalize = normalize;
    // No token: the offsets alone, as of any other call.
    if (tokens == 0) return launch_route(b.route, dtype == EXPERT_BF16, false, stream_of(stream));
    b.bias = bias;
    b.softmax = scores == EXPERT_SOFTMAX;
    b.sets = (int)sets;
    b.kept = (int)kept_sets;
    b.scale = scale;
    return launch_balance(b, dtype == EXPERT_BF16, false, stream_of(stream));
}

int expert_route_balanced_grad(int dtype, int64_t tokens, int64_t groups, int64_t choices, int scores, int normalize,
                               float scale, const void *logits, int64_t ld, const float *weights, const int *experts,
                               const float *grad, void *dlogits, int64_t ldd, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(tokens, 0) || groups < 1 || groups > kRouteMaxExperts || choices < 1 ||
        choices > groups || choices > kRouteMaxChoices || tokens * choices > kMaxInt || ld < groups || ldd < groups ||
        (scores != EXPERT_SIGMOID && scores != EXPERT_SOFTMAX) || (normalize != 0 && normalize != 1) ||
        !(scale > 0.0f && std::isfinite(scale)))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (tokens > 0 && (!here(logits, elem(dtype)) || !here(weights, 4) || !here(experts, 4) || !here(grad, 4) ||
                       !here(dlogits, elem(dtype))))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int st = current_device(nullptr, nullptr);
    if (st != GEMM_F32_SUCCESS) return st;
    if (tokens == 0) return GEMM_F32_SUCCESS;
    BalanceArgs b{};
    b.route.logits = logits;
    b.route.ld = ld;
    b.route.weights = const_cast<float *>(weights);
    b.route.experts = const_cast<int *>(experts);
    b.route.tokens = (int)tokens;
    b.route.groups = (int)groups;
    b.route.choices = (int)choices;
    b.route.normalize = normalize;
    b.route.grad = grad;
    b.route.dlogits = dlogits;
    b.route.ldd = ldd;
    b.softmax = scores == EXPERT_SOFTMAX;
    b.scale = scale;
    return launch_balance(b, dtype == EXPERT_BF16, true, stream_of(stream));
}

int expert_int8_quantize(int dtype, int64_t rows, int64_t k, const void *X, int layout, int64_t ld, void *codes,
                         float *scales, void *stream)
{
    if (!dtype_ok(dtype) || !layout_ok(layout) || !size_ok(rows, 0) || !size_ok(k, 1) || k > kInt8MaxColumns ||
        ld < (layout == GEMM_F32_COL_MAJOR ? rows : k))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (rows > 0 && (!here(X, elem(dtype)) || !here(codes, 16) || !here(scales, 4))) return GEMM_F32_ERR_INVALID_VALUE;
    const int st = current_device(nullptr, nullptr);
    if (st != GEMM_F32_SUCCESS) return st;
    if (rows == 0) return GEMM_F32_SUCCESS;
    const Int8Args a{static_cast<const char *>(X), static_cast<char *>(codes), scales, ld, (int)rows, (int)k, (int)padded16(k)};
    return launch_int8_quantize(a, dtype == EXPERT_BF16, layout == GEMM_F32_COL_MAJOR, stream_of(stream));
}

int expert_int8_dequantize(int dtype, int64_t rows, int64_t k, const void *codes, const float *scales, void *X,
                           int64_t ld, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(rows, 0) || !size_ok(k, 1) || k > kMaxInt - 1024 || ld < k)
        return GEMM_F32_ERR_INVALID_VALUE;
    if (rows > 0 && (!here(X, elem(dtype)) || !here(codes, 16) || !here(scales, 4))) return GEMM_F32_ERR_INVALID_VALUE;
    const int st = current_device(nullptr, nullptr);
    if (st != GEMM_F32_SUCCESS) return st;
    if (rows == 0) return GEMM_F32_SUCCESS;
    const Int8Args a{static_cast<const char *>(X), static_cast<char *>(const_cast<void *>(codes)), const_cast<float *>(scales), ld,
                     (int)rows, (int)k, (int)padded16(k)};
    return launch_int8_dequantize(a, dtype == EXPERT_BF16, stream_of(stream));
}

int64_t expert_int8_workspace(int64_t m, int64_t k)
{
    if (!size_ok(m, 1) || !size_ok(k, 1)) return 0;
    // X's codes and scales.
    return m * (padded(k) + 4);
}

int expert_int8_linear(int dtype, int64_t m, int64_t n, int64_t k, int64_t groups, const void *X, int64_t ldx,
                       const void *codes, const float *scales, const int *offsets, const float *bias, int activation,
                       void *Y, int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype) || !size_ok(m, 0) || !size_ok(n, 1) || !size_ok(k, 1) || k > kInt8MaxK || !size_ok(groups, 1) ||
        ldx < k || ldy < n || activation < 0 || activation > 2 || (!offsets && groups != 1))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t size = elem(dtype), kp = padded16(k), kpx = padded(k);
    if (ldx * size >= kMaxRowBytes || ldy * size >= kMaxRowBytes) return GEMM_F32_ERR_INVALID_VALUE;
    if ((offsets && !aligned(offsets, 4)) || !here(codes, 16) || !here(scales, 4) || (bias && !aligned(bias, 4)) ||
        (m > 0 && (!here(X, size) || !here(Y, size))))
        return GEMM_F32_ERR_INVALID_VALUE;
    if (!grid_ok(m, n, 16, 16, groups + 2) || !counts_ok(m, groups)) return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t need = expert_int8_workspace(m, k);
    if (need > 0 && !here(workspace, 16)) return GEMM_F32_ERR_INVALID_VALUE;
    if (workspace_bytes < need) return GEMM_F32_ERR_SCRATCH_TOO_SMALL;
    GroupedArgs a{};
    int cus = 0;
    const int st = current_device(&cus, &a.num_xcd);
    if (st != GEMM_F32_SUCCESS) return st;
    if (m == 0) return GEMM_F32_SUCCESS;
    char *const xc = static_cast<char *>(workspace);
    float *const xs = reinterpret_cast<float *>(xc + m * kpx);
    a.A = xc;
    a.B = static_cast<const char *>(codes);
    a.C = static_cast<char *>(Y);
    a.a_scales = reinterpret_cast<const u8 *>(xs);
    a.b_scales = reinterpret_cast<const u8 *>(scales);
    a.bias = bias;
    a.offsets = offsets;
    a.m = (int)m;
    a.n = (int)n;
    a.k = (int)k;
    a.groups = (int)groups;
    a.lda = kpx;
    a.ldb = kp;
    a.ldc = ldy * size;
    a.expert_stride = n * kp;
    a.bias_stride = n;
    a.group_m = 8;
    a.act = activation;
    a.a_kblocks = (int)(kpx / 128);
    const hipStream_t s = stream_of(stream);
    const bool bf16 = dtype == EXPERT_BF16;
    const int64_t rows = mean_rows(m, groups);
    const bool few = few_rows(false, true, rows, n, groups, cus);
    if (few && rows <= 2 && rows * kpx <= kInt8FewValues && (m < 16 ? m : 16) * (kpx + 16) <= kInt8FewBytes) {
        a.A = static_cast<const char *>(X);
        a.lda = ldx * size;
        return launch_int8_few(a, bf16, true, cus, s);
    }
    const int quantised =
        launch_int8_quantize(Int8Args{static_cast<const char *>(X), xc, xs, ldx, (int)m, (int)k, (int)kpx}, bf16, false, s);
    if (quantised != GEMM_F32_SUCCESS) return quantised;
    if (few) return launch_int8_few(a, bf16, false, cus, s);
    const LpCall c{false, bf16, true, false, wide_rows(Y, a.ldc, n, size), cus};
    return launch_int8_tiles(a, c, rows, s);
}

int64_t expert_orthogonalize_workspace(int dtype, int64_t batch, int64_t rows, int64_t cols)
{
    if (!ortho_sizes_ok(dtype, batch, rows, cols) || batch == 0) return 0;
    const OrthoPlan p(batch, rows, cols);
    return p.shares + p.chunk * p.matrix;
}

int expert_orthogonalize(int dtype, int64_t batch, int64_t rows, int64_t cols, const void *X, int64_t ldx,
                         int64_t stride_x, int steps, const float *coefficients, float scale, void *Y, int64_t ldy,
                         int64_t stride_y, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!ortho_sizes_ok(dtype, batch, rows, cols) || ldx < cols || ldy < cols || stride_x < 0 || steps < 1 ||
        steps > kOrthoMaxSteps || !coefficients || !std::isfinite(scale) || !ortho_bounded(coefficients, steps))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t size = elem(dtype);
    if (ldx * size >= kMaxRowBytes || ldy * size >= kMaxRowBytes) return GEMM_F32_ERR_INVALID_VALUE;
    if (batch > 1 && (stride_y < (rows - 1) * ldy + cols)) return GEMM_F32_ERR_INVALID_VALUE;
    if (batch > 0 && (!here(X, size) || !here(Y, size))) return GEMM_F32_ERR_INVALID_VALUE;
    const OrthoPlan p(batch, rows, cols);
    // A launch over the blocks of 64 x 64 holds less than 2^32 threads (256 each).
    constexpr int64_t kMostBlocks = (1 << 24) - 1;
    if (!p.strips && (p.m_pad / 64 > kMostBlocks / (p.n_pad / 64) ||
                      (p.chunk && p.m_pad / 64 * (p.n_pad / 64) > kMostBlocks / p.chunk)))
        return GEMM_F32_ERR_INVALID_VALUE;
    const int64_t need = expert_orthogonalize_workspace(dtype, batch, rows, cols);
    if (need > 0 && !here(workspace, 16)) return GEMM_F32_ERR_INVALID_VALUE;
    if (workspace_bytes < need) return GEMM_F32_ERR_SCRATCH_TOO_SMALL;
    int cus = 0, num_xcd = 0;
    const int st = current_device(&cus, &num_xcd);
    if (st != GEMM_F32_SUCCESS) return st;
    const hipStream_t s = stream_of(stream);
    const bool bf16 = dtype == EXPERT_BF16, turned = rows > cols;
    for (int64_t first = 0; first < batch; first += p.chunk) {
        const int64_t here_ = batch - first < p.chunk ? batch - first : p.chunk;
        char *const x0 = static_cast<char *>(workspace) + p.shares, *const x1 = x0 + p.chunk * 2 * p.x_plane;
        char *const g0 = x1 + p.chunk * 2 * p.x_plane, *const g1 = g0 + p.chunk * 2 * p.g_plane;
        OrthoStartArgs o{};
        o.x = static_cast<const char *>(X) + first * stride_x * size;
        o.ld = ldx;
        o.stride = stride_x;
        o.rows = (int)rows;
        o.cols = (int)cols;
        o.m_pad = (int)p.m_pad;
        o.n_pad = (int)p.n_pad;
        o.turned = turned;
        const int64_t parts = (rows * ((cols + 7) / 8) + 1023) / 1024;       // four chunks of eight a thread, or more
        o.parts = (int)(parts < kOrthoParts ? parts : kOrthoParts);
        o.planes = x0;
        o.plane = p.x_plane;
        o.matrix = 2 * p.x_plane;
        if (p.strips) {
            const int status = ortho_few_rows(p, o, steps, coefficients, scale, bf16, (int)here_,
                                              static_cast<char *>(Y) + first * stride_y * size, ldy, stride_y, s);
            if (status != GEMM_F32_SUCCESS) return status;
            continue;
        }
        o.sums = reinterpret_cast<double *>(g1 + p.chunk * 2 * p.g_plane);
        // bfloat16: X times a power of two is exact in one plane.
        if (bf16) o.factors = reinterpret_cast<float *>(o.sums + p.chunk * kOrthoParts);
        int status = launch_ortho_start(o, bf16, (int)here_, s);
        if (status != GEMM_F32_SUCCESS) return status;

        OrthoArgs gram{};                                                    // A = X X^T
        gram.a_stride = gram.b_stride = 2 * p.x_plane;
        gram.c_stride = 2 * p.g_plane;
        gram.lda = gram.ldb = (int)(p.n_pad * 2);
        gram.a_bytes = gram.b_bytes = 2 * p.x_plane;
        gram.k = (int)p.n_pad;
        gram.rows = gram.cols = (int)p.m_pad;
        gram.group_m = 8;
        gram.batch = (int)here_;
        gram.num_xcd = num_xcd;
        gram.a_low = gram.b_low = p.x_plane;
        gram.a_at = 2;
        gram.C = g0;
        gram.ldc = p.m_pad * 2;
        gram.c_plane = p.g_plane;
        gram.c = kPlaneBack;
        gram.symmetric = 1;
        gram.shares = p.shares ? static_cast<float *>(workspace) : nullptr;

        OrthoArgs poly = gram;                                               // B = a I + b A + c A A
        poly.A = poly.B = poly.G = g0;
        poly.a_stride = poly.b_stride = 2 * p.g_plane;
        poly.lda = poly.ldb = (int)(p.m_pad * 2);
        poly.a_bytes = poly.b_bytes = 2 * p.g_plane;
        poly.k = (int)p.m_pad;
        poly.a_low = poly.b_low = p.g_plane;
        poly.C = g1;
        poly.order = (int)p.m;
        poly.segments = 3;

        OrthoArgs step = poly;                                               // B X
        step.G = nullptr;
        step.symmetric = 0;
        step.A = g1;
        step.b_stride = step.c_stride = 2 * p.x_plane;
        step.ldb = (int)(p.n_pad * 2);
        step.b_bytes = 2 * p.x_plane;
        step.b_low = p.x_plane;
        step.cols = (int)p.n_pad;
        step.ldc = p.n_pad * 2;
        step.c_plane = p.x_plane;
        step.c = kPlaneBack;

        char *now = x0, *then = x1;
        for (int i = 0; i < steps; ++i) {
            const float *const f = coefficients + 3 * i;
            gram.A = gram.B = now;
            gram.factors = step.factors = i == 0 ? o.factors : nullptr;
            // (One plane of X: its product with itself is one pair, B X two.)
            gram.segments = gram.factors ? 1 : 3;
            step.segments = step.factors ? 2 : 3;
            step.a_at = step.factors ? 1 : 2;
            gram.power = 2;
            step.power = 1;
            status = launch_ortho(gram, OrthoCall{kOrthoGram, bf16, true}, cus, s);
            if (status != GEMM_F32_SUCCESS) return status;
            poly.a = f[0] * kPlaneScale;
            poly.b = f[1];
            poly.c = f[2] * kPlaneBack;
            status = launch_ortho(poly, OrthoCall{kOrthoGram, bf16, true}, cus, s);
            if (status != GEMM_F32_SUCCESS) return status;
            if (i + 1 < steps) {
                step.B = now;
                step.C = then;
                status = launch_ortho(step, OrthoCall{kOrthoStep, bf16, true}, cus, s);
                if (status != GEMM_F32_SUCCESS) return status;
                char *const t = now;
                now = then, then = t;
                continue;
            }
            OrthoArgs last = step;
            last.C = static_cast<char *>(Y) + first * stride_y * size;
            last.ldc = ldy * size;
            last.c_stride = stride_y * size;
            last.rows = (int)rows;
            last.cols = (int)cols;
            last.c = kPlaneBack * kPlaneBack;
            last.scale = scale;
            const bool wide = wide_rows(last.C, last.ldc, cols, size) && (here_ == 1 || last.c_stride % 16 == 0);
            if (turned) {
                // X^T B: X is the first operand, along its rows.
                last.A = now;
                last.a_stride = step.b_stride, last.lda = step.ldb, last.a_bytes = step.b_bytes;
                last.B = g1;
                last.b_stride = step.a_stride, last.ldb = step.lda, last.b_bytes = step.a_bytes;
                last.a_low = step.b_low, last.b_low = step.a_low, last.a_at = 3 - step.a_at;
            } else {
                last.B = now;
            }
            status = launch_ortho(last, OrthoCall{turned ? kOrthoTurned : kOrthoLast, bf16, wide}, cus, s);
            if (status != GEMM_F32_SUCCESS) return status;
        }
    }
    return GEMM_F32_SUCCESS;
}

}  // extern "C"
