// C entry points of include/expert_ops.h: argument checks, the choice of a
// kernel, and its launch.  No kernel is compiled in this unit.
#include "expert_ops.h"

#include "expert_launch.hpp"
#include "mx4.hpp"
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

}  // extern "C"
