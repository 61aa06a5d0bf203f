// Orthogonalising a matrix: all its singular values brought near one, its
// singular vectors kept.
//
//   X <- X / |X|,  then in every step  A = X X^T,  X <- (a I + b A + c A A) X
//
// (Newton-Schulz steps of degree five: a singular value s becomes a s + b s^3 +
// c s^5.)  X is m x n with m <= n; of a taller matrix the transposed is taken.
//
// Precision.  The steps multiply what is small in X by up to a each (3.4^5 = 480
// in five), X's roundings among it: with X in bfloat16 between the steps results
// are 1 to 30 % off, in half precision 0.2 to 4 % (the more, the faster the
// singular values fall).  Every matrix is therefore held as two half-precision
// planes, v * 2^11 = hi + lo: 22 bits, and products run on the matrix cores as
// hi hi + hi lo + lo hi, accumulated in 32 bits (v_mfma_f32_32x32x16_f16: three
// times the work of one plane, and still 2.5 times the rate of 32-bit instructions:
// large products reach 1139 TFLOPS in half precision, 153 in 32 bits).  The
// factor 2^11 keeps lo above the subnormals; entries stay below 2^15.9 / 2^11 = 31,
// which the host derives from the coefficients.
// bfloat16 matrices take the same products, for the result is rounded to them once
// (with A and B = a I + b A + c A A in one plane half the products would do, and 26 to
// 30 % of the entries came out a step off the rounded one; 0.2 % do).  In their first
// step X is exact in one plane: A = hi hi^T, one product, B X two.
// Random matrices come out as of 32-bit products (4096 x 4096: 3.5e-6 off in the 2-norm,
// those 4.6e-6); where singular values fall fast 22 bits show: 1000 x 2000 of rank 8 over
// noise of 1e-3 or 1e-5 6.6e-5, 32-bit products 5.2e-5.
//
// A plane is rows of whole 64 columns, rows a multiple of 64, zeros outside the
// matrix; a matrix's planes lie one after the other.  The contraction goes over the
// pairs of planes in turn: to the tile it is one longer contraction.
#pragma once

#include "lp_gemm.hpp"
#include "mx4.hpp"

namespace gemmf32 {

constexpr int kOrthoMaxSteps = 64;
constexpr float kPlaneScale = 2048.0f, kPlaneBack = 1.0f / 2048.0f;

struct OrthoArgs {
    // The product C = A . B (planes): matrix 0's, and bytes from matrix to matrix.
    const char *A, *B;
    long long a_stride, b_stride, c_stride;
    int lda, ldb;                      // bytes from row to row
    long long a_bytes, b_bytes;        // of a matrix's planes
    int segments, k;                   // pairs of planes; contraction of each, whole slabs
    // Where the lo planes lie, and in which pairs they take part: A's in pair
    // a_at, B's in the other one of 1 and 2 (pair 0 is hi hi).
    long long a_low, b_low;
    int a_at;
    int rows, cols;                    // of C
    int tiles_m, tiles_n, group_m, batch, num_xcd;
    // What becomes of the sums.
    char *C;                           // planes, or the result
    long long ldc, c_plane;            // bytes; from hi to lo
    const char *G;                     // A's planes in B = a I + b A + c A A (else NULL)
    int order;                         // rows of the matrix that I has
    float a, b, c;                     // (c: the factor of the sums in every product)
    float scale;                       // of the result, a product of its own: c times a small one is subnormal
    // C is symmetric: the tiles on and below its diagonal are computed, and stored
    // on both sides.
    int symmetric;
    // X / |X| of bfloat16 values is held as X times a power of two, exactly; what is
    // left of 1 / |X|, a factor a matrix, goes to A squared (power 2) and to B X (1).
    const float *factors;              // or NULL
    int power;
    // The pipelined kernel: tiles [0, whole) are a workgroup's each, the others'
    // slabs are shared out evenly (see ortho_pipe.hpp).
    int whole, shared_wgs;
    float *shares;
};

// What the sums of a matrix's product are multiplied by.
__device__ __forceinline__ float ortho_factor(const OrthoArgs &g, int matrix)
{
    if (!g.factors) return g.c;
    const float f = g.factors[matrix];
    return g.power == 2 ? g.c * (f * f) : g.c * f;
}

// Tiles of one matrix, and the place of tile `t`.
__device__ __host__ __forceinline__ int ortho_tiles(const OrthoArgs &g)
{
    return g.symmetric ? g.tiles_m * (g.tiles_m + 1) / 2 : g.tiles_m * g.tiles_n;
}

struct OrthoTile {
    int matrix, tm, tn;
};

// (In scalar registers: the copies' descriptors come from them.)
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoArgs &g, int logical)
{
    const int tiles = ortho_tiles(g), in = logical % tiles;
    int tm, tn;
    if (g.symmetric) {
        // Row by row: tm (tm + 1) / 2 <= in.
        tm = (int)((sqrtf(8.0f * (float)in + 1.0f) - 1.0f) * 0.5f);
        tm += (tm + 1) * (tm + 2) / 2 <= in ? 1 : 0;
        tm -= tm * (tm + 1) / 2 > in ? 1 : 0;
        tn = in - tm * (tm + 1) / 2;
    } else {
        const int width = g.group_m * g.tiles_n, first = in / width * g.group_m;
        const int size = min(g.tiles_m - first, g.group_m);
        tm = first + in % width % size;
        tn = in % width / size;
    }
    return OrthoTile{__builtin_amdgcn_readfirstlane(logical / tiles), __builtin_amdgcn_readfirstlane(tm),
                     __builtin_amdgcn_readfirstlane(tn)};
}

struct OrthoStartArgs {
    const char *x;
    long long ld, stride;              // elements
    int rows, cols;                    // of x
    int m_pad, n_pad;                  // of the planes
    int turned;                        // planes of the transposed
    int parts;
    double *sums;                      // (batch, parts): squares
    float *factors;                    // (batch), or NULL: X / |X| whole, in two planes
    char *planes;
    long long plane, matrix;           // bytes
};

// Sums of squares, in 64 bits: neither leaves the range for any 32-bit values.
// Bound by memory from large matrices on: 16 of 2048 x 4096 in bfloat16 64 us, 4.2 TB/s.
template <class E>
__global__ __launch_bounds__(256) void ortho_squares_kernel(OrthoStartArgs a)
{
    __shared__ double sums[4];
    const int part = blockIdx.x % a.parts, matrix = blockIdx.x / a.parts;
    const E *const x = reinterpret_cast<const E *>(a.x) + matrix * a.stride;
    const int chunks = (a.cols + 7) / 8;
    const long long all = (long long)a.rows * chunks;
    // Four chunks at a time; stepped by row and column, without a division each.
    const long long step = (long long)a.parts * 256, first = (long long)part * 256 + threadIdx.x;
    const int step_row = (int)(step / chunks), step_chunk = (int)(step % chunks);
    int row = (int)(first / chunks), chunk = (int)(first % chunks);
    double sum = 0.0;
    for (long long i = first; i < all; i += 4 * step) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            load8(x + row * a.ld + chunk * 8, i + u * step < all ? a.cols - chunk * 8 : 0, v[u]);
            row += step_row;
            chunk += step_chunk;
            if (chunk >= chunks) chunk -= chunks, ++row;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += (double)v[u][j] * (double)v[u][j];
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) a.sums[blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// A 32-bit number's planes (scaled already).
struct Planes {
    _Float16 hi, lo;

    __device__ __forceinline__ explicit Planes(float t)
    {
        hi = (_Float16)t;
        lo = (_Float16)(t - (float)hi);
    }
};

// x / |x| as planes, a block of 64 x 64 a workgroup; with factors x times a power
// of two, in one.  Bound by memory: 16 of 2048 x 4096 in bfloat16 134 us, 4.0 TB/s read and
// written.
template <class E>
__global__ __launch_bounds__(256) void ortho_start_kernel(OrthoStartArgs a)
{
    __shared__ float block[64][65];
    __shared__ double factor_of;
    const int tiles_n = a.n_pad / 64, tiles = a.m_pad / 64 * tiles_n;
    const int matrix = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int row0 = tile / tiles_n * 64, col0 = tile % tiles_n * 64;
    if (threadIdx.x < 64) {
        double sum = 0.0;
        for (int i = threadIdx.x; i < a.parts; i += 64) sum += a.sums[(long long)matrix * a.parts + i];
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
        if (threadIdx.x == 0) {
            // (A matrix of zeros stays one.)
            double whole = sum == 0.0 ? 0.0 : 1.0 / sqrt(sum);
            if (a.factors) {
                const double power = __builtin_bit_cast(double, __builtin_bit_cast(long long, whole) & 0x7ff0000000000000ll);
                if (tile == 0) a.factors[matrix] = sum == 0.0 ? 0.0f : (float)(whole / power);
                whole = power;
            }
            factor_of = whole * (double)kPlaneScale;
        }
    }
    const E *const x = reinterpret_cast<const E *>(a.x) + matrix * a.stride;
    const int r0 = a.turned ? col0 : row0, c0 = a.turned ? row0 : col0;      // in x
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + (threadIdx.x >> 3) + 32 * i, c = c0 + (threadIdx.x & 7) * 8;
        load8(x + r * a.ld + c, r < a.rows ? a.cols - c : 0, v[i]);
    }
    __syncthreads();
    const double factor = factor_of;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = (threadIdx.x >> 3) + 32 * i, c = (threadIdx.x & 7) * 8 + j;
            const float t = (float)((double)v[i][j] * factor);
            if (a.turned) block[c][r] = t;
            else block[r][c] = t;
        }
    __syncthreads();
    char *const out = a.planes + matrix * a.matrix;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (threadIdx.x >> 3) + 32 * i, c = (threadIdx.x & 7) * 8;
        f16x8 hi, lo;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Planes p(block[r][c + j]);
            hi[j] = p.hi;
            lo[j] = p.lo;
        }
        char *const q = out + ((long long)(row0 + r) * a.n_pad + col0 + c) * 2;
        *reinterpret_cast<f16x8 *>(q) = hi;
        if (!a.factors) *reinterpret_cast<f16x8 *>(q + a.plane) = lo;
    }
}

// Four lanes' four halves each, turned: of the lanes' halves number lane % 4.
__device__ __forceinline__ u32x2 turn4(unsigned p01, unsigned p23, int lane)
{
    // (All lanes take part in each exchange: none of them behind a condition.)
    unsigned x[4] = {mx_lane<0x00>(p01), mx_lane<0x55>(p01), mx_lane<0xaa>(p01), mx_lane<0xff>(p01)};
    const unsigned y[4] = {mx_lane<0x00>(p23), mx_lane<0x55>(p23), mx_lane<0xaa>(p23), mx_lane<0xff>(p23)};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = lane & 2 ? y[k] : x[k];
    const unsigned pick = lane & 1 ? 0x07060302u : 0x05040100u;
    return u32x2{__builtin_amdgcn_perm(x[1], x[0], pick), __builtin_amdgcn_perm(x[3], x[2], pick)};
}

// A 32 x 32 block of the sums as planes, in runs of eight columns.  G: a I + b G +
// c sums.  mirror: also at the place across the diagonal, where the lane's values
// are a column: four lanes turn theirs, for runs of four.
__device__ __forceinline__ void ortho_block(const OrthoArgs &g, int matrix, int row0, int col0, int lane, const f32x16 &acc,
                                            bool mirror)
{
    const int l32 = lane & 31, half = lane >> 5, row = row0 + l32;
    const float factor = ortho_factor(g, matrix);
    f16x8 plane[2][2];
#pragma unroll
    for (int v0 = 0; v0 < 16; v0 += 8) {
        const int col = col0 + half * 8 + v0 * 2;
        const long long at = row * g.ldc + (long long)col * 2;
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = acc[v0 + i] * factor;
        if (g.G) {
            const char *const p = g.G + matrix * g.c_stride + at;
            const f16x8 hi = *reinterpret_cast<const f16x8 *>(p);
            const f16x8 lo = *reinterpret_cast<const f16x8 *>(p + g.c_plane);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[i] += g.b * ((float)hi[i] + (float)lo[i]);
                if (col + i == row && row < g.order) t[i] += g.a;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Planes p(t[i]);
            plane[v0 / 8][0][i] = p.hi;
            plane[v0 / 8][1][i] = p.lo;
        }
        if (mirror)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                char *const q = g.C + matrix * g.c_stride + j * g.c_plane;
                const u32x4 w = __builtin_bit_cast(u32x4, plane[v0 / 8][j]);
                const long long across = (long long)(row0 + (l32 & ~3)) * 2;
                *reinterpret_cast<u32x2 *>(q + (col + (lane & 3)) * g.ldc + across) = turn4(w.x, w.y, lane);
                *reinterpret_cast<u32x2 *>(q + (col + 4 + (lane & 3)) * g.ldc + across) = turn4(w.z, w.w, lane);
            }
    }
    // Lanes 16 to 31 and 48 to 63 hand their first runs over for the second ones of
    // those 16 below: a store then writes 64 bytes of 16 rows.  (32 bytes of 32 rows:
    // lines leave the L2 half written, 787 MiB instead of 660 for 512 of planes of 16
    // matrices of 2048 x 4096; joining 4096 x 4096 took 44 us instead of 39.)
    const long long to = (row0 + (lane & 15)) * g.ldc + (long long)(col0 + half * 8 + (lane & 16)) * 2;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        char *const q = g.C + matrix * g.c_stride + j * g.c_plane;
        u32x4 x = __builtin_bit_cast(u32x4, plane[0][j]), y = __builtin_bit_cast(u32x4, plane[1][j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto pair = __builtin_amdgcn_permlane16_swap(x[i], y[i], false, false);
            x[i] = pair[0], y[i] = pair[1];
        }
        *reinterpret_cast<u32x4 *>(q + to) = x;
        *reinterpret_cast<u32x4 *>(q + to + 16 * g.ldc) = y;
    }
}

// The tile's.
template <class T>
__device__ __forceinline__ void ortho_store(const OrthoArgs &g, const OrthoTile &t, int wr, int wc, int lane,
                                            f32x16 (&acc)[T::MB][T::NB])
{
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) {
            const int row0 = t.tm * T::BM + wr * T::WM + mb * 32, col0 = t.tn * T::BN + wc * T::WN + nb * 32;
            if (row0 < g.rows && col0 < g.cols) ortho_block(g, t.matrix, row0, col0, lane, acc[mb][nb], g.symmetric && t.tm != t.tn);
        }
}

// A workgroup a tile.  E: what C holds, planes (_Float16) or the result's type.
// K: parts of the workgroup that share the slabs, each with a ring of its own; their
// sums meet in LDS.  A part of four wavefronts, one a SIMD, waits most of a slab for
// LDS and its own products.  X X^T of 1088 x 5056 in one pair of planes, 153 tiles of 64 x 64
// (one MI355X): 25 us in two parts, 32 in one (0.24 and 0.19 PFLOPS): the ring of a tile alone on
// its CU runs at the latency of its slabs.  In three pairs 64 in two parts.
template <class T, int K, bool A_KS, bool B_KS, class E, bool WIDE>
__global__ __launch_bounds__(T::THREADS * K) void ortho_kernel(OrthoArgs g)
{
    __shared__ i32x4 lds[K * T::STAGES * T::stage_chunks(kF16)];
    const int part = K > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / T::THREADS) : 0;
    const int tid = threadIdx.x % T::THREADS, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % T::WAVES_M, wc = wave / T::WAVES_M;
    const OrthoTile t = ortho_tile(g, xcd_contiguous(blockIdx.x, ortho_tiles(g) * g.batch, g.num_xcd));
    const int matrix = t.matrix, row = t.tm * T::BM, col = t.tn * T::BN;
    LpProblem q{};
    const long long skip_a = A_KS ? (long long)row * 2 : (long long)row * g.lda;
    const long long skip_b = B_KS ? (long long)col * 2 : (long long)col * g.ldb;
    q.a = {g.A + matrix * g.a_stride + skip_a, g.a_bytes - skip_a, g.lda, g.rows - row};
    q.b = {g.B + matrix * g.b_stride + skip_b, g.b_bytes - skip_b, g.ldb, g.cols - col};
    q.k = g.segments * g.k;
    q.segment = g.k / 64;
    q.a_second = g.a_at == 1 ? g.a_low : 0, q.a_third = g.a_at == 2 ? g.a_low : 0;
    q.b_second = g.a_at == 2 ? g.b_low : 0, q.b_third = g.a_at == 1 ? g.b_low : 0;
    q.share = K;
    q.turn = part;
    f32x16 acc[T::MB][T::NB];
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
    LpLoop<T, kF16, A_KS, B_KS, 16 / sizeof(E)> loop{q, lds + part * T::STAGES * T::stage_chunks(kF16), tid, lane, wave, wr, wc};
    loop.run(acc);
    if constexpr (K > 1) {
        constexpr int SUMS = T::MB * T::NB * 4;              // of four, a lane
        static_assert((K - 1) * T::THREADS * SUMS <= K * T::STAGES * T::stage_chunks(kF16), "the sums fit the rings");
        f32x4 *const sums = reinterpret_cast<f32x4 *>(lds) + tid;
        __syncthreads();
        if (part > 0)
#pragma unroll
            for (int i = 0; i < SUMS; ++i) {
                const f32x16 &x = acc[i / 4 / T::NB][i / 4 % T::NB];
                sums[((part - 1) * SUMS + i) * T::THREADS] = f32x4{x[i % 4 * 4], x[i % 4 * 4 + 1], x[i % 4 * 4 + 2], x[i % 4 * 4 + 3]};
            }
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int p = 0; p < K - 1; ++p)
#pragma unroll
            for (int i = 0; i < SUMS; ++i) {
                const f32x4 x = sums[(p * SUMS + i) * T::THREADS];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i / 4 / T::NB][i / 4 % T::NB][i % 4 * 4 + j] += x[j];
            }
    }
    if constexpr (__is_same(E, _Float16)) {
        ortho_store<T>(g, t, wr, wc, lane, acc);
    } else {
        const float factor = ortho_factor(g, matrix);
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = acc[mb][nb] * factor * g.scale;
        lp_store<T, E, WIDE>(g.C + matrix * g.c_stride + row * g.ldc + (long long)col * sizeof(E), g.ldc, g.rows - row,
                             g.cols - col, nullptr, 0, wr, wc, lane, acc);
    }
}

}  // namespace gemmf32
