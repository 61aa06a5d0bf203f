// Orthogonalising matrices of up to 64 or 128 rows (their smaller side): bound by
// launches and latency, so few of them.
//
// A workgroup holds all rows and a strip of S x 64 columns of one matrix in LDS,
// as planes (see orthogonal.hpp), ROWS (64 or 128) rows in blocks of 64 columns.  A matrix of
// one strip is done in one launch.  Of a longer one each strip is a workgroup's:
// one launch for X / |X| and the strips' shares of X X^T, then one launch a step,
// in which every workgroup adds the shares up (in the order of the strips: the
// same bits in every run), squares A for itself, updates its strip and writes its
// share of the next X X^T.
//
// Products run on hi hi + hi lo + lo hi in both types: three times little.
//
// One MI355X: four matrices of 64 x 192, five steps, one launch of 25.6 us, 4 of them a step
// and barrier after barrier (fifteen products of few instructions that wait for each
// other through LDS); as tiles, 17 launches, 82.
// LDS: row r of a block, 16-byte chunk c at [r][c ^ (r / 2) % 8], as the tiles have
// it; X is read along its columns (X X^T) as it is, along its rows (B X) by the
// transposing read.
#pragma once

#include "orthogonal.hpp"

namespace gemmf32 {

constexpr int strip_chunks(int rows) { return rows * 8; }       // of a plane's block of 64 columns

struct OrthoStripArgs {
    OrthoStartArgs start;              // x, its sums of squares (several strips), its shape; planes
    char *planes_out;                  // several strips: the next X
    const float *shares;               // (batch, strips, ROWS, ROWS): of X X^T, and of the next one
    float *shares_out;
    int strips, steps;
    int order, width;                  // rows of X, columns
    float f[3 * kOrthoMaxSteps];       // coefficients of the launch's steps
    float scale;
    char *y;
    long long ldy, stride_y;           // elements
};

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int block_chunk(int row, int chunk) { return row * 8 + (chunk ^ ((row >> 1) & 7)); }

// 16 x 16 block (br, bc) of P P^T, P planes of BLOCKS blocks of CHUNKS chunks (lo
// after all of hi).  Lane (l16, grp) gets row l16, columns 4 grp ...
template <int BLOCKS, int CHUNKS>
__device__ __forceinline__ f32x4 strip_gram(const i32x4 *p, int br, int bc, int lane)
{
    const int l16 = lane & 15, grp = lane >> 4;
    // (Three chains: a product waits for the one before it in its own.)
    f32x4 acc = {}, al_bh = {}, ah_bl = {};
    constexpr int LO = CHUNKS * BLOCKS;
#pragma unroll
    for (int s = 0; s < BLOCKS; ++s) {
        if (BLOCKS > 3) __builtin_amdgcn_sched_barrier(0);       // (else more reads at a time than registers)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int at = s * CHUNKS + block_chunk(br * 16 + l16, k * 4 + grp);
            const int bt = s * CHUNKS + block_chunk(bc * 16 + l16, k * 4 + grp);
            const f16x8 ah = __builtin_bit_cast(f16x8, p[at]), al = __builtin_bit_cast(f16x8, p[at + LO]);
            const f16x8 bh = __builtin_bit_cast(f16x8, p[bt]), bl = __builtin_bit_cast(f16x8, p[bt + LO]);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(bh, ah, acc, 0, 0, 0);
            ah_bl = __builtin_amdgcn_mfma_f32_16x16x32_f16(bl, ah, ah_bl, 0, 0, 0);
            al_bh = __builtin_amdgcn_mfma_f32_16x16x32_f16(bh, al, al_bh, 0, 0, 0);
        }
    }
    return acc + (ah_bl + al_bh);
}

// Four values of row `row` from column `col` on, as planes of BLOCKS blocks.
template <int BLOCKS, int CHUNKS>
__device__ __forceinline__ void put_planes(i32x4 *planes, int row, int col, const float (&t)[4])
{
    f16x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Planes p(t[i]);
        hi[i] = p.hi;
        lo[i] = p.lo;
    }
    char *const q = reinterpret_cast<char *>(planes + col / 64 * CHUNKS + block_chunk(row, col % 64 / 8)) + (col & 7) * 2;
    *reinterpret_cast<f16x4 *>(q) = hi;
    *reinterpret_cast<f16x4 *>(q + BLOCKS * CHUNKS * 16) = lo;
}

// SHARED: a strip of several.  FIRST (SHARED): X / |X| and its share.
template <class E, int ROWS, int S, int WAVES, bool SHARED, bool FIRST>
__global__ __launch_bounds__(WAVES * 64) void ortho_strip_kernel(OrthoStripArgs g)
{
    constexpr int THREADS = WAVES * 64, COLS = S * 64, SIDE = ROWS / 16, CHUNKS = strip_chunks(ROWS);
    constexpr int R = ROWS / 64;                                // blocks of A's and B's planes
    constexpr int BLOCKS = SIDE * 4 * S / WAVES;                // 16 x 16 blocks of X a wavefront
    constexpr int SQUARE = SIDE * SIDE / WAVES;                 // and of A and B
    static_assert(BLOCKS * WAVES == SIDE * 4 * S && SQUARE * WAVES == SIDE * SIDE, "whole blocks");
    // 128 rows: B takes A's place, for both would not fit.
    constexpr bool IN_PLACE = ROWS > 64;
    __shared__ i32x4 xs[2 * S * CHUNKS];
    __shared__ i32x4 as[FIRST ? 1 : 2 * R * CHUNKS], bs_own[FIRST || IN_PLACE ? 1 : 2 * R * CHUNKS];
    i32x4 *const bs = IN_PLACE ? as : bs_own;
    __shared__ double sums[WAVES];
    const int tid = threadIdx.x, lane_of = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int matrix = SHARED ? blockIdx.x / g.strips : blockIdx.x, strip = SHARED ? blockIdx.x % g.strips : 0;
    const int col0 = strip * COLS;
    const OrthoStartArgs &a = g.start;

    if constexpr (SHARED && !FIRST) {
        // This strip's planes.
        for (int i = tid; i < S * CHUNKS; i += THREADS) {
            const int row = i / (S * 8), chunk = i % (S * 8);
            const char *const p = a.planes + matrix * a.matrix + ((long long)row * a.n_pad + col0 + chunk * 8) * 2;
            const bool in = col0 + chunk * 8 < a.n_pad;
            i32x4 *const q = xs + chunk / 8 * CHUNKS + block_chunk(row, chunk % 8);
            q[0] = in ? *reinterpret_cast<const i32x4 *>(p) : i32x4{};
            q[S * CHUNKS] = in ? *reinterpret_cast<const i32x4 *>(p + a.plane) : i32x4{};
        }
    } else {
        // Chunks of eight values of x, along its rows, in registers until |x| is known.
        constexpr int ALL = ROWS * COLS / 8, EACH = (ALL + THREADS - 1) / THREADS;
        const E *const x = reinterpret_cast<const E *>(a.x) + matrix * a.stride;
        float v[EACH][8];
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int at = tid + i * THREADS;
            // (turned: x's rows are the columns here)
            const int line = a.turned ? col0 + at / (ROWS / 8) : at / (S * 8), chunk = a.turned ? at % (ROWS / 8) : at % (S * 8);
            const int first = a.turned ? chunk * 8 : col0 + chunk * 8;
            load8(x + line * a.ld + first, line < a.rows && (ALL % THREADS == 0 || at < ALL) ? a.cols - first : 0, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += (double)v[i][j] * (double)v[i][j];
        }
        if constexpr (SHARED) {
            sum = 0.0;
            for (int i = lane_of; i < a.parts; i += 64) sum += a.sums[(long long)matrix * a.parts + i];
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
        if constexpr (!SHARED) {
            if (lane_of == 0) sums[wave] = sum;
            __syncthreads();
            sum = 0.0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) sum += sums[w];
        }
        const double factor = sum == 0.0 ? 0.0 : (double)kPlaneScale / sqrt(sum);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int at = tid + i * THREADS;
            if (ALL % THREADS && at >= ALL) continue;
            f16x8 hi, lo;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Planes p((float)((double)v[i][j] * factor));
                hi[j] = p.hi;
                lo[j] = p.lo;
            }
            if (a.turned) {
                const int c = at / (ROWS / 8), r0 = at % (ROWS / 8) * 8;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    char *const q = reinterpret_cast<char *>(xs + c / 64 * CHUNKS + block_chunk(r0 + j, c % 64 / 8)) + (c & 7) * 2;
                    *reinterpret_cast<_Float16 *>(q) = hi[j];
                    *reinterpret_cast<_Float16 *>(q + S * CHUNKS * 16) = lo[j];
                }
            } else {
                const int row = at / (S * 8), chunk = at % (S * 8);
                i32x4 *const q = xs + chunk / 8 * CHUNKS + block_chunk(row, chunk % 8);
                q[0] = __builtin_bit_cast(i32x4, hi);
                q[S * CHUNKS] = __builtin_bit_cast(i32x4, lo);
                if constexpr (FIRST) {
                    char *const p = g.planes_out + matrix * a.matrix + ((long long)row * a.n_pad + col0 + chunk * 8) * 2;
                    if (col0 + chunk * 8 < a.n_pad) {
                        *reinterpret_cast<f16x8 *>(p) = hi;
                        *reinterpret_cast<f16x8 *>(p + a.plane) = lo;
                    }
                }
            }
        }
        if (FIRST && a.turned) {
            __syncthreads();
            for (int i = tid; i < S * CHUNKS; i += THREADS) {
                const int row = i / (S * 8), chunk = i % (S * 8);
                char *const p = g.planes_out + matrix * a.matrix + ((long long)row * a.n_pad + col0 + chunk * 8) * 2;
                const i32x4 *const q = xs + chunk / 8 * CHUNKS + block_chunk(row, chunk % 8);
                if (col0 + chunk * 8 < a.n_pad) {
                    *reinterpret_cast<i32x4 *>(p) = q[0];
                    *reinterpret_cast<i32x4 *>(p + a.plane) = q[S * CHUNKS];
                }
            }
        }
    }

    // The strip's share of X X^T.
    auto share = [&](float *out) {
        const int l16 = lane_of & 15, grp = lane_of >> 4;
#pragma unroll
        for (int j = 0; j < SQUARE; ++j) {
            const int b = wave + j * WAVES;
            const f32x4 t = strip_gram<S, CHUNKS>(xs, b / SIDE, b % SIDE, lane_of);
            *reinterpret_cast<f32x4 *>(out + (b / SIDE * 16 + l16) * ROWS + b % SIDE * 16 + 4 * grp) = t;
        }
    };
    const long long share_at = ((long long)matrix * g.strips + strip) * (ROWS * ROWS);
    if constexpr (FIRST) {
        __syncthreads();
        share(g.shares_out + share_at);
        return;
    } else {
        const int steps = SHARED ? 1 : g.steps;
        for (int step = 0; step < steps; ++step) {
            // (Opaque, once a step: all blocks' places would else be held in registers
            // through all steps.)
            int lane = lane_of, l16 = lane & 15, grp = lane >> 4;
            asm volatile("" : "+v"(lane), "+v"(l16), "+v"(grp));
            const float fa = g.f[3 * step], fb = g.f[3 * step + 1], fc = g.f[3 * step + 2];
            // A, scaled once.
            if constexpr (SHARED) {
                for (int i = tid; i < ROWS * ROWS / 4; i += THREADS) {
                    const float *const p = g.shares + (long long)matrix * g.strips * (ROWS * ROWS) + i * 4;
                    f32x4 t = {};
                    for (int s0 = 0; s0 < g.strips; s0 += 4) {
                        f32x4 u[4];
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            u[s] = s0 + s < g.strips ? *reinterpret_cast<const f32x4 *>(p + (long long)(s0 + s) * (ROWS * ROWS)) : f32x4{};
#pragma unroll
                        for (int s = 0; s < 4; ++s) t += u[s];
                    }
                    const float w[4] = {t[0] * kPlaneBack, t[1] * kPlaneBack, t[2] * kPlaneBack, t[3] * kPlaneBack};
                    put_planes<R, CHUNKS>(as, i / (ROWS / 4), i % (ROWS / 4) * 4, w);
                }
            } else {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < SQUARE; ++j) {
                    const int b = wave + j * WAVES;
                    const f32x4 t = strip_gram<S, CHUNKS>(xs, b / SIDE, b % SIDE, lane);
                    const float w[4] = {t[0] * kPlaneBack, t[1] * kPlaneBack, t[2] * kPlaneBack, t[3] * kPlaneBack};
                    put_planes<R, CHUNKS>(as, b / SIDE * 16 + l16, b % SIDE * 16 + 4 * grp, w);
                }
            }
            __syncthreads();
            // B = a I + b A + c A A.
            float w[SQUARE][4];
#pragma unroll
            for (int j = 0; j < SQUARE; ++j) {
                const int b = wave + j * WAVES;
                const f32x4 t = strip_gram<R, CHUNKS>(as, b / SIDE, b % SIDE, lane);
                const int row = b / SIDE * 16 + l16, col = b % SIDE * 16 + 4 * grp;
                const char *const q = reinterpret_cast<const char *>(as + col / 64 * CHUNKS + block_chunk(row, col % 64 / 8)) + (col & 7) * 2;
                const f16x4 hi = *reinterpret_cast<const f16x4 *>(q), lo = *reinterpret_cast<const f16x4 *>(q + R * CHUNKS * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[j][i] = fc * kPlaneBack * t[i] + fb * ((float)hi[i] + (float)lo[i]);
                    if (col + i == row && row < g.order) w[j][i] += fa * kPlaneScale;
                }
            }
            if (IN_PLACE) __syncthreads();
#pragma unroll
            for (int j = 0; j < SQUARE; ++j) {
                const int b = wave + j * WAVES;
                put_planes<R, CHUNKS>(bs, b / SIDE * 16 + l16, b % SIDE * 16 + 4 * grp, w[j]);
            }
            __syncthreads();
            // B X: blocks of 16 rows and 16 columns.
            f32x4 acc[BLOCKS];
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j) {
                const int b = wave + j * WAVES, br = b % SIDE, bc = b / SIDE;
                f32x4 al_bh = {}, ah_bl = {};
                acc[j] = f32x4{};
                const i32x4 *const block = xs + bc / 4 * CHUNKS;
                const int col = bc % 4 * 16 + (lane & 3) * 4;
                // Eight k-rows of the lane's column, by two transposing reads.
                auto turned = [&](const i32x4 *plane, int k) {
                    const int kr = 32 * k + 8 * grp + (l16 >> 2);
                    const char *const q0 = reinterpret_cast<const char *>(plane + block_chunk(kr, col / 8)) + (col & 7) * 2;
                    const char *const q1 = reinterpret_cast<const char *>(plane + block_chunk(kr + 4, col / 8)) + (col & 7) * 2;
                    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)q0));
                    const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)q1));
                    return __builtin_bit_cast(f16x8, (i32x4){(int)x.x, (int)x.y, (int)y.x, (int)y.y});
                };
#pragma unroll
                for (int k = 0; k < 2 * R; ++k) {
                    const int at = k / 2 * CHUNKS + block_chunk(br * 16 + l16, 4 * (k % 2) + grp);
                    const f16x8 bh = __builtin_bit_cast(f16x8, bs[at]), bl = __builtin_bit_cast(f16x8, bs[at + R * CHUNKS]);
                    const f16x8 xh = turned(block, k), xl = turned(block + S * CHUNKS, k);
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xh, bh, acc[j], 0, 0, 0);
                    ah_bl = __builtin_amdgcn_mfma_f32_16x16x32_f16(xl, bh, ah_bl, 0, 0, 0);
                    al_bh = __builtin_amdgcn_mfma_f32_16x16x32_f16(xh, bl, al_bh, 0, 0, 0);
                }
                acc[j] += ah_bl + al_bh;
                // (More blocks' reads at a time would not fit the registers.)
                if (BLOCKS > 3) __builtin_amdgcn_sched_barrier(0);
            }
            __syncthreads();
            const bool last = SHARED ? g.y != nullptr : step + 1 == steps;
            // The lane holds row l16 of each block, columns 4 grp ...
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j) {
                const int b = wave + j * WAVES, row = b % SIDE * 16 + l16, c = b / SIDE * 16 + 4 * grp;
                if (last) {
                    E *const y = reinterpret_cast<E *>(g.y) + matrix * g.stride_y;
                    struct __attribute__((packed, aligned(sizeof(E)))) Run {
                        E e[4];
                    } t;
#pragma unroll
                    for (int i = 0; i < 4; ++i) t.e[i] = (E)(acc[j][i] * (kPlaneBack * kPlaneBack) * g.scale);
                    if (row >= g.order) continue;
                    if (!a.turned && col0 + c + 4 <= g.width) {
                        *reinterpret_cast<Run *>(y + row * g.ldy + col0 + c) = t;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (col0 + c + i < g.width)
                                y[a.turned ? (col0 + c + i) * g.ldy + row : row * g.ldy + col0 + c + i] = t.e[i];
                    }
                } else {
                    f16x4 hi, lo;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const Planes p(acc[j][i] * kPlaneBack);
                        hi[i] = p.hi;
                        lo[i] = p.lo;
                    }
                    char *const q = reinterpret_cast<char *>(xs + c / 64 * CHUNKS + block_chunk(row, c % 64 / 8)) + (c & 7) * 2;
                    *reinterpret_cast<f16x4 *>(q) = hi;
                    *reinterpret_cast<f16x4 *>(q + S * CHUNKS * 16) = lo;
                    if constexpr (SHARED) {
                        char *const p = g.planes_out + matrix * a.matrix + ((long long)row * a.n_pad + col0 + c) * 2;
                        if (col0 + c < a.n_pad) {
                            *reinterpret_cast<f16x4 *>(p) = hi;
                            *reinterpret_cast<f16x4 *>(p + a.plane) = lo;
                        }
                    }
                }
            }
            if (SHARED && !last) {
                __syncthreads();
                share(g.shares_out + share_at);
            }
        }
    }
}

}  // namespace gemmf32
