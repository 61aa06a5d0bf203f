// 8-bit products where an expert has few rows (decoding): bound by the bytes of
// the experts' codes, each read once.
//
// A workgroup takes 16 rows of one expert and a strip of columns, KW of its
// wavefronts split k, as in grouped_few.hpp, and CW of them the strip (short k: a
// workgroup has to have work for all).  Codes go straight from memory into
// registers, 16 bytes a lane, one iteration's loads ahead of the products
// (v_mfma_i32_16x16x64_i8: four lanes share a column's 64 bytes).  The
// wavefronts' sums meet in LDS as integers: any order gives the same bits.
//
// QUANTISE: the workgroup takes the rows of X themselves and quantises them for
// itself into LDS, while its first loads of B are under way: one launch instead of
// two, for the same work in every strip's workgroup.
//
// One MI355X: 16 rows through eight experts of 14336 x 4096, two each on average, 72 us
// (5.7 TB/s of the codes that are read), 5 of quantisation before; 4 rows through one,
// partly from the last level of cache, 12.9 and 3.8.
#pragma once

#include "int8.hpp"
#include "lp_gemm.hpp"

namespace gemmf32 {

template <class X, int KW_, int CW_, int NB_>
struct Int8FewTile {
    using E = X;
    static constexpr int KW = KW_, CW = CW_, WAVES = KW * CW, THREADS = WAVES * 64, NB = NB_;
    static constexpr int BM = 16, WN = 16 * NB, BN = WN * CW, KI = 256;       // k of an iteration
};

template <class T>
struct Int8FewRegs {
    i32x4 a[4], b[4 * T::NB];
};

// Bytes from row to row of the codes in LDS: rows on different banks.
constexpr int int8_few_row(int kp) { return kp + 16; }

// The rows' codes to LDS, four rows at a time; their scales.
template <class T>
__device__ __forceinline__ void int8_few_quantise(const GroupedArgs &g, int row0, int rows, char *codes, float *scales,
                                                  unsigned (*tops)[4])
{
    using E = typename T::E;
    const int tid = threadIdx.x, kp = g.a_kblocks * 128, step = T::THREADS * 8;
    for (int r0 = 0; r0 < rows; r0 += 4) {
        Mx8<E> x[4];                                     // the thread's first eight values of each row
        unsigned largest[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const E *const p = reinterpret_cast<const E *>(g.A + (row0 + min(r0 + i, rows - 1)) * g.lda);
            x[i].load(p + tid * 8, g.k - tid * 8);
            largest[i] = x[i].largest();
            for (int c = tid * 8 + step; c < g.k; c += step) {
                Mx8<E> y;
                y.load(p + c, g.k - c);
                largest[i] = max(largest[i], y.largest());
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            largest[i] = wave_largest(largest[i]);
            if ((tid & 63) == 0) tops[tid >> 6][i] = largest[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (r0 + i >= rows) break;
            unsigned top = 0;
#pragma unroll
            for (int w = 0; w < T::WAVES; ++w) top = max(top, tops[w][i]);
            const Int8Row q(top);
            const E *const p = reinterpret_cast<const E *>(g.A + (row0 + r0 + i) * g.lda);
            char *const out = codes + (r0 + i) * int8_few_row(kp);
            for (int c = tid * 8; c < kp; c += step) {
                Mx8<E> y = x[i];
                if (c >= step) y.load(p + c, g.k - c);
                float v[8];
                y.values(v);
                *reinterpret_cast<u32x2 *>(out + c) = u32x2{pack4(q.code(v[0]), q.code(v[1]), q.code(v[2]), q.code(v[3])),
                                                            pack4(q.code(v[4]), q.code(v[5]), q.code(v[6]), q.code(v[7]))};
            }
            if (tid == 0) scales[r0 + i] = q.scale;
        }
        __syncthreads();
    }
}

template <class T, bool QUANTISE>
__global__ __launch_bounds__(T::THREADS) void int8_few_kernel(GroupedArgs g)
{
    using E = typename T::E;
    constexpr int BM = T::BM, BN = T::BN, ROW = BN + 4;
    __shared__ int red[T::KW][BM * ROW];
    __shared__ float row_scales[BM];
    __shared__ unsigned tops[T::WAVES][4];
    extern __shared__ i32x4 codes_lds[];
    char *const codes = reinterpret_cast<char *>(codes_lds);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    RowTile rt;
    int tn;
    if (!find_tile<BM>(g, blockIdx.x, lane, rt, tn)) return;
    const int col0 = tn * BN;
    const int l16 = lane & 15, grp = lane >> 4;
    const int rows = min(rt.rows, BM);
    const int kw = wave % T::KW, strip = wave / T::KW * T::WN;       // the wavefront's part of k, and of the columns
    // What the thread's first result is scaled by, loaded ahead of all else.
    const float *const sa = reinterpret_cast<const float *>(g.a_scales) + rt.row;
    const float *const sb = reinterpret_cast<const float *>(g.b_scales) + (long long)max(rt.expert, 0) * g.n + col0;
    const float *const bias = g.bias && rt.expert >= 0 ? g.bias + rt.expert * g.bias_stride + col0 : nullptr;
    const int first_col = min(tid % BN, g.n - 1 - col0);
    const float sb_first = sb[first_col], bias_first = bias ? bias[first_col] : 0.0f;
    float sa_first = 0.0f;
    if constexpr (!QUANTISE) sa_first = sa[min(tid / BN, rows - 1)];
    i32x4 acc[T::NB];
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) acc[nb] = i32x4{};
    if (rt.expert >= 0) {
        const char *const pa = QUANTISE ? codes + min(l16, rows - 1) * int8_few_row(g.a_kblocks * 128) + grp * 16
                                        : g.A + (rt.row + min(l16, rows - 1)) * g.lda + grp * 16;
        const char *const bx = g.B + rt.expert * g.expert_stride + grp * 16;
        const char *pb[T::NB];
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) pb[nb] = bx + min(col0 + strip + nb * 16 + l16, g.n - 1) * g.ldb;
        const int held = (int)g.ldb - grp * 16;               // bytes of B's rows from this lane's first on
        const int kp = g.a_kblocks * 128;                     // of A's rows
        auto load_a = [&](int it, Int8FewRegs<T> &r) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k0 = it * T::KI + s * 64;
                r.a[s] = k0 < kp ? *reinterpret_cast<const i32x4 *>(pa + k0) : i32x4{};
            }
        };
        auto load = [&](int it, Int8FewRegs<T> &r) {
            if constexpr (!QUANTISE) load_a(it, r);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k0 = it * T::KI + s * 64;
#pragma unroll
                for (int nb = 0; nb < T::NB; ++nb)
                    r.b[s * T::NB + nb] = k0 < held ? *reinterpret_cast<const i32x4 *>(pb[nb] + k0) : i32x4{};
            }
        };
        auto multiply = [&](const Int8FewRegs<T> &r) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int nb = 0; nb < T::NB; ++nb)
                    acc[nb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(r.b[s * T::NB + nb], r.a[s], acc[nb], 0, 0, 0);
        };
        const int its = (g.k + T::KI - 1) / T::KI;
        Int8FewRegs<T> r[2];
        if (kw < its) load(kw, r[0]);
        if constexpr (QUANTISE) {
            if (kw + T::KW < its) load(kw + T::KW, r[1]);
            int8_few_quantise<T>(g, rt.row, rows, codes, row_scales, tops);
        }
        int it = kw;
        while (it < its) {
            if (it + T::KW < its && !(QUANTISE && it == kw)) load(it + T::KW, r[1]);
            if constexpr (QUANTISE) load_a(it, r[0]);
            multiply(r[0]);
            it += T::KW;
            if (it >= its) continue;
            if (it + T::KW < its) load(it + T::KW, r[0]);
            if constexpr (QUANTISE) load_a(it, r[1]);
            multiply(r[1]);
            it += T::KW;
        }
    }
    // Lane (l16, grp) holds row l16 and columns 4 grp + v of each block.
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[kw][l16 * ROW + strip + nb * 16 + 4 * grp + v] = acc[nb][v];
    __syncthreads();
    for (int e = tid; e < rows * BN; e += T::THREADS) {
        const int row = e / BN, col = e % BN;
        if (col0 + col >= g.n) continue;
        int sum = 0;
#pragma unroll
        for (int w = 0; w < T::KW; ++w) sum += red[w][row * ROW + col];
        float x = 0.0f;
        if (rt.expert >= 0) {
            const bool first = e == tid;
            x = (float)sum * (QUANTISE ? row_scales[row] : first ? sa_first : sa[row]) * (first ? sb_first : sb[col]);
            if (bias) x += first ? bias_first : bias[col];
            x = activate(x, g.act);
        }
        *(reinterpret_cast<E *>(g.C + (rt.row + row) * g.ldc) + col0 + col) = (E)x;
    }
}

}  // namespace gemmf32
