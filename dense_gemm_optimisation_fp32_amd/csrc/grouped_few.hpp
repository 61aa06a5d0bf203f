// Products grouped by expert where an expert has few rows (decoding): bound
// by the bytes of the experts' matrices, each read once.
//
// A workgroup takes 16 rows of one expert and a strip of columns, and its
// wavefronts split k.  A and B go straight from memory into registers, 16
// bytes a lane, one iteration's loads ahead of the products; the products run
// on 16-row matrix instructions whose rows past the expert's are wasted,
// which costs nothing that the memory does not cover.  The order of k inside
// an instruction is free as long as A and B agree, which the layouts use:
//   k contiguous  a lane holds 16 bytes of one column: four neighbouring k
//                 (32 bits), eight (bfloat16) or a block of 32 (4-bit).  Four
//                 lanes share a column, so an iteration's four loads cover
//                 256 bytes of each column.
//   k strided     32 bits: a lane's 16 bytes are four columns of one k, and
//                 load s of lane group g takes k-row 4 g + s; bfloat16: eight
//                 columns of k-row 8 g + j, turned by one byte permute a
//                 register into pairs along k.
// The wavefronts' sums meet in LDS and are added in the order of k's parts:
// the result is the same in every run.
//
// 4-bit products quantise the rows of X on the way: each wavefront the 512
// columns of its own iteration, a lane a block of 32 of a row (which needs no
// other lane), through LDS of its own into the instruction's layout, so that no
// wavefront waits for another.  Loads come back in order: the next iteration's
// blocks of X are loaded ahead of its weights, else they would wait for those
// (4 rows, 14336 columns, k = 4096: 11.9 us with the workgroup's rows quantised
// together behind a barrier, 8.9 so).  16 rows over 8 experts of that size: 53 us,
// 4.7 TB/s of 4-bit weights.
//
// Small calls are bound by latency: they take strips of 16 columns and eight
// wavefronts, so that all of B is under way at once (see the launch).
#pragma once

#include "lp_gemm.hpp"
#include "mx4.hpp"

namespace gemmf32 {

enum FewKind { kFewF32 = 0, kFewBf16 = 1, kFewFp4 = 2 };

template <int KIND, bool B_KS, class X, int WAVES_, int NB_>
struct FewTile {
    using E = X;                                     // elements of A and C
    static constexpr int WAVES = WAVES_, THREADS = WAVES * 64;
    // 16-column blocks of a workgroup, and the k that one wavefront's
    // iteration covers.
    static constexpr int NB = B_KS ? (KIND == kFewF32 ? 4 : 8) : NB_;
    static constexpr int BM = 16, BN = 16 * NB;
    static constexpr int KI = KIND == kFewFp4 ? 512 : KIND == kFewF32 ? (B_KS ? 32 : 64) : (B_KS ? 32 : 128);
    static constexpr int LOADS = B_KS ? 8 : 4 * NB;  // 16-byte loads of B a lane and iteration
    static constexpr int A_LOADS = KIND == kFewFp4 ? 0 : KIND == kFewF32 ? KI / 16 : KI / 32;   // of A
    // 4-bit: bytes of a row's codes and scales in LDS (some more than there
    // are: rows on different banks).
    static constexpr int CODE_ROW = KI / 2 + 16, SCALE_ROW = KI / 32 + 4;
};

template <class T, int KIND>
struct FewRegs {
    i32x4 a[KIND == kFewFp4 ? 1 : T::A_LOADS];
    i32x4 b[T::LOADS];
    int s[KIND == kFewFp4 ? T::LOADS : 1];
};

template <int KIND, bool B_KS, class T>
__global__ __launch_bounds__(T::THREADS) void few_grouped_kernel(GroupedArgs g)
{
    using E = typename T::E;
    constexpr int BM = T::BM, BN = T::BN, ROW = BN + 4;
    __shared__ float red[T::WAVES][BM * ROW];
    __shared__ __align__(16) u8 codes_all[KIND == kFewFp4 ? T::WAVES : 1][KIND == kFewFp4 ? 16 * T::CODE_ROW : 16];
    __shared__ u8 scales_all[KIND == kFewFp4 ? T::WAVES : 1][KIND == kFewFp4 ? 16 * T::SCALE_ROW : 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    RowTile rt;
    int tn;
    if (!find_tile<BM>(g, blockIdx.x, lane, rt, tn)) return;
    const int col0 = tn * BN;
    const int l16 = lane & 15, grp = lane >> 4;
    const int rows = min(rt.rows, BM);

    f32x4 acc[T::NB];
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) acc[nb] = f32x4{};

    if (rt.expert >= 0) {
        constexpr int N = 16 / sizeof(E);
        const char *const bx = g.B + rt.expert * g.expert_stride;
        const E *const pa = reinterpret_cast<const E *>(g.A + (rt.row + min(l16, rows - 1)) * g.lda);
        // 4-bit: codes of 128 columns are 64 bytes; counted in k-blocks.
        const int blocks = g.a_kblocks;
        const u8 *sb = nullptr;
        const char *pb[B_KS ? 1 : T::NB];
        if constexpr (B_KS) {
            pb[0] = bx + (KIND == kFewF32 ? grp * 4 : grp * 8) * g.ldb +
                    (long long)(col0 + l16 * (KIND == kFewF32 ? 4 : 8)) * sizeof(E);
        } else {
#pragma unroll
            for (int nb = 0; nb < T::NB; ++nb)
                pb[nb] = bx + min(col0 + nb * 16 + l16, g.n - 1) * g.ldb + grp * 16;
            if constexpr (KIND == kFewFp4) sb = g.b_scales + (long long)rt.expert * blocks * g.n * 4 + grp;
        }
        const int cols_left = g.n - (col0 + l16 * (KIND == kFewF32 ? 4 : 8));   // (k strided)

        u8 *const codes = codes_all[KIND == kFewFp4 ? wave : 0], *const scales = scales_all[KIND == kFewFp4 ? wave : 0];

        auto load = [&](int it, FewRegs<T, KIND> &r) {
            const int k0 = it * T::KI;
            if constexpr (KIND != kFewFp4) {
#pragma unroll
                for (int s = 0; s < T::A_LOADS; ++s) {
                    const int kk = k0 + (s * 4 + grp) * N;
                    r.a[s] = load_chunk(pa + kk, g.k - kk);
                }
            }
            if constexpr (B_KS) {
                constexpr int PER = KIND == kFewF32 ? 4 : 8;
#pragma unroll
                for (int j = 0; j < T::LOADS; ++j) {
                    // (32 bits: two runs of 16 k-rows)
                    const int kr = KIND == kFewF32 ? (j / 4) * 16 + j % 4 : j;
                    const int kk = k0 + kr + grp * PER;
                    r.b[j] = load_chunk(reinterpret_cast<const E *>(pb[0] + (long long)(k0 + kr) * g.ldb),
                                        kk < g.k ? cols_left : 0);
                }
            } else if constexpr (KIND == kFewFp4) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int kb = min(it * 4 + s, blocks - 1);
#pragma unroll
                    for (int nb = 0; nb < T::NB; ++nb) {
                        r.b[s * T::NB + nb] = *reinterpret_cast<const i32x4 *>(pb[nb] + (long long)kb * 64);
                        r.s[s * T::NB + nb] = sb[((long long)kb * g.n + min(col0 + nb * 16 + l16, g.n - 1)) * 4];
                    }
                }
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int kk = k0 + (s * 4 + grp) * N;
#pragma unroll
                    for (int nb = 0; nb < T::NB; ++nb)
                        r.b[s * T::NB + nb] =
                            load_chunk(reinterpret_cast<const E *>(pb[nb] + (long long)(k0 + s * 4 * N) * sizeof(E)), g.k - kk);
                }
            }
        };
        auto multiply = [&](int it, const FewRegs<T, KIND> &r) {
            if constexpr (KIND == kFewFp4) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int kb = it * 4 + s;
                    if (kb >= blocks) break;
                    const int row = min(l16, rows - 1);
                    const i32x4 c = *reinterpret_cast<const i32x4 *>(codes + row * T::CODE_ROW + s * 64 + grp * 16);
                    const int byte = scales[row * T::SCALE_ROW + s * 4 + grp];
                    const i32x8 a = {c[0], c[1], c[2], c[3], 0, 0, 0, 0};
#pragma unroll
                    for (int nb = 0; nb < T::NB; ++nb) {
                        const i32x4 w = r.b[s * T::NB + nb];
                        const i32x8 b = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
                        acc[nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc[nb], 4, 4, 0,
                                                                                  r.s[s * T::NB + nb], 0, byte);
                    }
                }
            } else {
#pragma unroll
                for (int s = 0; s < T::A_LOADS; ++s) {
                    const i32x4 a = r.a[s];
                    if constexpr (KIND == kFewF32) {
                        const f32x4 af = __builtin_bit_cast(f32x4, a);
                        if constexpr (B_KS) {
                            // k-rows 4 grp + j of the run; set c: columns 4 i + c.
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const f32x4 bf = __builtin_bit_cast(f32x4, r.b[s * 4 + j]);
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    acc[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(bf[c], af[j], acc[c], 0, 0, 0);
                            }
                        } else {
#pragma unroll
                            for (int nb = 0; nb < T::NB; ++nb) {
                                const f32x4 bf = __builtin_bit_cast(f32x4, r.b[s * T::NB + nb]);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    acc[nb] = __builtin_amdgcn_mfma_f32_16x16x4f32(bf[j], af[j], acc[nb], 0, 0, 0);
                            }
                        }
                    } else {
                        const bf16x8 af = __builtin_bit_cast(bf16x8, a);
#pragma unroll
                        for (int nb = 0; nb < T::NB; ++nb) {
                            i32x4 b;
                            if constexpr (B_KS) {
                                // Column nb of the lane's eight, its k-rows in pairs.
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    b[i] = (int)__builtin_amdgcn_perm((unsigned)r.b[2 * i + 1][nb / 2],
                                                                      (unsigned)r.b[2 * i][nb / 2],
                                                                      nb & 1 ? 0x07060302u : 0x05040100u);
                            } else {
                                b = r.b[s * T::NB + nb];
                            }
                            acc[nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), af,
                                                                              acc[nb], 0, 0, 0);
                        }
                    }
                }
            }
        };
        // 4-bit: the lane's block of row 4 part + grp.
        Mx8<E> x[4];
        auto load_x = [&](int it, int part) {
            const int row = min(part * 4 + grp, rows - 1), k = it * T::KI + l16 * 32;
            const E *const p = reinterpret_cast<const E *>(g.A + (rt.row + row) * g.lda) + k;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i].load(p + 8 * i, g.k - k - 8 * i);
        };
        auto quantise = [&](int it) {
            for (int part = 0;;) {
                unsigned largest = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) largest = max(largest, x[i].largest());
                const MxBlock m = mx_block(largest);
                i32x4 a;
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = m.byte == 255 ? 0 : (int)x[i].codes(m.scale);
                const int row = part * 4 + grp;
                *reinterpret_cast<i32x4 *>(codes + row * T::CODE_ROW + l16 * 16) = a;
                scales[row * T::SCALE_ROW + l16] = (u8)m.byte;
                if (++part * 4 >= rows) break;
                load_x(it, part);
            }
        };
        // The loads of an iteration, and what its products need besides.
        auto fetch = [&](int it, FewRegs<T, KIND> &r) {
            if constexpr (KIND == kFewFp4) load_x(it, 0);
            load(it, r);
        };
        auto prepare = [&](int it) {
            if constexpr (KIND == kFewFp4) {
                wave_sync();
                quantise(it);
                wave_sync();
            }
        };

        const int its = KIND == kFewFp4 ? (blocks + 3) / 4 : (g.k + T::KI - 1) / T::KI;
        FewRegs<T, KIND> r[2];
        if (wave < its) fetch(wave, r[0]);
        int it = wave;
        while (it < its) {
            prepare(it);
            if (it + T::WAVES < its) fetch(it + T::WAVES, r[1]);
            multiply(it, r[0]);
            it += T::WAVES;
            if (it >= its) continue;
            prepare(it);
            if (it + T::WAVES < its) fetch(it + T::WAVES, r[0]);
            multiply(it, r[1]);
            it += T::WAVES;
        }
    }

    // Lane (l16, grp) holds row l16 and columns 4 grp + v of each block:
    // column 16 nb + i (k contiguous) or NB i + nb (k strided) of the strip.
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int i = 4 * grp + v;
            red[wave][l16 * ROW + (B_KS ? T::NB * i + nb : nb * 16 + i)] = acc[nb][v];
        }
    __syncthreads();
    const float *const bias = g.bias && rt.expert >= 0 ? g.bias + rt.expert * g.bias_stride + col0 : nullptr;
    for (int e = tid; e < rows * BN; e += T::THREADS) {
        const int row = e / BN, col = e % BN;
        if (col0 + col >= g.n) continue;
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < T::WAVES; ++w) x += red[w][row * ROW + col];
        if (rt.expert < 0) {
            x = 0.0f;
        } else {
            if (bias) x += bias[col];
            x = activate(x, g.act);
        }
        *(reinterpret_cast<E *>(g.C + (rt.row + row) * g.ldc) + col0 + col) = (E)x;
    }
}

}  // namespace gemmf32
