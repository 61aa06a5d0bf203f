// Products grouped by expert on the low-precision matrix cores: bfloat16
// (v_mfma_f32_32x32x16_bf16) and microscaled 4-bit operands
// (v_mfma_scale_f32_32x32x64_f8f6f4), accumulated in 32 bits.
//
//   C_e = act(A_e . B_e + bias_e)   A_e: the rows of expert e
//   dB_e = A_e^T . G_e              (A_KS: the contraction runs over A's rows)
//
// The two types share one kernel because they share its data flow: a lane's
// operand of one matrix instruction is 16 contiguous bytes, 8 bfloat16 or 32
// 4-bit values of one row, an instruction covers 32 bytes of each row, and
// takes as long (32 cycles).  A slab is 128 bytes along k: 64 bfloat16, 256
// 4-bit values; four k-steps.
//
// Operands travel from memory straight into LDS (buffer_load ... lds, 16
// bytes a lane) into a ring of STAGES slabs; the kernel is bound by the
// matrix cores and by the LDS reads that feed them (a 128 x 64 wavefront
// tile reads 96 bytes a cycle and CU of the 128 there are).  The last k-step
// of a slab comes after the barrier that hands the next slab over, so its
// products cover the first reads of that slab.
//
// LDS layouts (a copy places lane i's 16 bytes at the wavefront's base + 16 i,
// so a layout is chosen by which global chunk each lane fetches):
//   k contiguous   row r, chunk c at [r][c ^ (r / 2) % 8]: 128-byte rows, two
//                  to the 256 bytes of the banks; the 16 rows a fragment read
//                  touches at a time fall on 16 distinct places.
//   k strided      (row-major B; both operands of the weight gradient) k-row
//                  kr, chunk c at [kr][c ^ 4 (kr % 4)]; the fragment is read
//                  with the transposing LDS read (ds_read_b64_tr_b16), which
//                  hands lane i of 16 column i of four k-rows: the four rows'
//                  64-byte pieces fall on distinct quarters of the banks.
// The rows of B (columns of C) of a block of 32 are read in the order
// 16 ((i / 4) % 2) + 4 (i / 8) + i % 4, which gives each lane 16 neighbouring
// columns of one row of C: 16-byte stores.  Contiguous B is put in that order
// by the copy, strided B by the addresses of the transposing read.
//
// Rows past an expert's end are another expert's (or, past the matrix, its
// last row again): they only feed rows of C that are not stored.  Elements
// past k are made zero in both operands: k-rows past the end by the buffer's
// range check, the tail of contiguous rows in LDS after the copy has landed.
#pragma once

#include "expert_common.hpp"

namespace gemmf32 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4_t;
typedef __attribute__((address_space(3))) void *lds_void_t;

enum LpKind { kBf16 = 0, kFp4 = 1 };

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_>
struct LpTile {
    static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
    static constexpr int THREADS = WAVES_M * WAVES_N * 64;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    static constexpr int MB = WM / 32, NB = WN / 32;      // 32 x 32 blocks of a wavefront
    static constexpr int A_CHUNKS = BM * 8, B_CHUNKS = BN * 8;
    static constexpr int A_PER_T = A_CHUNKS / THREADS, B_PER_T = B_CHUNKS / THREADS;
    static constexpr int PIECES = A_PER_T + B_PER_T;
    static constexpr int SCALE_CHUNKS = (BM + BN) / 2;    // two words of scales a row and slab
    static_assert(A_CHUNKS % THREADS == 0 && B_CHUNKS % THREADS == 0, "whole copies");
    static_assert(WM % 32 == 0 && WN % 32 == 0, "32 x 32 blocks");
    static constexpr int stage_chunks(int kind) { return A_CHUNKS + B_CHUNKS + (kind == kFp4 ? SCALE_CHUNKS : 0); }
};

// One operand of one tile, seen from its first row and column.
struct LpOperand {
    const char *p;
    long long bytes;      // extent from p to the operand's end
    int ld;               // bytes from row to row
    int rows;             // rows that may be read (k contiguous), or columns (k strided)
};

__device__ __forceinline__ void lp_copy16(__amdgpu_buffer_rsrc_t r, uint32_t off, i32x4 *wave_chunk)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t)wave_chunk, 16, (int)off, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t lp_rsrc(const char *p, long long bytes)
{
    // Up to the end of the last 32-bit word: a word that holds one 16-bit
    // element of the operand is read whole.
    bytes = (bytes + 3) & ~3ll;
    return make_rsrc(p, bytes < 0 ? 0u : bytes > 0x7ffffffcll ? 0x7ffffffcu : (uint32_t)bytes);
}

// Row of a tile that LDS row r of B holds.
__device__ __forceinline__ int lp_b_row(int r)
{
    const int i = r & 31;
    return (r & ~31) + 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3);
}

template <int WIDTH>
__device__ __forceinline__ int lp_strided_swizzle(int kr)
{
    return WIDTH >= 128 ? 4 * (kr & 3) : 4 * ((kr >> 1) & 1);
}

// Byte offset, in its operand at slab 0, of the chunk that lane `tid` copies
// as piece j.
template <class T, bool IS_B, bool KS>
__device__ __forceinline__ uint32_t lp_offset(const LpOperand &o, int j, int tid, int &kr)
{
    constexpr int W = IS_B ? T::BN : T::BM;
    const int c = tid + j * T::THREADS;
    if constexpr (KS) {
        kr = c / (W / 8);
        return (uint32_t)kr * (uint32_t)o.ld + (uint32_t)((c % (W / 8)) ^ lp_strided_swizzle<W>(kr)) * 16u;
    } else {
        kr = 0;
        const int r = c / 8;
        const int row = min(IS_B ? lp_b_row(r) : r, o.rows - 1);
        return (uint32_t)row * (uint32_t)o.ld + (uint32_t)((c % 8) ^ ((r >> 1) & 7)) * 16u;
    }
}

// Zero the elements at or past k of the chunks that this lane copied.
template <class T, bool IS_B>
__device__ __forceinline__ void lp_zero_tail(i32x4 *region, int tid, int left)
{
    constexpr int N = IS_B ? T::B_PER_T : T::A_PER_T;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = tid + j * T::THREADS;
        const int k0 = ((c % 8) ^ ((c / 8 >> 1) & 7)) * 8;
        i32x4 v = region[c];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] &= (k0 + 2 * i < left ? 0xffff : 0) | (k0 + 2 * i + 1 < left ? (int)0xffff0000u : 0);
        region[c] = v;
    }
}

template <int N>
__device__ __forceinline__ void lp_barrier()
{
    // At most N copies in flight, LDS reads and writes done, then the bare
    // barrier (a fence would wait for every copy).
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
    asm volatile("s_barrier" ::: "memory");
}

template <class T, int KIND>
struct LpFrags {
    i32x4 a[2][T::MB], b[2][T::NB];
    int sa[2][KIND == kFp4 ? T::MB : 1], sb[2][KIND == kFp4 ? T::NB : 1];
};

// Fragments of k-step p.
template <class T, int KIND, bool A_KS, bool B_KS>
__device__ __forceinline__ void lp_read(const i32x4 *As, const i32x4 *Bs, int p, int wr, int wc, int lane,
                                        LpFrags<T, KIND> &f)
{
    const int l32 = lane & 31, half = lane >> 5;
    auto contiguous = [&](const i32x4 *region, int row) {
        return region[row * 8 + ((2 * p + half) ^ ((l32 >> 1) & 7))];
    };
    // Two transposing reads: k-rows 8 half + 0..3 and + 4..7 of the step.
    auto strided = [&](const i32x4 *region, int width, int col, int swz) {
        const int kr = 16 * p + 8 * half + ((lane & 15) >> 2);
        const char *q = reinterpret_cast<const char *>(region + kr * (width / 8) + ((col / 8) ^ swz)) + (col & 7) * 2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)q);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(q + 4 * width * 2));
        const u32x2 x = __builtin_bit_cast(u32x2, lo), y = __builtin_bit_cast(u32x2, hi);
        return i32x4{(int)x.x, (int)x.y, (int)y.x, (int)y.y};
    };
    const int quad = ((lane >> 4) & 1) * 4 + (lane & 3);         // of the 8 column quads of a block
    const int krow = (lane & 15) >> 2;
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) {
        const int row = wr * T::WM + mb * 32;
        if constexpr (A_KS) f.a[p & 1][mb] = strided(As, T::BM, row + 4 * quad, lp_strided_swizzle<T::BM>(krow));
        else f.a[p & 1][mb] = contiguous(As, row + l32);
    }
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) {
        const int row = wc * T::WN + nb * 32;
        if constexpr (B_KS)
            f.b[p & 1][nb] = strided(Bs, T::BN, row + 4 * (4 * (quad & 1) + (quad >> 1)),
                                     lp_strided_swizzle<T::BN>(krow));
        else f.b[p & 1][nb] = contiguous(Bs, row + l32);
    }
}

// Scale words of k-steps 2 q and 2 q + 1, shifted so that the lane's block of
// step 2 q is byte 0 and of step 2 q + 1 byte 2.
template <class T, int KIND>
__device__ __forceinline__ void lp_read_scales(const i32x4 *Ss, int q, int wr, int wc, int lane, LpFrags<T, KIND> &f)
{
    if constexpr (KIND == kFp4) {
        const int l32 = lane & 31, half = lane >> 5;
        const unsigned *w = reinterpret_cast<const unsigned *>(Ss) + q * (T::BM + T::BN);
        const int i = l32;
        const int b_row = 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3);
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb) f.sa[q][mb] = (int)(w[wr * T::WM + mb * 32 + l32] >> (8 * half));
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) f.sb[q][nb] = (int)(w[T::BM + wc * T::WN + nb * 32 + b_row] >> (8 * half));
    }
}

template <class T, int KIND>
__device__ __forceinline__ void lp_mfma(int i, int p, const LpFrags<T, KIND> &f, f32x16 (&acc)[T::MB][T::NB])
{
    const int mb = i / T::NB, nb = i % T::NB;
    const i32x4 a = f.a[p & 1][mb], b = f.b[p & 1][nb];
    // B first: the lane's column of the result is a row of A, its sixteen
    // values are columns of C.
    if constexpr (KIND == kBf16) {
        acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b),
                                                              __builtin_bit_cast(bf16x8, a), acc[mb][nb], 0, 0, 0);
    } else {
        const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
        if (p & 1)
            acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[mb][nb], 4, 4, 2,
                                                                          f.sb[p >> 1][nb], 2, f.sa[p >> 1][mb]);
        else
            acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[mb][nb], 4, 4, 0,
                                                                          f.sb[p >> 1][nb], 0, f.sa[p >> 1][mb]);
    }
}

// What a tile needs of its operands.
struct LpProblem {
    LpOperand a, b;
    const u8 *a_scales, *b_scales;     // of the tile's first rows, k-block 0
    long long a_scale_bytes, b_scale_bytes;   // extents
    long long a_scale_step, b_scale_step;     // bytes from k-block to k-block
    int k;                             // contraction (4-bit: kp)
};

// REG: operands whose rows are not 4-byte aligned (bfloat16 rows of odd
// length) cannot be copied straight into LDS; their chunks pass through
// registers, one slab ahead, with the tails made zero on the way.
template <class T, int KIND, bool A_KS, bool B_KS, bool REG = false>
struct LpLoop {
    static_assert(!REG || (KIND == kBf16 && T::STAGES == 2), "register copies: bfloat16, two stages");
    static constexpr int KSLAB = KIND == kFp4 ? 256 : 64;
    static constexpr int SCALE_PER_T = (T::SCALE_CHUNKS + T::THREADS - 1) / T::THREADS;
    static_assert(KIND != kFp4 || (T::BM % 64 == 0 && T::BN % 64 == 0), "scale words in whole copies");
    const LpProblem &q;
    i32x4 *lds;
    int tid, lane, wave, wr, wc;
    int slabs, tail;               // slabs; elements of the last one, 0: full
    uint32_t a_off[T::A_PER_T], b_off[T::B_PER_T];
    int a_kr[T::A_PER_T], b_kr[T::B_PER_T];
    i32x4 regs[REG ? T::PIECES : 1];
    uint32_t s_off[KIND == kFp4 ? SCALE_PER_T : 1];

    __device__ __forceinline__ i32x4 *stage(int s) const { return lds + s * T::stage_chunks(KIND); }

    __device__ __forceinline__ void setup()
    {
#pragma unroll
        for (int j = 0; j < T::A_PER_T; ++j) a_off[j] = lp_offset<T, false, A_KS>(q.a, j, tid, a_kr[j]);
#pragma unroll
        for (int j = 0; j < T::B_PER_T; ++j) b_off[j] = lp_offset<T, true, B_KS>(q.b, j, tid, b_kr[j]);
        if constexpr (KIND == kFp4)
#pragma unroll
            for (int j = 0; j < SCALE_PER_T; ++j) {
                const int c = j * T::THREADS + tid, at = c % (T::SCALE_CHUNKS / 2);
                const bool is_a = at < T::BM / 4;
                s_off[j] = (c < T::SCALE_CHUNKS / 2 ? 0u : (uint32_t)(is_a ? q.a_scale_step : q.b_scale_step)) +
                           (uint32_t)(is_a ? at : at - T::BM / 4) * 16u;
            }
        slabs = (q.k + KSLAB - 1) / KSLAB;
        tail = q.k % KSLAB;
    }

    // Copy slab kt into its stage.
    __device__ __forceinline__ void copy(int kt) const
    {
        i32x4 *const st = stage(kt % T::STAGES);
        const int left = q.k - kt * KSLAB;             // elements from the slab's first on
        const long long sa = A_KS ? (long long)kt * KSLAB * q.a.ld : (long long)kt * 128;
        const long long sb = B_KS ? (long long)kt * KSLAB * q.b.ld : (long long)kt * 128;
        const __amdgpu_buffer_rsrc_t ra = lp_rsrc(q.a.p + sa, q.a.bytes - sa);
        const __amdgpu_buffer_rsrc_t rb = lp_rsrc(q.b.p + sb, q.b.bytes - sb);
#pragma unroll
        for (int j = 0; j < T::A_PER_T; ++j)
            lp_copy16(ra, A_KS && a_kr[j] >= left ? kOobOffset : a_off[j], st + j * T::THREADS + wave * 64);
#pragma unroll
        for (int j = 0; j < T::B_PER_T; ++j)
            lp_copy16(rb, B_KS && b_kr[j] >= left ? kOobOffset : b_off[j],
                      st + T::A_CHUNKS + j * T::THREADS + wave * 64);
        if constexpr (KIND == kFp4) {
            // Words of scales: [k-block][rows of A, rows of B], four rows a
            // chunk; the wavefronts take 64 chunks each.  A block past the
            // last one is past the extents and reads as zero.
            const long long ka = (long long)(2 * kt) * q.a_scale_step, kb = (long long)(2 * kt) * q.b_scale_step;
            const __amdgpu_buffer_rsrc_t rsa =
                lp_rsrc(reinterpret_cast<const char *>(q.a_scales) + ka, q.a_scale_bytes - ka);
            const __amdgpu_buffer_rsrc_t rsb =
                lp_rsrc(reinterpret_cast<const char *>(q.b_scales) + kb, q.b_scale_bytes - kb);
            i32x4 *const ss = st + T::A_CHUNKS + T::B_CHUNKS;
#pragma unroll
            for (int j = 0; j < SCALE_PER_T; ++j) {
                const int w0 = j * T::THREADS + wave * 64;
                if (w0 < T::SCALE_CHUNKS) {
                    if ((w0 + lane) % (T::SCALE_CHUNKS / 2) < T::BM / 4) lp_copy16(rsa, s_off[j], ss + w0);
                    else lp_copy16(rsb, s_off[j], ss + w0);
                }
            }
        }
    }

    // Register copies: the chunks of slab kt, and their places in LDS.
    __device__ __forceinline__ void load(int kt)
    {
        const int left = q.k - kt * KSLAB;
        auto chunk = [&](const LpOperand &o, bool ks, uint32_t off, int kr, int c, int width, int swz) {
            if (ks) {
                const int col = ((c % (width / 8)) ^ swz) * 8;
                return load_chunk(reinterpret_cast<const __bf16 *>(o.p + (long long)kt * KSLAB * o.ld + off),
                                  kr < left ? o.rows - col : 0);
            }
            const int k0 = ((c % 8) ^ ((c / 8 >> 1) & 7)) * 8;
            return load_chunk(reinterpret_cast<const __bf16 *>(o.p + (long long)kt * 128 + off), left - k0);
        };
#pragma unroll
        for (int j = 0; j < T::A_PER_T; ++j)
            regs[j] = chunk(q.a, A_KS, a_off[j], a_kr[j], tid + j * T::THREADS, T::BM, lp_strided_swizzle<T::BM>(a_kr[j]));
#pragma unroll
        for (int j = 0; j < T::B_PER_T; ++j)
            regs[T::A_PER_T + j] =
                chunk(q.b, B_KS, b_off[j], b_kr[j], tid + j * T::THREADS, T::BN, lp_strided_swizzle<T::BN>(b_kr[j]));
    }

    __device__ __forceinline__ void store(int kt) const
    {
        i32x4 *const st = stage(kt % T::STAGES);
#pragma unroll
        for (int j = 0; j < T::PIECES; ++j) st[tid + j * T::THREADS] = regs[j];
    }

    __device__ __forceinline__ void fix_tail(int kt) const
    {
        if constexpr (KIND == kBf16) {
            i32x4 *const st = stage(kt % T::STAGES);
            if constexpr (!A_KS) lp_zero_tail<T, false>(st, tid, tail);
            if constexpr (!B_KS) lp_zero_tail<T, true>(st + T::A_CHUNKS, tid, tail);
        }
    }

    __device__ __forceinline__ void read(int kt, int p, LpFrags<T, KIND> &f) const
    {
        const i32x4 *const st = stage(kt % T::STAGES);
        if (KIND == kFp4 && (p & 1) == 0) lp_read_scales<T, KIND>(st + T::A_CHUNKS + T::B_CHUNKS, p >> 1, wr, wc, lane, f);
        lp_read<T, KIND, A_KS, B_KS>(st, st + T::A_CHUNKS, p, wr, wc, lane, f);
    }

    // One slab.  WAIT: copies that may stay in flight when the next slab is
    // taken over; -1: there is no next slab.
    template <int WAIT, bool COPY>
    __device__ __forceinline__ void slab(int kt, LpFrags<T, KIND> &f, f32x16 (&acc)[T::MB][T::NB])
    {
        constexpr int NM = T::MB * T::NB;
        // A 4-bit slab of one k-block (the last one of an odd number) holds
        // two k-steps' values; the others' codes are another row's.
        const bool half_slab = KIND == kFp4 && WAIT < 0 && tail != 0;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            if (KIND == kFp4 && WAIT < 0 && p >= 2 && half_slab) break;
            __builtin_amdgcn_s_setprio(1);
            lp_mfma<T, KIND>(0, p, f, acc);
            __builtin_amdgcn_sched_barrier(0);
            read(kt, p + 1, f);
#pragma unroll
            for (int i = 1; i < NM; ++i) lp_mfma<T, KIND>(i, p, f, acc);
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (WAIT >= 0) {
            if constexpr (REG) {
                store(kt + 1);
            } else if (kt + 2 == slabs && tail != 0 && KIND == kBf16 && !(A_KS && B_KS)) {
                __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (15 << 8));
                fix_tail(kt + 1);
            }
            lp_barrier<WAIT>();
            if constexpr (COPY && REG) load(kt + 2);
            else if constexpr (COPY) copy(kt + T::STAGES);
            __builtin_amdgcn_sched_barrier(0);
            lp_mfma<T, KIND>(0, 3, f, acc);
            __builtin_amdgcn_sched_barrier(0);
            read(kt + 1, 0, f);
#pragma unroll
            for (int i = 1; i < NM; ++i) lp_mfma<T, KIND>(i, 3, f, acc);
            __builtin_amdgcn_sched_barrier(0);
        } else if (!half_slab) {
#pragma unroll
            for (int i = 0; i < NM; ++i) lp_mfma<T, KIND>(i, 3, f, acc);
        }
    }

    __device__ __forceinline__ void run(f32x16 (&acc)[T::MB][T::NB])
    {
        constexpr int P = T::PIECES;
        setup();
        if (slabs == 0) return;
        LpFrags<T, KIND> f;
        if constexpr (REG) {
            load(0);
            store(0);
            if (slabs > 1) load(1);
        } else {
#pragma unroll
            for (int s = 0; s < T::STAGES; ++s)
                if (s < slabs) copy(s);
        }
        if constexpr (REG) {
            lp_barrier<63>();
        } else if (slabs == 1) {
            __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (15 << 8));
            if (tail) fix_tail(0);
            lp_barrier<0>();
        } else if (KIND == kBf16 && slabs >= T::STAGES) {
            lp_barrier<(T::STAGES - 1) * P>();
        } else {
            lp_barrier<0>();
        }
        read(0, 0, f);
        int kt = 0;
        // (4-bit: the wavefronts' numbers of scale copies differ, so every
        // copy in flight is counted as the values' alone: a wait for fewer.)
        constexpr int WAIT = REG ? 63 : (T::STAGES - 2) * P;
        for (; kt + T::STAGES < slabs; ++kt) slab<WAIT, true>(kt, f, acc);
        for (; kt + 1 < slabs; ++kt) slab<REG ? 63 : 0, false>(kt, f, acc);
        slab<-1, false>(kt, f, acc);
    }
};

// C's 32 x 32 blocks: lane l32 holds row l32 of the block, columns 16 half ..
// + 15.  WIDE: rows and column runs of C are 16-byte aligned and n is a
// multiple of the elements in 16 bytes.
template <class T, class E, bool WIDE>
__device__ __forceinline__ void lp_store(char *c, long long ldc, int rows, int cols, const float *bias, int act,
                                         bool zero, int wr, int wc, int lane, const f32x16 (&acc)[T::MB][T::NB])
{
    const int l32 = lane & 31, half = lane >> 5;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) {
        const int col = wc * T::WN + nb * 32 + 16 * half;
        float b[16];
#pragma unroll
        for (int v = 0; v < 16; ++v) b[v] = bias && col + v < cols ? bias[col + v] : 0.0f;
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb) {
            const int row = wr * T::WM + mb * 32 + l32;
            E y[16];
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                float x = acc[mb][nb][v] + b[v];
                if (act) x = activate(x, act);
                // One rounding, to the type of C.
                y[v] = (E)(zero ? 0.0f : x);
            }
            E *const p = reinterpret_cast<E *>(c + row * ldc) + col;
            if (row < rows) {
                if constexpr (WIDE) {
                    constexpr int N = 16 / sizeof(E);
#pragma unroll
                    for (int v = 0; v < 16; v += N)
                        if (col + v < cols) {
                            struct alignas(16) Run {
                                E e[N];
                            } r;
#pragma unroll
                            for (int i = 0; i < N; ++i) r.e[i] = y[v + i];
                            *reinterpret_cast<Run *>(p + v) = r;
                        }
                } else {
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (col + v < cols) p[v] = y[v];
                }
            }
        }
    }
}

// C_e = act(A_e . B_e + bias_e).
template <class T, int KIND, bool B_KS, class E, bool WIDE, bool REG = false>
__global__ __launch_bounds__(T::THREADS) void lp_grouped_kernel(GroupedArgs g)
{
    __shared__ i32x4 lds[T::STAGES * T::stage_chunks(KIND)];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    RowTile rt;
    int tn;
    if (!find_tile<T::BM>(g, blockIdx.x, lane, rt, tn)) return;
    const int col0 = tn * T::BN, cols = g.n - col0;
    const int wr = wave % T::WAVES_M, wc = wave / T::WAVES_M;
    f32x16 acc[T::MB][T::NB];
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
    if (rt.expert >= 0) {
        LpProblem q;
        const long long row_bytes = KIND == kFp4 ? (long long)g.a_kblocks * 64 : (long long)g.k * 2;
        q.a = {g.A + rt.row * g.lda, (g.m - 1 - rt.row) * g.lda + row_bytes, (int)g.lda, g.m - rt.row};
        const char *const b = g.B + rt.expert * g.expert_stride;
        if constexpr (B_KS)
            q.b = {b + (long long)col0 * 2, (long long)(g.k - 1) * g.ldb + (long long)cols * 2, (int)g.ldb, cols};
        else
            q.b = {b + col0 * g.ldb, (cols - 1) * g.ldb + row_bytes, (int)g.ldb, cols};
        q.k = g.k;
        if constexpr (KIND == kFp4) {
            q.k = g.a_kblocks * 128;
            q.a_scales = g.a_scales + (long long)rt.row * 4;
            q.a_scale_step = (long long)g.m * 4;
            q.a_scale_bytes = g.a_kblocks * q.a_scale_step - (long long)rt.row * 4;
            q.b_scale_step = (long long)g.n * 4;
            q.b_scales = g.b_scales + rt.expert * (g.a_kblocks * q.b_scale_step) + (long long)col0 * 4;
            q.b_scale_bytes = g.a_kblocks * q.b_scale_step - (long long)col0 * 4;
        }
        LpLoop<T, KIND, false, B_KS, REG> loop{q, lds, tid, lane, wave, wr, wc};
        loop.run(acc);
    }
    const float *bias = g.bias && rt.expert >= 0 ? g.bias + rt.expert * g.bias_stride + col0 : nullptr;
    lp_store<T, E, WIDE>(g.C + rt.row * g.ldc + (long long)col0 * sizeof(E), g.ldc, rt.rows, cols, bias, g.act,
                         rt.expert < 0, wr, wc, lane, acc);
}

// dB_e = A_e^T . G_e: g.m rows of A (g.k columns) and G (g.n columns); tiles of
// the experts' k x n matrices.  An expert without rows gets zeros.
template <class T, bool WIDE, bool REG = false>
__global__ __launch_bounds__(T::THREADS) void lp_weight_grad_kernel(GroupedArgs g)
{
    __shared__ i32x4 lds[T::STAGES * T::stage_chunks(kBf16)];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = g.tiles_m * g.tiles_n;
    const int logical = xcd_contiguous(blockIdx.x, per * g.groups, g.num_xcd);
    const int expert = logical / per;
    const int r = logical % per;
    const int width = g.group_m * g.tiles_n;
    const int first = r / width * g.group_m, size = min(g.tiles_m - first, g.group_m);
    const int tm = first + r % width % size, tn = r % width / size;
    int lo, hi;
    entry_rows(g, expert, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int row0 = tm * T::BM, col0 = tn * T::BN;
    const int wr = wave % T::WAVES_M, wc = wave / T::WAVES_M;
    f32x16 acc[T::MB][T::NB];
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
    LpProblem q;
    const long long last = hi - lo - 1;      // -1: no rows, no bytes are read
    q.a = {g.A + lo * g.lda + (long long)row0 * 2, last * g.lda + (long long)(g.k - row0) * 2, (int)g.lda, g.k - row0};
    q.b = {g.B + lo * g.ldb + (long long)col0 * 2, last * g.ldb + (long long)(g.n - col0) * 2, (int)g.ldb, g.n - col0};
    q.k = hi - lo;
    LpLoop<T, kBf16, true, true, REG> loop{q, lds, tid, lane, wave, wr, wc};
    loop.run(acc);
    lp_store<T, __bf16, WIDE>(g.C + expert * g.expert_stride + row0 * g.ldc + (long long)col0 * 2, g.ldc,
                              g.k - row0, g.n - col0, nullptr, 0, false, wr, wc, lane, acc);
}

}  // namespace gemmf32
