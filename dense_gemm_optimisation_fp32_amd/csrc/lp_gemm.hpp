// Products grouped by expert on the low-precision matrix cores: bfloat16
// (v_mfma_f32_32x32x16_bf16) and microscaled 4-bit operands
// (v_mfma_scale_f32_32x32x64_f8f6f4), accumulated in 32 bits, and 8-bit
// integers (v_mfma_i32_32x32x32_i8), accumulated exactly in 32-bit integers.
//
//   C_e = act(A_e . B_e + bias_e)   A_e: the rows of expert e
//   dB_e = A_e^T . G_e              (A_KS: the contraction runs over A's rows)
//
// The types share one kernel because they share its data flow: a lane's
// operand of one matrix instruction is 16 contiguous bytes, 8 bfloat16, 16
// integers or 32 4-bit values of one row, an instruction covers 32 bytes of each
// row, and takes as long (32 cycles).  A slab is 128 bytes along k: 64 bfloat16,
// 128 integers, 256 4-bit values; four k-steps.
//
// Operands travel from memory straight into LDS (buffer_load ... lds, 16
// bytes a lane) into a ring of STAGES slabs.  The last k-step of a slab comes
// after the barrier that hands the next slab over, so its products cover the
// first reads of that slab.  What bounds the products: see lp_pipe.hpp; few of
// them are bound by how many slabs are under way, hence the longer rings of
// the smaller tiles.
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
// The rows of B (columns of C) of a block of 32 are read in an order
// (lp_column) that gives each lane runs of 16 bytes of C, two lanes' side by
// side.  Contiguous B is put in that order by the copy, strided B by the
// addresses of the transposing read.
//
// Rows past an expert's end are another expert's (or, past the matrix, its
// last row again): they only feed rows of C that are not stored.  Elements
// past k are made zero in both operands: k-rows past the end by the buffer's
// range check, the tail of contiguous rows in LDS after the copy has landed.
// (Integers: A's rows are whole slabs, with zeros past k; what B has there, the
// next row's codes, is finite and counts nothing.)
#pragma once

#include "expert_common.hpp"

namespace gemmf32 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4_t;
typedef __attribute__((address_space(3))) void *lds_void_t;

// (kF16: half-precision planes of 32-bit numbers, see orthogonal.hpp; whole slabs.)
enum LpKind { kBf16 = 0, kFp4 = 1, kInt8 = 2, kF16 = 3 };

// Values of a 16-byte chunk.
constexpr int lp_values(int kind) { return kind == kFp4 ? 32 : kind == kInt8 ? 16 : 8; }

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_>
struct LpTile {
    static constexpr int CPR = 8;                         // 16-byte chunks of a row and slab
    static constexpr int STEPS = CPR / 2;                 // k-steps of a slab
    static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
    static constexpr int THREADS = WAVES_M * WAVES_N * 64;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    static constexpr int MB = WM / 32, NB = WN / 32;      // 32 x 32 blocks of a wavefront
    static constexpr int A_CHUNKS = BM * CPR, B_CHUNKS = BN * CPR;
    static constexpr int A_PER_T = A_CHUNKS / THREADS, B_PER_T = B_CHUNKS / THREADS;
    static constexpr int PIECES = A_PER_T + B_PER_T;
    // 4-bit: a word of scales for 64 bytes of a row, A's and B's each in whole
    // wavefront copies of 64 chunks.
    static constexpr int KBLOCKS = CPR / 4;
    static constexpr int SCALE_WAVES_A = (BM * KBLOCKS / 4 + 63) / 64, SCALE_WAVES_B = (BN * KBLOCKS / 4 + 63) / 64;
    static constexpr int SCALE_CHUNKS = (SCALE_WAVES_A + SCALE_WAVES_B) * 64;
    static_assert(A_CHUNKS % THREADS == 0 && B_CHUNKS % THREADS == 0, "whole copies");
    static_assert(WM % 32 == 0 && WN % 32 == 0, "32 x 32 blocks");
    // Where chunk c of row r of a contiguous operand lies: the 16 rows that a
    // fragment read touches at a time fall on 16 places of the 256 bytes of
    // the banks.
    static __device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 7; }
    static constexpr int stage_chunks(int kind) { return A_CHUNKS + B_CHUNKS + (kind == kFp4 ? SCALE_CHUNKS : 0); }
};

// One operand of one tile, seen from its first row and column.
struct LpOperand {
    const char *p;
    long long bytes;      // extent from p to the operand's end
    int ld;               // bytes from row to row
    int rows;             // rows that may be read (k contiguous), or columns (k strided)
};

// A raw buffer descriptor of `bytes` from p on (word 3 as in make_rsrc).
__device__ __forceinline__ i32x4 lp_rsrc(const char *p, long long bytes)
{
    // Up to the end of the last 32-bit word: a word that holds one 16-bit
    // element of the operand is read whole.
    bytes = (bytes + 3) & ~3ll;
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    return i32x4{(int)(uint32_t)at, (int)((uint32_t)(at >> 32) & 0xffffu),
                 (int)(bytes < 0 ? 0u : bytes > 0x7ffffffcll ? 0x7ffffffcu : (uint32_t)bytes), kRawBufferWord3};
}

// One 16-byte copy a lane from memory to LDS chunk wave_chunk + lane.  As
// assembly, because the transposing LDS reads, which the compiler cannot
// tell apart from the copies' destinations, would else each wait for every
// copy in flight (counted in the built code: vmcnt(0) before each; the
// product with row-major B ran at 560 TFLOPS).  It writes no register, and
// lp_wait and lp_barrier count the copies, so nothing else has to know it.  The
// no-ops are the wait that a memory instruction needs after a vector
// instruction has written its scalar operands (five issue slots), which the
// compiler does not see to inside assembly.
__device__ __forceinline__ void lp_copy16(i32x4 r, uint32_t off, i32x4 *wave_chunk)
{
    const uint32_t at = (uint32_t)(uintptr_t)(lds_void_t)wave_chunk;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(at), "v"(off), "s"(r)
                 : "memory", "m0");
}

// Column of C, in a block of 32, that row i of the first operand of a matrix
// instruction feeds.  The instruction hands lane half h the results of rows
// 8 q + 4 h + w, as its values 4 q + w; with this order its values are runs of
// RUN neighbouring columns (16 bytes of C), the two halves' side by side.
template <int RUN>
__device__ __forceinline__ int lp_column(int i)
{
    const int v = 4 * (i >> 3) + (i & 3), h = (i >> 2) & 1;
    return v / RUN * (2 * RUN) + h * RUN + v % RUN;
}

template <int WIDTH>
__device__ __forceinline__ int lp_strided_swizzle(int kr)
{
    return WIDTH >= 128 ? 4 * (kr & 3) : 4 * ((kr >> 1) & 1);
}

// Byte offset, in its operand at slab 0, of the chunk that lane `tid` copies
// as piece j.
template <class T, bool IS_B, bool KS, int RUN>
__device__ __forceinline__ uint32_t lp_offset(const LpOperand &o, int j, int tid, int &kr)
{
    constexpr int W = IS_B ? T::BN : T::BM;
    const int c = tid + j * T::THREADS;
    if constexpr (KS) {
        kr = c / (W / 8);
        return (uint32_t)kr * (uint32_t)o.ld + (uint32_t)((c % (W / 8)) ^ lp_strided_swizzle<W>(kr)) * 16u;
    } else {
        kr = 0;
        const int r = c / T::CPR;
        const int row = min(IS_B ? (r & ~31) + lp_column<RUN>(r & 31) : r, o.rows - 1);
        return (uint32_t)row * (uint32_t)o.ld + (uint32_t)((c % T::CPR) ^ T::swizzle(r)) * 16u;
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
        const int k0 = ((c % T::CPR) ^ T::swizzle(c / T::CPR)) * 8;
        i32x4 v = region[c];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] &= (k0 + 2 * i < left ? 0xffff : 0) | (k0 + 2 * i + 1 < left ? (int)0xffff0000u : 0);
        region[c] = v;
    }
}

// The same for A's 4-bit codes; `left` is a whole number of chunks.
template <class T>
__device__ __forceinline__ void lp_zero_tail4(i32x4 *region, int tid, int left)
{
#pragma unroll
    for (int j = 0; j < T::A_PER_T; ++j) {
        const int c = tid + j * T::THREADS;
        if (((c % T::CPR) ^ T::swizzle(c / T::CPR)) * 32 >= left) region[c] = i32x4{};
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

template <int N>
__device__ __forceinline__ void lp_wait()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

template <class T, int KIND>
struct LpFrags {
    i32x4 a[2][T::MB], b[2][T::NB];
    // 4-bit: scales of this pair of k-steps, and the words of the next one.
    int sa[KIND == kFp4 ? T::MB : 1], sb[KIND == kFp4 ? T::NB : 1];
    unsigned na[KIND == kFp4 ? T::MB : 1], nb[KIND == kFp4 ? T::NB : 1];
};

// Fragment r, of MB + NB, of k-step p.
template <class T, int KIND, bool A_KS, bool B_KS, int RUN>
__device__ __forceinline__ void lp_read(const i32x4 *As, const i32x4 *Bs, int r, int p, int wr, int wc, int lane,
                                        LpFrags<T, KIND> &f)
{
    const int l32 = lane & 31, half = lane >> 5;
    auto contiguous = [&](const i32x4 *region, int row) {
        return region[row * T::CPR + ((2 * p + half) ^ T::swizzle(l32))];
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
    // In the order in which the products of the next step want them.
    if (r == 0 || (r >= 2 && r > T::NB)) {
        const int mb = r == 0 ? 0 : r - T::NB, row = wr * T::WM + mb * 32;
        if constexpr (A_KS) f.a[p & 1][mb] = strided(As, T::BM, row + 4 * quad, lp_strided_swizzle<T::BM>(krow));
        else f.a[p & 1][mb] = contiguous(As, row + l32);
    } else {
        const int nb = r - 1, row = wc * T::WN + nb * 32;
        if constexpr (B_KS)
            f.b[p & 1][nb] = strided(Bs, T::BN, row + lp_column<RUN>(4 * quad),
                                     lp_strided_swizzle<T::BN>(krow));
        else f.b[p & 1][nb] = contiguous(Bs, row + l32);
    }
}

// Scale words of k-block q of a slab, k-steps 2 q and 2 q + 1.
template <class T, int KIND, int RUN>
__device__ __forceinline__ void lp_read_scales(const i32x4 *Ss, int q, int wr, int wc, int lane, LpFrags<T, KIND> &f)
{
    if constexpr (KIND == kFp4) {
        const int l32 = lane & 31;
        const unsigned *wa = reinterpret_cast<const unsigned *>(Ss) + q * T::BM;
        const unsigned *wb = reinterpret_cast<const unsigned *>(Ss) + T::SCALE_WAVES_A * 256 + q * T::BN;
        const int b_row = lp_column<RUN>(l32);
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb) f.na[mb] = wa[wr * T::WM + mb * 32 + l32];
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) f.nb[nb] = wb[wc * T::WN + nb * 32 + b_row];
    }
}

// The words just read become those in use, shifted so that the lane's block
// of the pair's first step is byte 0 and of its second byte 2.
template <class T, int KIND>
__device__ __forceinline__ void lp_take_scales(int lane, LpFrags<T, KIND> &f)
{
    if constexpr (KIND == kFp4) {
        const int shift = 8 * (lane >> 5);
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb) f.sa[mb] = (int)(f.na[mb] >> shift);
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) f.sb[nb] = (int)(f.nb[nb] >> shift);
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
    } else if constexpr (KIND == kF16) {
        acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a),
                                                             acc[mb][nb], 0, 0, 0);
    } else if constexpr (KIND == kInt8) {
        // (The sums' bits, in the registers of the other kinds: lp_scale makes
        // numbers of them.)
        acc[mb][nb] = __builtin_bit_cast(f32x16, __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, __builtin_bit_cast(i32x16, acc[mb][nb]),
                                                                                      0, 0, 0));
    } else {
        const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
        if (p & 1)
            acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[mb][nb], 4, 4, 2,
                                                                          f.sb[nb], 2, f.sa[mb]);
        else
            acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[mb][nb], 4, 4, 0,
                                                                          f.sb[nb], 0, f.sa[mb]);
    }
}

// Bytes of a row of B (and, but for integers, of A) that are its own.
template <int KIND>
__device__ __forceinline__ long long lp_row_bytes(const GroupedArgs &g)
{
    return KIND == kFp4 ? (long long)g.a_kblocks * 64 : KIND == kInt8 ? g.ldb : (long long)g.k * 2;
}

// What a tile needs of its operands.
struct LpProblem {
    LpOperand a, b;
    const u8 *a_scales, *b_scales;     // of the tile's first rows, k-block 0
    long long a_scale_bytes, b_scale_bytes;   // extents
    long long a_scale_step, b_scale_step;     // bytes from k-block to k-block
    int k;                             // contraction (4-bit: kp; planes: of all segments)
    // Planes: the contraction goes over up to three pairs of planes in turn, `segment`
    // slabs each; where the second and the third lie from p on.
    int segment;
    long long a_second, a_third, b_second, b_third;
    // Planes: of every `share` neighbouring slabs this workgroup's part of the
    // wavefronts multiplies number `turn`.
    int share, turn;
};

// REG: operands whose rows are not 4-byte aligned (bfloat16 rows of odd
// length) cannot be copied straight into LDS; their chunks pass through
// registers, one slab ahead, with the tails made zero on the way.
template <class T, int KIND, bool A_KS, bool B_KS, int RUN, bool REG = false>
struct LpLoop {
    static_assert(!REG || (KIND == kBf16 && T::STAGES == 2), "register copies: bfloat16, two stages");
    static constexpr int KSLAB = T::CPR * lp_values(KIND);
    // Scale words of a slab: [A, B][k-block][row], four a chunk.  The first
    // wavefronts copy A's, the next ones B's, and further ones the same again:
    // a branch around the copy would split the slab's schedule.
    static constexpr int SCALE_COPIES = T::SCALE_WAVES_A + T::SCALE_WAVES_B;
    static_assert(KIND != kFp4 || T::THREADS / 64 >= SCALE_COPIES, "one copy of scales a wavefront");
    const LpProblem &q;
    i32x4 *lds;
    int tid, lane, wave, wr, wc;
    int slabs, tail;               // slabs; elements of the last one, 0: full
    uint32_t a_off[T::A_PER_T], b_off[T::B_PER_T];
    int a_kr[T::A_PER_T], b_kr[T::B_PER_T];
    i32x4 regs[REG ? T::PIECES : 1];
    uint32_t s_off;                // 4-bit: the lane's scale chunk
    int s_wave;
    bool s_is_a;

    __device__ __forceinline__ i32x4 *stage(int s) const { return lds + s * T::stage_chunks(KIND); }

    __device__ __forceinline__ void setup()
    {
#pragma unroll
        for (int j = 0; j < T::A_PER_T; ++j) a_off[j] = lp_offset<T, false, A_KS, RUN>(q.a, j, tid, a_kr[j]);
#pragma unroll
        for (int j = 0; j < T::B_PER_T; ++j) b_off[j] = lp_offset<T, true, B_KS, RUN>(q.b, j, tid, b_kr[j]);
        if constexpr (KIND == kFp4) {
            s_wave = wave % SCALE_COPIES;
            s_is_a = s_wave < T::SCALE_WAVES_A;
            const int per = s_is_a ? T::BM / 4 : T::BN / 4;        // chunks of a k-block (128 columns)
            const int c = (s_wave - (s_is_a ? 0 : T::SCALE_WAVES_A)) * 64 + lane;
            const uint32_t step = (uint32_t)(s_is_a ? q.a_scale_step : q.b_scale_step);
            s_off = c >= T::KBLOCKS * per ? kOobOffset : (c < per ? 0u : step) + (uint32_t)(c < per ? c : c - per) * 16u;
        }
        slabs = (q.k + KSLAB - 1) / KSLAB;
        tail = q.k % KSLAB;
        if constexpr (KIND == kF16) slabs = (slabs + q.share - 1) / q.share;
    }

    // Copies of slab kt: descriptors of the operands from the slab's first k on.
    struct Source {
        i32x4 a, b, s;
        i32x4 *st;
        int left;                  // elements from the slab's first on
    };
    __device__ __forceinline__ Source source(int kt) const
    {
        Source c;
        c.st = stage(kt % T::STAGES);
        c.left = q.k - kt * KSLAB;
        int at = kt;
        long long pa = 0, pb = 0, none = 0;
        if constexpr (KIND == kF16) {
            at = kt * q.share + q.turn;
            // (Past the last slab, where they are not whole shares: no bytes, zeros.)
            none = at * KSLAB >= q.k ? 1ll << 62 : 0;
            if (at >= q.segment) at -= q.segment, pa = q.a_second, pb = q.b_second;
            if (at >= q.segment) at -= q.segment, pa = q.a_third, pb = q.b_third;
        }
        const long long sa = pa + (A_KS ? (long long)at * KSLAB * q.a.ld : (long long)at * (T::CPR * 16));
        const long long sb = pb + (B_KS ? (long long)at * KSLAB * q.b.ld : (long long)at * (T::CPR * 16));
        c.a = lp_rsrc(q.a.p + sa, q.a.bytes - sa - none);
        c.b = lp_rsrc(q.b.p + sb, q.b.bytes - sb - none);
        if constexpr (KIND == kFp4) {
            const long long k = (long long)(T::KBLOCKS * kt) * (s_is_a ? q.a_scale_step : q.b_scale_step);
            c.s = lp_rsrc(reinterpret_cast<const char *>(s_is_a ? q.a_scales : q.b_scales) + k,
                          (s_is_a ? q.a_scale_bytes : q.b_scale_bytes) - k);
        }
        return c;
    }
    static constexpr int COPIES = T::PIECES + (KIND == kFp4 ? 1 : 0);

    // Copy i, of COPIES.
    __device__ __forceinline__ void copy(const Source &c, int i) const
    {
        if (i < T::A_PER_T) {
            lp_copy16(c.a, A_KS && a_kr[i] >= c.left ? kOobOffset : a_off[i], c.st + i * T::THREADS + wave * 64);
        } else if (i < T::PIECES) {
            const int j = i - T::A_PER_T;
            lp_copy16(c.b, B_KS && b_kr[j] >= c.left ? kOobOffset : b_off[j],
                      c.st + T::A_CHUNKS + j * T::THREADS + wave * 64);
        } else if constexpr (KIND == kFp4) {
            // A block past the last one is past the extents and reads as zero.
            lp_copy16(c.s, s_off, c.st + T::A_CHUNKS + T::B_CHUNKS + s_wave * 64);
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
            const int k0 = ((c % T::CPR) ^ T::swizzle(c / T::CPR)) * 8;
            return load_chunk(reinterpret_cast<const __bf16 *>(o.p + (long long)kt * (T::CPR * 16) + off), left - k0);
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

    static constexpr int READS = T::MB + T::NB;
    __device__ __forceinline__ void read(int kt, int p, int r, LpFrags<T, KIND> &f) const
    {
        const i32x4 *const st = stage(kt % T::STAGES);
        if (KIND == kFp4 && r == 0 && (p & 1) == 0)
            lp_read_scales<T, KIND, RUN>(st + T::A_CHUNKS + T::B_CHUNKS, p >> 1, wr, wc, lane, f);
        lp_read<T, KIND, A_KS, B_KS, RUN>(st, st + T::A_CHUNKS, r, p, wr, wc, lane, f);
    }

    // The products of k-step p, one read of the next step (slab kt_next, step
    // p_next) and, in COPY's step, one copy after each.
    template <bool READ, bool COPY>
    __device__ __forceinline__ void step(int p, int kt_next, int p_next, const Source &c, LpFrags<T, KIND> &f,
                                         f32x16 (&acc)[T::MB][T::NB]) const
    {
        constexpr int NM = T::MB * T::NB;
        if ((p & 1) == 0) lp_take_scales<T, KIND>(lane, f);
        constexpr int RPM = (READS + NM - 1) / NM, CPM = (COPIES + NM - 1) / NM;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            lp_mfma<T, KIND>(i, p, f, acc);
            if constexpr (READ)
#pragma unroll
                for (int r = i * RPM; r < (i + 1) * RPM && r < READS; ++r) read(kt_next, p_next, r, f);
            if constexpr (COPY)
#pragma unroll
                for (int j = i * CPM; j < (i + 1) * CPM && j < COPIES; ++j) copy(c, j);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // One slab.  COPY: the slab STAGES ahead is copied, as soon as this one's
    // last fragments are read.  LAST: there is no next slab.
    template <bool COPY, bool LAST>
    __device__ __forceinline__ void slab(int kt, LpFrags<T, KIND> &f, f32x16 (&acc)[T::MB][T::NB])
    {
        // 4-bit slabs of two k-blocks: the last one of an odd number holds
        // half the steps' values; the others' codes are another row's.
        const bool half_slab = KIND == kFp4 && LAST && tail != 0;
        Source c;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int p = 0; p + 1 < T::STEPS; ++p)
            if (p < T::STEPS / 2 || !half_slab) step<true, false>(p, kt, p + 1, c, f, acc);
        __builtin_amdgcn_s_setprio(0);
        if constexpr (!LAST) {
            if constexpr (REG) {
                store(kt + 1);
                lp_barrier<63>();
            } else if constexpr (COPY) {
                lp_barrier<(T::STAGES - 2) * COPIES>();
            } else {
                // The slabs after the next one may still be on their way.
                if (T::STAGES > 3 && slabs - 2 - kt >= 2) lp_wait<2 * COPIES>();
                else if (T::STAGES > 2 && slabs - 2 - kt >= 1) lp_wait<COPIES>();
                else lp_wait<0>();
                if (kt + 2 == slabs && tail != 0) fix_tail(kt + 1);
                lp_barrier<63>();
            }
            if constexpr (COPY && REG) load(kt + 2);
            if constexpr (COPY && !REG) c = source(kt + T::STAGES);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
            step<true, COPY && !REG>(T::STEPS - 1, kt + 1, 0, c, f, acc);
        } else if (!half_slab) {
            step<false, false>(T::STEPS - 1, 0, 0, c, f, acc);
        }
    }

    __device__ __forceinline__ void run(f32x16 (&acc)[T::MB][T::NB])
    {
        setup();
        if (slabs == 0) return;
        LpFrags<T, KIND> f;
        if constexpr (REG) {
            load(0);
            store(0);
            if (slabs > 1) load(1);
            lp_barrier<63>();
        } else {
#pragma unroll
            for (int s = 0; s < T::STAGES; ++s)
                if (s < slabs) {
                    const Source c = source(s);
#pragma unroll
                    for (int i = 0; i < COPIES; ++i) copy(c, i);
                }
            if (slabs == 1) {
                lp_wait<0>();
                if (tail) fix_tail(0);
                lp_barrier<63>();
            } else if (slabs >= T::STAGES) {
                lp_barrier<(T::STAGES - 1) * COPIES>();
            } else {
                lp_barrier<0>();
            }
        }
#pragma unroll
        for (int r = 0; r < READS; ++r) read(0, 0, r, f);
        int kt = 0;
        for (; kt + T::STAGES < slabs; ++kt) slab<true, false>(kt, f, acc);
        for (; kt + 1 < slabs; ++kt) slab<false, false>(kt, f, acc);
        slab<false, true>(kt, f, acc);
    }
};

// C's 32 x 32 blocks: lane l32 holds row l32 of the block, in runs of RUN
// columns.  WIDE: rows and column runs of C are 16-byte aligned and n is a
// multiple of RUN.  Bias and activation are passes of their own over the
// accumulators, so that a call without them jumps over two pieces of code
// and not, element by element, through all of it: with the activation's
// branch at each element the epilogue waited for instructions (34000 cycles a
// tile of 256 x 256).
template <class T, class E, bool WIDE>
__device__ __forceinline__ void lp_store(char *c, long long ldc, int rows, int cols, const float *bias, int act, int wr,
                                         int wc, int lane, f32x16 (&acc)[T::MB][T::NB])
{
    constexpr int RUN = 16 / sizeof(E);
    const int l32 = lane & 31, half = lane >> 5;
    const int col0 = wc * T::WN + half * RUN;
    if (bias) {
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int col = col0 + nb * 32 + v / RUN * (2 * RUN) + v % RUN;
                const float b = col < cols ? bias[col] : 0.0f;
#pragma unroll
                for (int mb = 0; mb < T::MB; ++mb) acc[mb][nb][v] += b;
            }
    }
    if (act == 1) {
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
            for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[mb][nb][v] = activate(acc[mb][nb][v], 1);
    } else if (act == 2) {
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
            for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[mb][nb][v] = gelu_rcp(acc[mb][nb][v]);
    }
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) {
        const int row = wr * T::WM + mb * 32 + l32;
        if (row >= rows) continue;
        E *const p = reinterpret_cast<E *>(c + row * ldc);
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
            for (int v0 = 0; v0 < 16; v0 += RUN) {
                const int col = col0 + nb * 32 + v0 * 2;
                // One rounding, to the type of C.
                struct alignas(16) Run {
                    E e[RUN];
                } r;
#pragma unroll
                for (int i = 0; i < RUN; ++i) r.e[i] = (E)acc[mb][nb][v0 + i];
                if constexpr (WIDE) {
                    if (col < cols) *reinterpret_cast<Run *>(p + col) = r;
                } else if (col + RUN <= cols) {
                    // (Wide stores need no alignment here; 2049 x 4099 x 2049 of 32 experts in
                    // 8 bits, 32-bit results: 126 us element by element.)
                    struct __attribute__((packed, aligned(sizeof(E)))) Loose {
                        E e[RUN];
                    } t;
#pragma unroll
                    for (int i = 0; i < RUN; ++i) t.e[i] = r.e[i];
                    *reinterpret_cast<Loose *>(p + col) = t;
                } else {
#pragma unroll
                    for (int i = 0; i < RUN; ++i)
                        if (col + i < cols) p[col + i] = r.e[i];
                }
            }
    }
}

// Integer sums times their rows' and columns' scales, as 32-bit numbers.
template <class T, class E>
__device__ __forceinline__ void lp_scale(const GroupedArgs &g, int expert, int row, int rows, int col, int wr, int wc, int lane,
                                         f32x16 (&acc)[T::MB][T::NB])
{
    constexpr int RUN = 16 / sizeof(E);
    const float *const sa = reinterpret_cast<const float *>(g.a_scales) + row;
    const float *const sb = reinterpret_cast<const float *>(g.b_scales) + (long long)expert * g.n;
    float of_row[T::MB];
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) of_row[mb] = sa[min(wr * T::WM + mb * 32 + (lane & 31), rows - 1)];
    const int col0 = col + wc * T::WN + (lane >> 5) * RUN;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) {
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const float b = sb[min(col0 + nb * 32 + v / RUN * (2 * RUN) + v % RUN, g.n - 1)];
#pragma unroll
            for (int mb = 0; mb < T::MB; ++mb) acc[mb][nb][v] = (float)__float_as_int(acc[mb][nb][v]) * of_row[mb] * b;
            if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb) asm volatile("" : "+v"(acc[mb][nb]));
    }
}

// One tile of C_e = act(A_e . B_e + bias_e): rows from `row` on, of which the
// expert has `rows`, columns from col on.  Expert -1: zeros.
template <class T, int KIND, bool B_KS, class E, bool WIDE, bool REG = false>
__device__ __forceinline__ void lp_tile(const GroupedArgs &g, i32x4 *lds, int tid, int lane, int wave, int expert,
                                        int row, int rows, int col)
{
    const int cols = g.n - col;
    const int wr = wave % T::WAVES_M, wc = wave / T::WAVES_M;
    f32x16 acc[T::MB][T::NB];
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
    if (expert >= 0) {
        LpProblem q;
        const long long row_bytes = lp_row_bytes<KIND>(g);
        q.a = {g.A + row * g.lda, (g.m - 1 - row) * g.lda + (KIND == kInt8 ? g.lda : row_bytes), (int)g.lda, g.m - row};
        const char *const b = g.B + expert * g.expert_stride;
        if constexpr (B_KS)
            q.b = {b + (long long)col * 2, (long long)(g.k - 1) * g.ldb + (long long)cols * 2, (int)g.ldb, cols};
        else
            q.b = {b + col * g.ldb, (cols - 1) * g.ldb + row_bytes, (int)g.ldb, cols};
        q.k = KIND == kBf16 ? g.k : g.a_kblocks * 128;
        if constexpr (KIND == kFp4) {
            q.a_scales = g.a_scales + (long long)row * 4;
            q.a_scale_step = (long long)g.m * 4;
            q.a_scale_bytes = g.a_kblocks * q.a_scale_step - (long long)row * 4;
            q.b_scale_step = (long long)g.n * 4;
            q.b_scales = g.b_scales + expert * (g.a_kblocks * q.b_scale_step) + (long long)col * 4;
            q.b_scale_bytes = g.a_kblocks * q.b_scale_step - (long long)col * 4;
        }
        LpLoop<T, KIND, false, B_KS, 16 / sizeof(E), REG> loop{q, lds, tid, lane, wave, wr, wc};
        loop.run(acc);
        if constexpr (KIND == kInt8) lp_scale<T, E>(g, expert, row, rows, col, wr, wc, lane, acc);
    }
    const float *bias = g.bias && expert >= 0 ? g.bias + expert * g.bias_stride + col : nullptr;
    lp_store<T, E, WIDE>(g.C + row * g.ldc + (long long)col * sizeof(E), g.ldc, rows, cols, bias, expert < 0 ? 0 : g.act,
                         wr, wc, lane, acc);
}

// One tile of dB_e = A_e^T . G_e: g.m rows of A (g.k columns) and G (g.n
// columns), the expert's lo .. hi; zeros where it has none.
template <class T, bool WIDE, bool REG = false>
__device__ __forceinline__ void lp_grad_tile(const GroupedArgs &g, i32x4 *lds, int tid, int lane, int wave, int expert,
                                             int lo, int hi, int row, int col)
{
    const int wr = wave % T::WAVES_M, wc = wave / T::WAVES_M;
    f32x16 acc[T::MB][T::NB];
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
    LpProblem q;
    const long long last = hi - lo - 1;      // -1: no rows, no bytes are read
    q.a = {g.A + lo * g.lda + (long long)row * 2, last * g.lda + (long long)(g.k - row) * 2, (int)g.lda, g.k - row};
    q.b = {g.B + lo * g.ldb + (long long)col * 2, last * g.ldb + (long long)(g.n - col) * 2, (int)g.ldb, g.n - col};
    q.k = hi - lo;
    LpLoop<T, kBf16, true, true, 8, REG> loop{q, lds, tid, lane, wave, wr, wc};
    loop.run(acc);
    lp_store<T, __bf16, WIDE>(g.C + expert * g.expert_stride + row * g.ldc + (long long)col * 2, g.ldc, g.k - row,
                              g.n - col, nullptr, 0, wr, wc, lane, acc);
}

template <class T, int KIND, bool B_KS, class E, bool WIDE, bool REG = false>
__global__ __launch_bounds__(T::THREADS) void lp_grouped_kernel(GroupedArgs g)
{
    __shared__ i32x4 lds[T::STAGES * T::stage_chunks(KIND)];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    RowTile rt;
    int tn;
    if (!find_tile<T::BM>(g, blockIdx.x, lane, rt, tn)) return;
    lp_tile<T, KIND, B_KS, E, WIDE, REG>(g, lds, tid, lane, wave, rt.expert, rt.row, rt.rows, tn * T::BN);
}

template <class T, bool WIDE, bool REG = false>
__global__ __launch_bounds__(T::THREADS) void lp_weight_grad_kernel(GroupedArgs g)
{
    __shared__ i32x4 lds[T::STAGES * T::stage_chunks(kBf16)];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    GradTile t;
    if (!grad_tile(g, blockIdx.x % g.num_xcd, blockIdx.x / g.num_xcd, t)) return;
    const Rows rows = entry_rows(g, t.expert);
    lp_grad_tile<T, WIDE, REG>(g, lds, tid, lane, wave, t.expert, __builtin_amdgcn_readfirstlane(rows.lo),
                               __builtin_amdgcn_readfirstlane(rows.hi), t.tm * T::BM, t.tn * T::BN);
}

}  // namespace gemmf32
