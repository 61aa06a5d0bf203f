// The grouped bfloat16 and 4-bit products as one continuous pipeline: a
// workgroup a CU takes tile after tile, and the copies run ahead of the
// products across tile borders, so that a tile's first slabs arrive while the
// tile before it is still multiplied and stored.  (One workgroup a tile left
// 13 us a 256 x 256 tile in which nothing multiplied: its search, its first
// copies and its stores; 10 % at k = 4096, 21 % at 2048.)
//
// Layouts, fragments and products are those of lp_gemm.hpp.  A stage is
// refilled as soon as the barrier has freed it: three quarters of its copies
// among the products behind the barrier, the rest among the next slab's
// first.  Measured in TFLOPS on 16384 x 14336 x 4096 in bfloat16, normal
// values, 8 experts: so 1154; all copies behind the barrier 1143; slabs of 64
// instead of 128 bytes a row, four stages deep, 1054; 4 instead of 8
// wavefronts 1046; touching lines two slabs ahead of their copies 1139.
//
// What bounds it: by the counters (profiles/expert_layer_counters.md) the matrix
// cores are busy 63 % of the time there, 50 and 44 % in the two products of a
// training step of 8192 rows over 16 uneven experts (k = 2048, n = 4096), 40 % in
// its weight gradient and 50 % in 4 bits (8192 rows, one matrix).  The clock falls
// with the operands' bits (a library product of the same sizes 1339 with normal
// values, 2062 with zeros; this kernel with one expert 1266 and 1406).  The
// copies cost: the same products without them ran at 1331 and 1944 (n = 8192).
// It is not LDS reads (LDS serves them a quarter of the time), nor conflicts of
// banks (none counted).  One expert takes 1520 us, eight 1800: their half-empty
// last tiles explain about 6 %, the rest is not explained.  Rows that are not a
// power of two of bytes apart run 6 % faster (k = 4160 for 4096).
//
// Every slab issues the same number of copies, so one count of copies in
// flight serves every wait: past the last tile they read nothing (a
// descriptor of no bytes).  A tile's stores count too: copies return in order
// among themselves, so that at most n operations in flight leaves at most the
// n newest copies, whatever the stores do.
#pragma once

#include "lp_gemm.hpp"

namespace gemmf32 {

constexpr int kPipeMaxGroups = 1022;       // entries of the tile table in LDS, less two

// What a tile is: rows of A and C, columns of B and C, and its contraction.
struct LpJob {
    int expert, row, rows, col;            // weight gradient: row, col of dB; rows: of the expert
    int k;                                 // contraction; 0: C is zero
};

// Bias and activation, over the accumulators.
template <class T, class E>
__device__ __forceinline__ void lp_epilogue(int cols, const float *bias, int act, int wc, int lane,
                                            f32x16 (&acc)[T::MB][T::NB])
{
    constexpr int RUN = 16 / sizeof(E);
    const int col0 = wc * T::WN + (lane >> 5) * RUN;
    if (bias) {
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(bias, (uint32_t)cols * 4u);
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const float b = buf_load_x1(rb, (uint32_t)(col0 + nb * 32 + v / RUN * (2 * RUN) + v % RUN) * 4u);
#pragma unroll
                for (int mb = 0; mb < T::MB; ++mb) acc[mb][nb][v] += b;
                if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int mb = 0; mb < T::MB; ++mb) asm volatile("" : "+v"(acc[mb][nb]));
        }
    }
    if (act) {
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
            for (int mb = 0; mb < T::MB; ++mb) {
                // A block at a time, in the registers that it has: across the
                // branch the compiler else moved the accumulators around.
                if (act == 1) {
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[mb][nb][v] = activate(acc[mb][nb][v], 1);
                } else {
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        acc[mb][nb][v] = gelu_rcp(acc[mb][nb][v]);
                        if (v % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                    }
                }
                asm volatile("" : "+v"(acc[mb][nb]));
            }
    }
}

// GRAD: the weight gradient (both operands k strided).
template <class T, int KIND, bool GRAD, bool B_KS, class E, bool WIDE>
struct LpPipe {
    static constexpr bool A_KS = GRAD;
    static constexpr int RUN = 16 / sizeof(E);
    static constexpr int S = T::STAGES, KSLAB = T::CPR * (KIND == kFp4 ? 32 : 8);
    static constexpr int STAGE = T::stage_chunks(KIND);              // chunks
    static constexpr int COPIES = T::PIECES + (KIND == kFp4 ? 1 : 0);
    static constexpr int FIRST = COPIES * 3 / 4;                     // copies right behind the barrier
    static constexpr int READS = T::MB + T::NB;
    static constexpr int SCALE_COPIES = T::SCALE_WAVES_A + T::SCALE_WAVES_B;
    static_assert((S - 1) * COPIES <= 63, "copies in flight fit the counter");

    const GroupedArgs &g;
    i32x4 *lds;
    const int *table;          // LDS: running sums of row tiles, then first rows, then rows (not GRAD)
    int entries, total;        // of the table; tiles
    int tid, lane, wave, wr, wc;

    // --- the sequence of tiles -------------------------------------------------

    // Tile number `logical` of all (weight gradient: of this XCD's; expert -1: none).
    __device__ __forceinline__ LpJob job(int logical) const
    {
        LpJob j;
        int tm;
        if constexpr (GRAD) {
            GradTile t;
            if (!grad_tile(g, blockIdx.x % g.num_xcd, logical, t)) return LpJob{-1, 0, 0, 0, 0};
            j.expert = t.expert;
            tm = t.tm;
            j.col = t.tn * T::BN;
            const Rows rows = entry_rows(g, j.expert);
            j.row = __builtin_amdgcn_readfirstlane(rows.lo);
            j.k = __builtin_amdgcn_readfirstlane(rows.hi) - j.row;
            j.rows = tm * T::BM;                       // first row of dB
        } else {
            const int rows_all = total / g.tiles_n, width = g.group_m * g.tiles_n;
            const int first = logical / width * g.group_m, size = min(rows_all - first, g.group_m);
            const int r = logical % width;
            tm = first + r % size;
            j.col = r / size * T::BN;
            int base = 0;
            unsigned long long past;
            while (!(past = __ballot(base + lane < entries && table[min(base + lane, entries - 1)] > tm))) base += 64;
            const int at = base + __builtin_ctzll(past);
            const int before = at ? __builtin_amdgcn_readfirstlane(table[at - 1]) : 0;
            const int skip = (tm - before) * T::BM;
            j.row = __builtin_amdgcn_readfirstlane(table[entries + at]) + skip;
            j.rows = __builtin_amdgcn_readfirstlane(table[2 * entries + at]) - skip;
            j.expert = g.offsets && at >= g.groups ? -1 : at;
            j.k = j.expert < 0 ? 0 : KIND == kFp4 ? g.a_kblocks * 128 : g.k;
        }
        return j;
    }

    // --- copies -----------------------------------------------------------------

    int next_tile, tile_step, tile_end;     // tiles of this workgroup still to copy
    const char *pa, *pb, *ps;               // first bytes of the slab to copy, and what lies from there on
    long long la, lb, ls;
    long long da, db, ds;                   // to the next slab
    int left;                               // elements of the contraction from this slab on; <= 0: the tile is done
    int put;                                // stage that the next copies go to, in chunks
    uint32_t a_off[T::A_PER_T], b_off[T::B_PER_T], s_off;
    bool s_is_a;
    int s_wave;

    __device__ __forceinline__ void begin(const LpJob &j)
    {
        LpOperand a, b;
        left = j.k;
        if constexpr (GRAD) {
            const long long last = j.k - 1;
            a = {g.A + j.row * g.lda + (long long)j.rows * 2, last * g.lda + (long long)(g.k - j.rows) * 2, (int)g.lda, 0};
            b = {g.B + j.row * g.ldb + (long long)j.col * 2, last * g.ldb + (long long)(g.n - j.col) * 2, (int)g.ldb, 0};
        } else {
            const long long row_bytes = KIND == kFp4 ? (long long)g.a_kblocks * 64 : (long long)g.k * 2;
            const int cols = g.n - j.col;
            const char *const w = g.B + j.expert * g.expert_stride;
            a = {g.A + j.row * g.lda, (g.m - 1 - j.row) * g.lda + row_bytes, (int)g.lda, g.m - j.row};
            if constexpr (B_KS)
                b = {w + (long long)j.col * 2, (long long)(g.k - 1) * g.ldb + (long long)cols * 2, (int)g.ldb, cols};
            else
                b = {w + j.col * g.ldb, (cols - 1) * g.ldb + row_bytes, (int)g.ldb, cols};
        }
        // (Opaque, once a tile: the places in the tile would else be held in
        // registers through all products.)
        int kr, t = tid;
        asm volatile("" : "+v"(t));
#pragma unroll
        for (int i = 0; i < T::A_PER_T; ++i) a_off[i] = lp_offset<T, false, A_KS, RUN>(a, i, t, kr);
#pragma unroll
        for (int i = 0; i < T::B_PER_T; ++i) b_off[i] = lp_offset<T, true, B_KS, RUN>(b, i, t, kr);
        pa = a.p, la = a.bytes, da = A_KS ? (long long)KSLAB * a.ld : T::CPR * 16;
        pb = b.p, lb = b.bytes, db = B_KS ? (long long)KSLAB * b.ld : T::CPR * 16;
        if constexpr (KIND == kFp4) {
            const long long step = (long long)(s_is_a ? g.m : g.n) * 4, skip = (long long)(s_is_a ? j.row : j.col) * 4;
            ps = reinterpret_cast<const char *>(s_is_a ? g.a_scales : g.b_scales + j.expert * (g.a_kblocks * step)) + skip;
            ls = g.a_kblocks * step - skip;
            ds = T::KBLOCKS * step;
        }
    }

    // The slab to copy next: the following one of the tile, or the first of
    // the next tile that has any; past the last tile, nothing.
    __device__ __forceinline__ void advance()
    {
        pa += da, la -= da;
        pb += db, lb -= db;
        if constexpr (KIND == kFp4) ps += ds, ls -= ds;
        left -= KSLAB;
        put = put + STAGE == S * STAGE ? 0 : put + STAGE;
        if (left <= 0) next();
    }

    __device__ __forceinline__ void next()
    {
        la = lb = ls = 0;
        da = db = ds = 0;
        left = 0x7fffffff;
        while (next_tile < tile_end) {
            const LpJob j = job(next_tile);
            next_tile += tile_step;
            if (j.k > 0) {
                begin(j);
                break;
            }
        }
    }

    struct Source {
        i32x4 a, b, s;
    };
    __device__ __forceinline__ Source source() const
    {
        Source c;
        c.a = lp_rsrc(pa, la);
        c.b = lp_rsrc(pb, lb);
        if constexpr (KIND == kFp4) c.s = lp_rsrc(ps, ls);
        return c;
    }

    __device__ __forceinline__ void copy(const Source &c, int i) const
    {
        i32x4 *const st = lds + put;
        if (i < T::A_PER_T) {
            const int kr = (tid + i * T::THREADS) / (T::BM / 8);
            lp_copy16(c.a, A_KS && kr >= left ? kOobOffset : a_off[i], st + i * T::THREADS + wave * 64);
        } else if (i < T::PIECES) {
            const int j = i - T::A_PER_T, kr = (tid + j * T::THREADS) / (T::BN / 8);
            lp_copy16(c.b, B_KS && kr >= left ? kOobOffset : b_off[j],
                      st + T::A_CHUNKS + j * T::THREADS + wave * 64);
        } else if constexpr (KIND == kFp4) {
            lp_copy16(c.s, s_off, st + T::A_CHUNKS + T::B_CHUNKS + s_wave * 64);
        }
    }

    // --- products ---------------------------------------------------------------

    int get;                                // stage of the slab in work, in chunks

    __device__ __forceinline__ void read(int at, int p, int r, LpFrags<T, KIND> &f) const
    {
        const i32x4 *const st = lds + at;
        if (KIND == kFp4 && r == 0 && (p & 1) == 0)
            lp_read_scales<T, KIND, RUN>(st + T::A_CHUNKS + T::B_CHUNKS, p >> 1, wr, wc, lane, f);
        lp_read<T, KIND, A_KS, B_KS, RUN>(st, st + T::A_CHUNKS, r, p, wr, wc, lane, f);
    }

    // The products of k-step p, with the reads of the next step and copies
    // [C0, C1) among them.
    template <int C0, int C1, bool READ = true>
    __device__ __forceinline__ void step(int p, int at, int p_next, const Source &c, LpFrags<T, KIND> &f,
                                         f32x16 (&acc)[T::MB][T::NB]) const
    {
        constexpr int NM = T::MB * T::NB;
        constexpr int RPM = (READS + NM - 1) / NM;
        if ((p & 1) == 0) lp_take_scales<T, KIND>(lane, f);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            lp_mfma<T, KIND>(i, p, f, acc);
#pragma unroll
            for (int r = i * RPM; r < (i + 1) * RPM && r < READS; ++r)
                if constexpr (READ) read(at, p_next, r, f);
#pragma unroll
            for (int j = C0; j < C1; ++j)
                if ((j - C0) * NM / (C1 - C0) == i) copy(c, j);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    __device__ __forceinline__ void fix_tail(int at, int elements) const
    {
        // (Opaque: the masks would else be held in registers all along.)
        int t = tid;
        asm volatile("" : "+v"(t));
        if constexpr (KIND == kFp4) {
            // Half a slab: zero codes in A, for B's are finite, and so are the
            // scales that are read past the last k-block (as zero).
            lp_zero_tail4<T>(lds + at, t, elements);
        } else {
            if constexpr (!A_KS) lp_zero_tail<T, false>(lds + at, t, elements);
            if constexpr (!B_KS) lp_zero_tail<T, true>(lds + at + T::A_CHUNKS, t, elements);
        }
    }

    // One slab: the products of stage `get`, the last quarter of the copies
    // under way, and behind the barrier the first three of the next ones.
    // fix: elements of the next slab, if fewer than it has room for (else 0).
    // LAST: of its tile; the next tile reads its own first fragments, so that
    // the epilogue has their registers.
    template <bool FIX, bool LAST>
    __device__ __forceinline__ void slab(int fix, Source &c, LpFrags<T, KIND> &f, f32x16 (&acc)[T::MB][T::NB])
    {
        const int now = get, then = get + STAGE == S * STAGE ? 0 : get + STAGE;
        get = then;
        __builtin_amdgcn_s_setprio(1);
        step<FIRST, COPIES>(0, now, 1, c, f, acc);
#pragma unroll
        for (int p = 1; p + 1 < T::STEPS; ++p) step<0, 0>(p, now, p + 1, c, f, acc);
        __builtin_amdgcn_s_setprio(0);
        // The products stay on this side of the branches.
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < T::NB; ++nb) asm volatile("" : "+v"(acc[mb][nb]));
        advance();
        c = source();
        if (FIX && fix) {
            lp_wait<0>();
            fix_tail(then, fix);
            lp_barrier<63>();
        } else {
            lp_barrier<0>();
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        step<0, FIRST, !LAST>(T::STEPS - 1, then, 0, c, f, acc);
        __builtin_amdgcn_s_setprio(0);
    }

    // A slab of a wavefront whose rows are past the tile's last: its copies
    // and the barrier.
    template <bool FIX>
    __device__ __forceinline__ void idle_slab(int fix, Source &c)
    {
        const int then = get + STAGE == S * STAGE ? 0 : get + STAGE;
        get = then;
#pragma unroll
        for (int j = FIRST; j < COPIES; ++j) copy(c, j);
        advance();
        c = source();
        if (FIX && fix) {
            lp_wait<0>();
            fix_tail(then, fix);
            lp_barrier<63>();
        } else {
            lp_barrier<0>();
        }
#pragma unroll
        for (int j = 0; j < FIRST; ++j) copy(c, j);
    }

    __device__ __forceinline__ void run()
    {
        // Tiles of this workgroup: the XCDs share the tiles in contiguous runs
        // (workgroups go to the XCDs in turn), an XCD's workgroups take its
        // tiles in turn.
        const int x = blockIdx.x % g.num_xcd, per = total / g.num_xcd, rem = total % g.num_xcd;
        const int begin = GRAD ? 0 : x * per + min(x, rem);
        const int first = begin + (int)(blockIdx.x / g.num_xcd);
        tile_end = GRAD ? total : (x + 1) * per + min(x + 1, rem);
        tile_step = gridDim.x / g.num_xcd;
        next_tile = first;
        // A last round that would leave half the XCD's workgroups without a
        // tile is split: halves of 128 x 256 or quarters of 128 x 128.
        const int last = (tile_end - begin) % tile_step;
        const int parts = 4 * last <= tile_step ? 4 : 2 * last <= tile_step ? 2 : 0;
        if (parts) tile_end -= last;
        if (first < tile_end) whole_tiles(first);
        // The copies past the last tile still write LDS: they are waited for
        // before it is used again, or given back.
        lp_wait<0>();
        const int q = (int)(blockIdx.x / g.num_xcd);
        if (parts && q < parts * last) {
            __syncthreads();
            LpJob j = job(tile_end + q / parts);
            const int part = q % parts;
            if (parts == 4) {
                j.col += part / 2 * 128;
                part_tile<LpTile<128, 128, 2, 4, 2>>(j, part % 2 * 128);
            } else {
                part_tile<LpTile<128, 256, 2, 4, 2>>(j, part * 128);
            }
        }
    }

    // The tile of T2 that begins `down` rows below j's first.
    template <class T2>
    __device__ __forceinline__ void part_tile(LpJob j, int down)
    {
        static_assert(T2::THREADS == T::THREADS && T2::STAGES * T2::stage_chunks(KIND) <= S * STAGE, "the same workgroup");
        if (j.col >= g.n) return;
        if constexpr (GRAD) {
            if (j.expert < 0 || j.rows + down >= g.k) return;
            lp_grad_tile<T2, WIDE>(g, lds, tid, lane, wave, j.expert, j.row, j.row + j.k, j.rows + down, j.col);
        } else {
            if (down >= j.rows) return;
            lp_tile<T2, KIND, B_KS, E, WIDE>(g, lds, tid, lane, wave, j.expert, j.row + down, j.rows - down, j.col);
        }
    }

    __device__ __forceinline__ void whole_tiles(int first)
    {
        if constexpr (KIND == kFp4) {
            s_wave = wave % SCALE_COPIES;
            s_is_a = s_wave < T::SCALE_WAVES_A;
            const int c = (s_wave - (s_is_a ? 0 : T::SCALE_WAVES_A)) * 64 + lane;
            const int per_block = s_is_a ? T::BM / 4 : T::BN / 4;          // chunks of a k-block
            const uint32_t step = (uint32_t)(s_is_a ? g.m : g.n) * 4u;
            s_off = c >= T::KBLOCKS * per_block ? kOobOffset
                                                : c < per_block ? c * 16u : step + (uint32_t)(c - per_block) * 16u;
        }
        put = get = 0;
        next();
        Source c;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            c = source();
#pragma unroll
            for (int i = 0; i < COPIES; ++i) copy(c, i);
            if (s + 1 < S) advance();
        }
        // The last of these slabs' last quarter is issued again by the first
        // slab's work below: the same bytes to the same place.
        bool started = false;
        for (int tile = first; tile < tile_end; tile += tile_step) {
            const LpJob j = job(tile);
            const int slabs = (j.k + KSLAB - 1) / KSLAB;
            const int tail = A_KS && B_KS ? 0 : j.k % KSLAB;
            if (slabs > 0 && !started) {
                started = true;
                lp_wait<(S - 1) * COPIES>();
                if (slabs == 1 && tail) {
                    lp_wait<0>();
                    fix_tail(0, tail);
                }
                lp_barrier<63>();
            }
            if (!GRAD && wr * T::WM >= j.rows) {
                // Nothing to multiply or store: LDS and the power are the other
                // wavefronts' (the three products of 8192 rows over 16 uneven
                // experts, k = 2048, n = 4096: 520 us multiplied all the same,
                // 510 so; with wavefronts of different rows on a SIMD 509, but
                // full tiles then take 1.7 % longer).
                int kt = 0;
                for (; kt + 2 < slabs; ++kt) idle_slab<false>(0, c);
                for (; kt < slabs; ++kt) idle_slab<true>(slabs == 1 || kt + 2 == slabs ? tail : 0, c);
                continue;
            }
            f32x16 acc[T::MB][T::NB];
#pragma unroll
            for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
                for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
            if (slabs > 0) {
                LpFrags<T, KIND> f;
#pragma unroll
                for (int r = 0; r < READS; ++r) read(get, 0, r, f);
                int kt = 0;
                for (; kt + 2 < slabs; ++kt) slab<false, false>(0, c, f, acc);
                if (kt + 1 < slabs) slab<true, false>(tail, c, f, acc);
                // (One slab a tile: the next slab is the next tile's only one.)
                slab<true, true>(slabs == 1 ? tail : 0, c, f, acc);
            }
            // The lane, opaque to the compiler once a tile: the epilogue's
            // offsets would else be computed before the first tile and held
            // in registers through all products.
            int lane_e = lane;
            asm volatile("" : "+v"(lane_e));
            if constexpr (GRAD) {
                if (j.expert < 0) continue;
                char *const out = g.C + j.expert * g.expert_stride + j.rows * g.ldc + (long long)j.col * 2;
                lp_store<T, E, WIDE>(out, g.ldc, g.k - j.rows, g.n - j.col, nullptr, 0, wr, wc, lane_e, acc);
            } else {
                const int cols = g.n - j.col;
                char *const out = g.C + j.row * g.ldc + (long long)j.col * (long long)sizeof(E);
                if (j.expert >= 0)
                    lp_epilogue<T, E>(cols, g.bias ? g.bias + j.expert * g.bias_stride + j.col : nullptr, g.act, wc, lane_e,
                                      acc);
                lp_store<T, E, WIDE>(out, g.ldc, j.rows, cols, nullptr, 0, wr, wc, lane_e, acc);
            }
        }
    }
};

template <class T, int KIND, bool GRAD, bool B_KS, class E, bool WIDE>
__global__ __launch_bounds__(T::THREADS) void lp_pipe_kernel(GroupedArgs g)
{
    constexpr int TABLE = GRAD ? 0 : 3 * (kPipeMaxGroups + 2) / 4;       // chunks
    __shared__ i32x4 lds[T::STAGES * T::stage_chunks(KIND) + TABLE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int entries = g.offsets ? g.groups + 2 : 1;
    int total;
    int *const table = reinterpret_cast<int *>(lds + T::STAGES * T::stage_chunks(KIND));
    if constexpr (GRAD) {
        total = grad_share(g) * g.groups;        // of an XCD
    } else {
        // Every wavefront sums the row tiles for itself and writes the same table.
        int sum = 0;
        for (int b = 0; b < entries; b += 64) {
            const Rows rows = entry_rows(g, b + lane);
            const int s = sum + wave_inclusive_sum((rows.hi - rows.lo + T::BM - 1) / T::BM);
            if (b + lane < entries) {
                table[b + lane] = s;
                table[entries + b + lane] = rows.lo;
                table[2 * entries + b + lane] = rows.hi - rows.lo;
            }
            sum = __builtin_amdgcn_readlane(s, 63);
        }
        total = min(sum, g.tiles_m) * g.tiles_n;
        __syncthreads();
    }
    LpPipe<T, KIND, GRAD, B_KS, E, WIDE> pipe{g, lds, table, entries, total, tid, lane, wave, wave % T::WAVES_M,
                                              wave / T::WAVES_M};
    pipe.run();
}

}  // namespace gemmf32
