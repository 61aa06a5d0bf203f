// The orthogonalising products as one continuous pipeline, as in lp_pipe.hpp: a
// workgroup a CU takes tile after tile, and the copies run ahead of the products
// across their borders.
//
// Tiles that make whole rounds of the workgroups are one workgroup's each.  The
// others' slabs, tile after tile, are shared out evenly over `shared_wgs`
// workgroups: each multiplies its run of slabs, of one tile or several, and writes
// the sums as they are in its registers; a second launch adds each tile's up, in
// the order of the contraction, and stores them.  The part of workgroup w of tile
// t is number w + t: along the run one of the two goes up from part to part.
//
// One MI355X, 256 x 256 tiles: B X of 4096 x 4096 in three pairs of planes, a tile a
// workgroup, 340 us (1.21 PFLOPS; matrix cores 71 % busy).  X X^T of 136 such tiles, all
// shared, 214 and 39 for joining them (136 workgroups with a tile each: 330); what
// the shares cost is their bytes, 64 MiB written and read.  B X of 16 matrices of 2048 x
// 4096, three pairs, 1500 (1.10 PFLOPS, 62 % busy), eight tiles a workgroup: a tile's stores
// leave in a burst of all CUs, and the next tile's first barrier waits for them too (vmcnt
// counts loads and stores together): about 18 us a tile.  Tiles taken in an order rotated
// from workgroup to workgroup, so that bursts do not meet, read more from beyond the L2
// and took 1251 us instead of 991 in two pairs; planes with rows 128 bytes longer than whole KiB made 1 % of it, and lost
// as much at 4096 x 4096.
#pragma once

#include "orthogonal.hpp"

namespace gemmf32 {

struct OrthoJob {
    OrthoTile tile;
    int first, last;       // slabs
    int part;              // of shared tiles, else -1
};

// Slabs of shared tile `t` (of those after the whole ones) begin at t * slabs.
__device__ __forceinline__ int ortho_shared_slabs(const OrthoArgs &g, int tiles) { return (tiles - g.whole) * (g.segments * (g.k / 64)); }

template <class T, bool A_KS, bool B_KS, class E, bool WIDE>
struct OrthoPipe {
    static constexpr bool kPlanes = __is_same(E, _Float16);
    static constexpr int RUN = 16 / sizeof(E);
    static constexpr int S = T::STAGES, STAGE = T::stage_chunks(kF16);
    static constexpr int COPIES = T::PIECES, FIRST = COPIES * 3 / 4, READS = T::MB + T::NB;
    static_assert(S == 2, "a barrier waits for every copy");

    const OrthoArgs &g;
    i32x4 *lds;
    int tid, lane, wave, wr, wc;

    // --- the workgroup's jobs ------------------------------------------------------

    int first_tile, tile_step, whole_jobs, jobs, shared_tile, shared_lo, shared_hi, slabs;

    __device__ __forceinline__ void plan()
    {
        const int tiles = ortho_tiles(g) * g.batch;
        slabs = g.segments * (g.k / 64);
        const int x = blockIdx.x % g.num_xcd, per = g.whole / g.num_xcd, rem = g.whole % g.num_xcd;
        const int q = blockIdx.x / g.num_xcd;
        tile_step = gridDim.x / g.num_xcd;
        first_tile = x * per + min(x, rem) + q;
        const int end = (x + 1) * per + min(x + 1, rem);
        whole_jobs = __builtin_amdgcn_readfirstlane(first_tile < end ? (end - first_tile + tile_step - 1) / tile_step : 0);
        jobs = whole_jobs;
        shared_lo = shared_hi = shared_tile = 0;
        // (XCD by XCD, as the tiles.)
        const int w = xcd_contiguous(blockIdx.x, gridDim.x, g.num_xcd);
        if (kPlanes && g.whole < tiles && w < g.shared_wgs) {
            const long long all = ortho_shared_slabs(g, tiles);
            shared_lo = __builtin_amdgcn_readfirstlane((int)(all * w / g.shared_wgs));
            shared_hi = __builtin_amdgcn_readfirstlane((int)(all * (w + 1) / g.shared_wgs));
            shared_tile = __builtin_amdgcn_readfirstlane(shared_lo / slabs);
            if (shared_lo < shared_hi) jobs += __builtin_amdgcn_readfirstlane((shared_hi - 1) / slabs) - shared_tile + 1;
        }
    }

    __device__ __forceinline__ OrthoJob job(int i) const
    {
        if (i < whole_jobs) return OrthoJob{ortho_tile(g, first_tile + i * tile_step), 0, slabs, -1};
        const int t = shared_tile + i - whole_jobs;
        return OrthoJob{ortho_tile(g, g.whole + t), max(shared_lo - t * slabs, 0), min(shared_hi - t * slabs, slabs),
                        xcd_contiguous(blockIdx.x, gridDim.x, g.num_xcd) + t};
    }

    // --- copies ----------------------------------------------------------------------

    int next_job;                       // still to copy
    const char *pa, *pb;                // first bytes of the slab to copy, and what lies from there on
    long long la, lb, da, db;           // (da, db: to the next slab)
    int todo;                           // slabs of the job from this one on
    int turn, segment;                  // slabs to the next pair of planes, and its number
    int put;                            // stage that the next copies go to, in chunks
    uint32_t a_off[T::A_PER_T], b_off[T::B_PER_T];

    __device__ __forceinline__ void begin(const OrthoJob &j)
    {
        const int row = j.tile.tm * T::BM, col = j.tile.tn * T::BN, per = g.k / 64;
        const LpOperand a{nullptr, 0, g.lda, g.rows - row}, b{nullptr, 0, g.ldb, g.cols - col};
        int kr, t = tid;
        asm volatile("" : "+v"(t));
#pragma unroll
        for (int i = 0; i < T::A_PER_T; ++i) a_off[i] = lp_offset<T, false, A_KS, RUN>(a, i, t, kr);
#pragma unroll
        for (int i = 0; i < T::B_PER_T; ++i) b_off[i] = lp_offset<T, true, B_KS, RUN>(b, i, t, kr);
        da = A_KS ? 64ll * g.lda : 128;
        db = B_KS ? 64ll * g.ldb : 128;
        segment = (j.first >= per ? 1 : 0) + (j.first >= 2 * per ? 1 : 0);
        const int at = j.first - segment * per;
        turn = per - at;
        todo = j.last - j.first;
        const long long skip_a = (A_KS ? (long long)row * 2 : (long long)row * g.lda) + at * da + a_plane(segment);
        const long long skip_b = (B_KS ? (long long)col * 2 : (long long)col * g.ldb) + at * db + b_plane(segment);
        pa = g.A + j.tile.matrix * g.a_stride + skip_a, la = g.a_bytes - skip_a;
        pb = g.B + j.tile.matrix * g.b_stride + skip_b, lb = g.b_bytes - skip_b;
    }
    __device__ __forceinline__ long long a_plane(int s) const { return s == g.a_at ? g.a_low : 0; }
    __device__ __forceinline__ long long b_plane(int s) const { return s == 3 - g.a_at ? g.b_low : 0; }

    __device__ __forceinline__ void advance()
    {
        long long sa = da, sb = db;
        if (--turn == 0) {
            // From the end of one pair of planes to the start of the next.
            const int per = g.k / 64;
            sa += a_plane(segment + 1) - a_plane(segment) - per * da;
            sb += b_plane(segment + 1) - b_plane(segment) - per * db;
            ++segment;
            turn = per;
        }
        pa += sa, la -= sa;
        pb += sb, lb -= sb;
        put = put + STAGE == S * STAGE ? 0 : put + STAGE;
        if (--todo == 0) next();
    }

    // Past the last job the copies read nothing.
    __device__ __forceinline__ void next()
    {
        if (next_job < jobs) {
            begin(job(next_job++));
        } else {
            la = lb = 0;
            da = db = 0;
            todo = turn = 0x7fffffff;
        }
    }

    struct Source {
        i32x4 a, b;
    };
    __device__ __forceinline__ Source source() const { return Source{lp_rsrc(pa, la), lp_rsrc(pb, lb)}; }

    __device__ __forceinline__ void copy(const Source &c, int i) const
    {
        i32x4 *const st = lds + put;
        if (i < T::A_PER_T) lp_copy16(c.a, a_off[i], st + i * T::THREADS + wave * 64);
        else lp_copy16(c.b, b_off[i - T::A_PER_T], st + T::A_CHUNKS + (i - T::A_PER_T) * T::THREADS + wave * 64);
    }

    // --- products ----------------------------------------------------------------------

    int get;

    template <int C0, int C1, bool READ = true>
    __device__ __forceinline__ void step(int p, int at, int p_next, const Source &c, LpFrags<T, kF16> &f,
                                         f32x16 (&acc)[T::MB][T::NB]) const
    {
        constexpr int NM = T::MB * T::NB, RPM = (READS + NM - 1) / NM;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            lp_mfma<T, kF16>(i, p, f, acc);
#pragma unroll
            for (int r = i * RPM; r < (i + 1) * RPM && r < READS; ++r)
                if constexpr (READ)
                    lp_read<T, kF16, A_KS, B_KS, RUN>(lds + at, lds + at + T::A_CHUNKS, r, p_next, wr, wc, lane, f);
#pragma unroll
            for (int j = C0; j < C1; ++j)
                if ((j - C0) * NM / (C1 - C0) == i) copy(c, j);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // LAST: of its job; the next one reads its own first fragments.
    template <bool LAST>
    __device__ __forceinline__ void slab(Source &c, LpFrags<T, kF16> &f, f32x16 (&acc)[T::MB][T::NB])
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
        lp_barrier<0>();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        step<0, FIRST, !LAST>(T::STEPS - 1, then, 0, c, f, acc);
        __builtin_amdgcn_s_setprio(0);
    }

    __device__ __forceinline__ void run()
    {
        plan();
        if (jobs == 0) return;
        next_job = put = get = 0;
        next();
        Source c;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            c = source();
#pragma unroll
            for (int i = 0; i < COPIES; ++i) copy(c, i);
            if (s + 1 < S) advance();
        }
        // (The last of these slabs' last quarter is issued again by the first
        // slab's work below: the same bytes to the same place.)
        lp_wait<(S - 1) * COPIES>();
        lp_barrier<63>();
        for (int i = 0; i < jobs; ++i) {
            const OrthoJob j = job(i);
            f32x16 acc[T::MB][T::NB];
#pragma unroll
            for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
                for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
            LpFrags<T, kF16> f;
#pragma unroll
            for (int r = 0; r < READS; ++r)
                lp_read<T, kF16, A_KS, B_KS, RUN>(lds + get, lds + get + T::A_CHUNKS, r, 0, wr, wc, lane, f);
            for (int kt = j.first; kt + 1 < j.last; ++kt) slab<false>(c, f, acc);
            slab<true>(c, f, acc);
            int lane_e = lane;
            asm volatile("" : "+v"(lane_e));
            if constexpr (kPlanes) {
                if (j.part >= 0) {
                    f32x4 *const out = reinterpret_cast<f32x4 *>(g.shares + (long long)j.part * (T::BM * T::BN)) +
                                       wave * (T::MB * T::NB * 256) + lane_e;
#pragma unroll
                    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
                        for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                out[((mb * T::NB + nb) * 4 + v) * 64] = f32x4{acc[mb][nb][4 * v], acc[mb][nb][4 * v + 1],
                                                                             acc[mb][nb][4 * v + 2], acc[mb][nb][4 * v + 3]};
                } else {
                    ortho_store<T>(g, j.tile, wr, wc, lane_e, acc);
                }
            } else {
                const float factor = ortho_factor(g, j.tile.matrix);
#pragma unroll
                for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
                    for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
                        for (int v = 0; v < 16; ++v) acc[mb][nb][v] = acc[mb][nb][v] * factor * g.scale;
                const int row = j.tile.tm * T::BM, col = j.tile.tn * T::BN;
                lp_store<T, E, WIDE>(g.C + j.tile.matrix * g.c_stride + row * g.ldc + (long long)col * (long long)sizeof(E), g.ldc,
                                     g.rows - row, g.cols - col, nullptr, 0, wr, wc, lane_e, acc);
            }
        }
        // The copies past the last job still write LDS.
        lp_wait<0>();
    }
};

template <class T, bool A_KS, bool B_KS, class E, bool WIDE>
__global__ __launch_bounds__(T::THREADS) void ortho_pipe_kernel(OrthoArgs g)
{
    __shared__ i32x4 lds[T::STAGES * T::stage_chunks(kF16)];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    OrthoPipe<T, A_KS, B_KS, E, WIDE> pipe{g, lds, tid, tid & 63, wave, wave % T::WAVES_M, wave / T::WAVES_M};
    pipe.run();
}

// The shared tiles' sums: a wavefront a block of 32 x 32.
template <class T>
__global__ __launch_bounds__(256) void ortho_join_kernel(OrthoArgs g)
{
    constexpr int BLOCKS = T::BM / 32 * (T::BN / 32);
    const int lane = threadIdx.x & 63;
    const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    const int t = unit / BLOCKS, block = unit % BLOCKS;
    const int slabs = g.segments * (g.k / 64);
    const long long all = ortho_shared_slabs(g, ortho_tiles(g) * g.batch);
    // Workgroup w has slabs all w / n .. all (w + 1) / n: those whose runs meet the tile's.
    const long long lo = (long long)t * slabs, hi = lo + slabs;
    int w = (int)(lo * g.shared_wgs / all);
    while (all * (w + 1) / g.shared_wgs <= lo) ++w;
    f32x16 acc{};
    for (; w < g.shared_wgs && all * w / g.shared_wgs < hi; ++w) {
        if (all * w / g.shared_wgs == all * (w + 1) / g.shared_wgs) continue;
        const f32x4 *const in = reinterpret_cast<const f32x4 *>(g.shares + (long long)(w + t) * (T::BM * T::BN)) + block * 256 + lane;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const f32x4 x = in[v * 64];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[4 * v + i] += x[i];
        }
    }
    const OrthoTile at = ortho_tile(g, g.whole + t);
    const int wave = block / (T::MB * T::NB), mb = block % (T::MB * T::NB) / T::NB, nb = block % T::NB;
    const int row0 = at.tm * T::BM + wave % T::WAVES_M * T::WM + mb * 32, col0 = at.tn * T::BN + wave / T::WAVES_M * T::WN + nb * 32;
    if (row0 < g.rows && col0 < g.cols) ortho_block(g, at.matrix, row0, col0, lane, acc, g.symmetric && at.tm != at.tn);
}

}  // namespace gemmf32
