// Products grouped by expert in 32 bits, on the direct-to-LDS tiles of
// mfma_dma_gemm.hpp: a tile of an expert's product is a tile of an ordinary
// product whose operands begin at the tile's rows, so the tile loop and its
// range checks are those of the plain product.  Bound by the
// matrix cores (v_mfma_f32_32x32x2_f32), as there.
//
//   C_e = act(A_e . B_e + bias_e), dB_e = A_e^T . G_e (column-major A_e).
#pragma once

#include "expert_common.hpp"
#include "mfma_dma_gemm.hpp"

namespace gemmf32 {

// Operands of a tile are addressed from its first row, and its expert's
// matrix, with 32-bit byte offsets (the host checks these extents; the whole
// of A, B and C may be larger).
__device__ __forceinline__ uint32_t extent_bytes(long long bytes)
{
    return bytes < 0 ? 0u : (uint32_t)min(bytes, 0x7ffffffcll);
}

// Accumulators -> C with bias and activation; the lanes' rows and columns are
// those of dma_store_c.  A NaN stays one.
template <class T, bool B_COL>
__device__ __forceinline__ void f32_grouped_store(const GemmArgs &g, __amdgpu_buffer_rsrc_t rc, int col0, int wr,
                                                  int wc, int l32, int half, const f32x16 (&acc)[T::MB][T::NB])
{
    const __amdgpu_buffer_rsrc_t rbias = make_rsrc(g.bias, g.bias ? (uint32_t)g.n * 4u : 0u);
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) {
        const int c = B_COL ? col0 + wc * T::WN + nb * 32 + l32 : col0 + wc * T::WN + T::NB * l32 + nb;
        const float bias = buf_load_x1(rbias, elem_off(c < g.n, 0, 0, c));
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int r = wr * T::WM + mb * 32 + 8 * (v >> 2) + 4 * half + (v & 3);
                float x = acc[mb][nb][v] + bias;
                if (g.act) x = activate(x, g.act);
                buf_store_x1(x, rc, elem_off(r < g.m && c < g.n, r, g.ldc, c));
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

template <class T, bool B_COL>
__global__ __launch_bounds__(T::THREADS) void f32_grouped_kernel(GroupedArgs a)
{
    __shared__ f32x4 lds[T::STAGES * (T::A_CHUNKS + T::B_CHUNKS)];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % T::WAVES_M, wc = wave / T::WAVES_M;
    const int l32 = lane & 31, half = lane >> 5;
    RowTile rt;
    int tn;
    if (!find_tile<T::BM>(a, blockIdx.x, lane, rt, tn)) return;
    const int col0 = tn * T::BN;
    GemmArgs g{};
    g.m = min(rt.rows, T::BM);
    g.n = a.n;
    g.k = a.k;
    g.lda = (int)(a.lda / 4);
    g.ldb = (int)(a.ldb / 4);
    g.ldc = (int)(a.ldc / 4);
    g.k_tiles = (a.k + T::BK - 1) / T::BK;
    g.act = a.act;
    g.bias = a.bias && rt.expert >= 0 ? a.bias + rt.expert * a.bias_stride : nullptr;
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc(a.A + rt.row * a.lda, extent_bytes((g.m - 1) * a.lda + a.k * 4ll));
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(a.B + max(rt.expert, 0) * a.expert_stride,
                  extent_bytes(B_COL ? (a.n - 1) * a.ldb + a.k * 4ll : (a.k - 1) * a.ldb + a.n * 4ll));
    const __amdgpu_buffer_rsrc_t rc =
        make_rsrc(a.C + rt.row * a.ldc, extent_bytes((g.m - 1) * a.ldc + a.n * 4ll));
    f32x16 acc[T::MB][T::NB];
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
    if (rt.expert >= 0)
        dma_range<T, B_COL>(g, lds, lds + T::STAGES * T::A_CHUNKS, ra, rb, 0, col0, 0, g.k_tiles, tid, wave, wr, wc, l32,
                            half, acc);
    else
        g.act = 0;
    f32_grouped_store<T, B_COL>(g, rc, col0, wr, wc, l32, half, acc);
}

// The contraction runs over an expert's rows.  Rows are taken in runs whose
// byte extents fit 31 bits, each run the k range of one pass of the tile
// loop, so that the matrices themselves may be of any size.
template <class T>
__global__ __launch_bounds__(T::THREADS) void f32_weight_grad_kernel(GroupedArgs a)
{
    __shared__ f32x4 lds[T::STAGES * (T::A_CHUNKS + T::B_CHUNKS)];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % T::WAVES_M, wc = wave / T::WAVES_M;
    const int l32 = lane & 31, half = lane >> 5;
    GradTile t;
    if (!grad_tile(a, blockIdx.x % a.num_xcd, blockIdx.x / a.num_xcd, t)) return;
    const int expert = t.expert, row0 = t.tm * T::BM, col0 = t.tn * T::BN;
    const Rows rows = entry_rows(a, expert);
    int lo = __builtin_amdgcn_readfirstlane(rows.lo);
    const int hi = __builtin_amdgcn_readfirstlane(rows.hi);
    GemmArgs g{};
    g.m = a.k;
    g.n = a.n;
    g.lda = (int)(a.lda / 4);
    g.ldb = (int)(a.ldb / 4);
    g.ldc = (int)(a.ldc / 4);
    const int run = (int)min((long long)0x7ffffff0, 0x7fff0000ll / max(a.lda, a.ldb));
    f32x16 acc[T::MB][T::NB];
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
    // (Counted by the rows left: lo + run could pass 32 bits.)
    for (int left = hi - lo; left > 0; left -= g.k, lo += g.k) {
        g.k = min(run, left);
        g.k_tiles = (g.k + T::BK - 1) / T::BK;
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A + lo * a.lda, extent_bytes((g.k - 1) * a.lda + a.k * 4ll));
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B + lo * a.ldb, extent_bytes((g.k - 1) * a.ldb + a.n * 4ll));
        dma_range<T, false, true>(g, lds, lds + T::STAGES * T::A_CHUNKS, ra, rb, row0, col0, 0, g.k_tiles, tid, wave,
                                  wr, wc, l32, half, acc);
    }
    const __amdgpu_buffer_rsrc_t rc =
        make_rsrc(a.C + expert * a.expert_stride, extent_bytes((a.k - 1) * a.ldc + a.n * 4ll));
    dma_store_c<T, false, true>(g, rc, row0, col0, wr, wc, l32, half, acc);
}

}  // namespace gemmf32
