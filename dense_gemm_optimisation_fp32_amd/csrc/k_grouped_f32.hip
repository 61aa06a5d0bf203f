// Kernel translation unit: products grouped by expert in 32 bits.
#include "expert_launch.hpp"
#include "grouped_f32.hpp"

namespace gemmf32 {

namespace {

using Tile128 = DmaTile<128, 128, 16, 2, 2, 3, false>;
using Tile64x128 = DmaTile<64, 128, 16, 2, 2, 2>;
using Tile64 = DmaTile<64, 64, 16, 2, 2, 2>;
using Tile64Ring = DmaTile<64, 64, 16, 2, 2, 4>;

// Tiles of 64 rows below 608 rows an expert: an expert's last tile is half
// empty on average, and 128 x 128 tiles run at 147 TFLOPS, 64 x 128 at about
// 140, where they are full.  64 columns where the last 128 would be at most
// half full.  Measured, 16 experts, us for 128 x 128 / 64 x 128 / 64 x 64: 5003
// rows, k = 2049, n = 1027: 288 / 291 / 237 (B contiguous: 283 / 248 / 254);
// 8192 rows, k = n = 1024: 139 / 134 / 146; 8 experts of 1024 rows, k = n =
// 4096: 1982 / 2098 / 2207.  Near 608 rows an expert the two larger tiles change
// places with every step in the number of tiles, 128 x 128 / 64 x 128: k = 2048,
// n = 4096, 576 rows 1185 / 1156, 608 rows 1190 / 1253, 640 rows 1206 / 1279, 704
// rows 1420 / 1411, uneven experts 576 rows 1301 / 1247, 640 rows 1308 / 1327; k = n =
// 1024, 608 rows 182 / 161, 704 rows 183 / 190, uneven 704 rows 244 / 198.
int tile_of(int rows, int n) { return rows >= 608 ? 0 : n % 128 > 64 || n % 128 == 0 ? 1 : 2; }

// Few tiles are bound by the latency of one slab after the other: 64 x 64 in four
// slabs up to two a CU.  Measured, us, above / so: 3 experts, k = 6544, n = 1216,
// 256 rows 282 / 130; one expert, k = n = 4096, 256 rows 188 / 87, k = 4096, n =
// 14336, 128 rows 152 / 137; weight gradient of k = n = 1024, 64 rows 6.7 / 5.0,
// 4096 rows 252 / 77.
bool few_tiles(int groups, int rows, int n, int cu_count)
{
    return (long long)groups * ((rows + 63) / 64) * ((n + 63) / 64) <= 2ll * cu_count;
}

template <class T>
int launch_tile(GroupedArgs a, bool b_contiguous, hipStream_t s)
{
    a.tiles_m = grouped_row_tiles(a, T::BM);
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    return launch(b_contiguous ? f32_grouped_kernel<T, true> : f32_grouped_kernel<T, false>,
                  (long long)a.tiles_m * a.tiles_n, T::THREADS, 0, s, a);
}

template <class T>
int launch_grad(GroupedArgs a, hipStream_t s)
{
    a.tiles_m = (a.k + T::BM - 1) / T::BM;
    a.tiles_n = (a.n + T::BN - 1) / T::BN;
    return launch(f32_weight_grad_kernel<T>, grad_workgroups(a), T::THREADS, 0, s, a);
}

}  // namespace

int launch_f32_grouped(const GroupedArgs &a, bool b_contiguous, int cu_count, hipStream_t s)
{
    const int rows = (a.m + a.groups - 1) / a.groups;
    if (few_tiles(a.groups, rows, a.n, cu_count)) return launch_tile<Tile64Ring>(a, b_contiguous, s);
    switch (tile_of(rows, a.n)) {
    case 0: return launch_tile<Tile128>(a, b_contiguous, s);
    case 1: return launch_tile<Tile64x128>(a, b_contiguous, s);
    default: return launch_tile<Tile64>(a, b_contiguous, s);
    }
}

// Here the expert's rows are the contraction: smaller tiles where it is short
// (the same sizes, us: 250 / 241 / 239; 161 / 133 / 138; 1904 / 1946 / 1993).  By
// rows an expert, 128 x 128 / 64 x 128: k = 2048, n = 4096, 512 rows 1003 / 1018, 608
// rows 1164 / 1201, 704 rows 1336 / 1377; k = n = 1024, where the large tiles leave CUs
// idle, 608 rows 186 / 156, 768 rows 231 / 193, uneven 170 / 168 and 208 / 207.
int launch_f32_weight_grad(const GroupedArgs &a, int cu_count, hipStream_t s)
{
    if (few_tiles(a.groups, a.k, a.n, cu_count)) return launch_grad<Tile64Ring>(a, s);
    switch (tile_of((a.m + a.groups - 1) / a.groups, a.n)) {
    case 0: return launch_grad<Tile128>(a, s);
    case 1: return launch_grad<Tile64x128>(a, s);
    default: return launch_grad<Tile64>(a, s);
    }
}

}  // namespace gemmf32
