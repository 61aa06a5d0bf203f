// Kernel translation unit: 8-bit quantisation and its inverse.
#include "expert_launch.hpp"
#include "int8.hpp"

namespace gemmf32 {

namespace {

template <class E>
int launch_rows(const Int8Args &a, hipStream_t s)
{
    // A wavefront a row where that holds it in registers.
    if (a.k <= 512 * kInt8Pieces) return launch(int8_quantize_rows_kernel<E, 1>, (a.rows + 3ll) / 4, 256, 0, s, a);
    return launch(int8_quantize_rows_kernel<E, 4>, a.rows, 256, 0, s, a);
}

}  // namespace

int launch_int8_quantize(const Int8Args &a, bool bf16, bool columns, hipStream_t s)
{
    if (columns)
        return launch(bf16 ? int8_quantize_columns_kernel<__bf16> : int8_quantize_columns_kernel<float>,
                      (a.rows + 63ll) / 64, 1024, 0, s, a);
    return bf16 ? launch_rows<__bf16>(a, s) : launch_rows<float>(a, s);
}

int launch_int8_dequantize(const Int8Args &a, bool bf16, hipStream_t s)
{
    const int run = bf16 ? 512 : 256;
    const long long grid = ((long long)a.rows * ((a.k + run - 1) / run) + 3) / 4;
    return launch(bf16 ? int8_dequantize_kernel<__bf16> : int8_dequantize_kernel<float>, grid, 256, 0, s, a);
}

}  // namespace gemmf32
