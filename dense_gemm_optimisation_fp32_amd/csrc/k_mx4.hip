// Kernel translation unit: 4-bit quantisation and its inverse.
#include "expert_launch.hpp"
#include "mx4.hpp"

namespace gemmf32 {

int launch_mx4_quantize(const Mx4Args &a, bool bf16, bool columns, hipStream_t s)
{
    if (columns) {
        const long long grid = (long long)((a.rows + 63) / 64) * (a.kp / 128);
        return launch(bf16 ? mx4_quantize_columns_kernel<__bf16> : mx4_quantize_columns_kernel<float>, grid, 256, 0, s, a);
    }
    const long long grid = ((long long)a.rows * ((a.kp + 511) / 512) + 3) / 4;
    return launch(bf16 ? mx4_quantize_rows_kernel<__bf16> : mx4_quantize_rows_kernel<float>, grid, 256, 0, s, a);
}

int launch_mx4_dequantize(const Mx4Args &a, bool bf16, hipStream_t s)
{
    const long long grid = ((long long)a.rows * ((a.k + 511) / 512) + 3) / 4;
    return launch(bf16 ? mx4_dequantize_kernel<__bf16> : mx4_dequantize_kernel<float>, grid, 256, 0, s, a);
}

}  // namespace gemmf32
