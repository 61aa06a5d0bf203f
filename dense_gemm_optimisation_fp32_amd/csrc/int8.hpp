// 8-bit integers with a scale for each row: quantisation and its inverse.
//
//   scale = largest magnitude / 127, code = the whole number nearest to
//   x * (127 / largest magnitude), ties to even; all in 32 bits, each step
//   rounded once, so that the codes are the same wherever they are computed.
//   (|x| <= largest, so the product rounds to at most 127.)
//
// A row whose largest magnitude is below 2^-119 has scale 0 and codes 0 (the
// inverse would leave the 32-bit range); one with an infinity or a NaN has
// scale NaN and codes 0, so that it shows in every result that uses the row.
//
// Codes are (rows, kp) with zeros from k to kp: weights have kp = k rounded up
// to 16, rows of the first operand of a product kp = k rounded up to 128.
#pragma once

#include "mx4.hpp"

namespace gemmf32 {

struct Int8Args {
    const char *x;          // values (quantise: in, dequantise: out)
    char *codes;            // (rows, kp)
    float *scales;          // (rows)
    long long ld;           // elements from row to row (columns layout: from column to column)
    int rows, k, kp;
};

constexpr float kInt8Least = 0x1p-119f;

// A row's scale and the factor of its codes, from its largest magnitude's bits
// (as an unsigned number a NaN is larger than an infinity, which is larger than
// any finite value).
struct Int8Row {
    float scale, inverse;

    __device__ __forceinline__ explicit Int8Row(unsigned largest)
    {
        const float m = __uint_as_float(largest);
        const bool bad = largest >= 0x7f800000u, none = m < kInt8Least;
        scale = bad ? __builtin_nanf("") : none ? 0.0f : m / 127.0f;
        inverse = bad || none ? 0.0f : 127.0f / m;
    }
    // (A row with an infinity: inf * 0 is NaN; its codes are 0 as well.)
    __device__ __forceinline__ int code(float x) const
    {
        const float r = rintf(x * inverse);
        return r == r ? (int)r : 0;
    }
};

// Four codes a word, eight a pair.
__device__ __forceinline__ unsigned pack4(int a, int b, int c, int d)
{
    return (unsigned)(a & 255) | (unsigned)(b & 255) << 8 | (unsigned)(c & 255) << 16 | (unsigned)d << 24;
}

// Largest over the lanes of a wavefront, in every lane.
__device__ __forceinline__ unsigned wave_largest(unsigned x)
{
    x = max(x, mx_lane<0xb1>(x));
    x = max(x, mx_lane<0x4e>(x));
    x = max(x, mx_lane<0x141>(x));
    x = max(x, mx_lane<0x140>(x));
    x = max(x, (unsigned)__shfl_xor((int)x, 16));
    return max(x, (unsigned)__shfl_xor((int)x, 32));
}

// Rows contiguous along k: WAVES wavefronts a row, eight values a lane and
// piece.  A row of up to PIECES pieces stays in registers between its largest
// magnitude and its codes; of a longer one the rest is read twice.  Bound by memory:
// 14336 x 4096 in bfloat16, one MI355X: 30.6 us, 5.8 TB/s read and written.
constexpr int kInt8Pieces = 4;

template <class E, int WAVES>
__global__ __launch_bounds__(256) void int8_quantize_rows_kernel(Int8Args a)
{
    constexpr int STEP = WAVES * 512;                        // columns of a piece
    __shared__ unsigned tops[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rows_here = 4 / WAVES;
    const long long row = (long long)blockIdx.x * rows_here + wave / WAVES;
    if (WAVES == 1 && row >= a.rows) return;
    const int c0 = (wave % WAVES) * 512 + lane * 8;
    const E *const p = reinterpret_cast<const E *>(a.x) + row * a.ld;
    Mx8<E> x[kInt8Pieces];
    unsigned largest = 0;
#pragma unroll
    for (int i = 0; i < kInt8Pieces; ++i) {
        const int col = c0 + i * STEP;
        if (i * STEP < a.k) {
            x[i].load(p + col, a.k - col);
            largest = max(largest, x[i].largest());
        }
    }
    for (int i = kInt8Pieces; i * STEP < a.k; ++i) {
        Mx8<E> y;
        y.load(p + c0 + i * STEP, a.k - c0 - i * STEP);
        largest = max(largest, y.largest());
    }
    largest = wave_largest(largest);
    if constexpr (WAVES > 1) {
        if (lane == 0) tops[wave] = largest;
        __syncthreads();
        largest = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    }
    const Int8Row r(largest);
    char *const out = a.codes + row * a.kp;
    auto store = [&](const Mx8<E> &y, int col) {
        float v[8];
        y.values(v);
        u32x2 w;
        w.x = pack4(r.code(v[0]), r.code(v[1]), r.code(v[2]), r.code(v[3]));
        w.y = pack4(r.code(v[4]), r.code(v[5]), r.code(v[6]), r.code(v[7]));
        if (col < a.kp) *reinterpret_cast<u32x2 *>(out + col) = w;
    };
#pragma unroll
    for (int i = 0; i < kInt8Pieces; ++i) {
        const int col = c0 + i * STEP;
        if (i * STEP < a.kp) {
            if (i * STEP >= a.k) x[i].load(p + col, a.k - col);      // (padding: zeros, nothing is read)
            store(x[i], col);
        }
    }
    for (int i = kInt8Pieces; i * STEP < a.kp; ++i) {
        Mx8<E> y;
        y.load(p + c0 + i * STEP, a.k - c0 - i * STEP);
        store(y, c0 + i * STEP);
    }
    if (lane == 0 && wave % WAVES == 0) a.scales[row] = r.scale;
}

// Rows contiguous along the other axis (x(r, c) = x[c * ld + r]): a workgroup
// takes 64 rows, a lane one of them in each of its 16 wavefronts, which share
// the columns 16 at a time; the second reading comes from the caches.  Far from
// memory's rate: a lane loads one value at a time, and a CU has 64 rows, so that few
// long rows go column after column on few CUs.  One MI355X, us, bfloat16 / 32 bits (rows
// contiguous along k): 14336 rows of 4096 177 / 204 (27 / 42), 4096 of 14336 594 / 653
// (33 / 56), 1024 of 4096 87 / 87 (4 / 4), 4096 of 1024 25 / 25 (4 / 4).
template <class E>
__global__ __launch_bounds__(1024) void int8_quantize_columns_kernel(Int8Args a)
{
    __shared__ unsigned tops[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = blockIdx.x * 64 + lane;
    const bool live = row < a.rows;
    const E *const p = reinterpret_cast<const E *>(a.x) + (live ? row : a.rows - 1);
    unsigned largest = 0;
    for (int c = wave * 16; c < a.k; c += 256) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (c + i < a.k) largest = max(largest, magnitude(to_f32(p[(long long)(c + i) * a.ld])));
    }
    tops[wave][lane] = largest;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) largest = max(largest, tops[w][lane]);
    const Int8Row r(largest);
    if (!live) return;
    char *const out = a.codes + (long long)row * a.kp;
    for (int c = wave * 16; c < a.kp; c += 256) {
        int code[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) code[i] = c + i < a.k ? r.code(to_f32(p[(long long)(c + i) * a.ld])) : 0;
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack4(code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]);
        *reinterpret_cast<u32x4 *>(out + c) = w;
    }
    if (wave == 0) a.scales[row] = r.scale;
}

// Codes back to values, rounded once to the type: 16 bytes of them a lane and store.
// Bound by memory: 14336 x 4096 to bfloat16 33.8 us, 5.2 TB/s.
template <class E>
__global__ __launch_bounds__(256) void int8_dequantize_kernel(Int8Args a)
{
    constexpr int N = 16 / sizeof(E), RUN = 64 * N;
    const int lane = threadIdx.x & 63;
    const unsigned segments = (unsigned)((a.k + RUN - 1) / RUN);
    const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const long long row = unit / segments;
    if (row >= a.rows) return;
    const int col = (int)(unit % segments) * RUN + lane * N;
    if (col >= a.k) return;
    struct __attribute__((packed, aligned(sizeof(E)))) Run {
        E e[N];
    } t;
    const char *const p = a.codes + row * a.kp + col;
    const float scale = a.scales[row];
    const unsigned lo = *reinterpret_cast<const unsigned *>(p), hi = N == 8 ? *reinterpret_cast<const unsigned *>(p + 4) : 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) t.e[i] = (E)((float)(signed char)((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 255) * scale);
    E *const out = reinterpret_cast<E *>(const_cast<char *>(a.x)) + row * a.ld + col;
    if (col + N <= a.k) {
        *reinterpret_cast<Run *>(out) = t;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (col + i < a.k) out[i] = t.e[i];
    }
}

}  // namespace gemmf32
