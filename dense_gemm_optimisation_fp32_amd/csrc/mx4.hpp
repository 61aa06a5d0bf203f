// Microscaled 4-bit floating point: quantisation and its inverse.
//
// Blocks of 32 values along k share a power of two, 2^e; each value is the
// nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} times the scale (ties to the even
// code) with its sign.  e = floor(log2(largest magnitude)) - 2, at least -127,
// so the largest magnitude lands in [4, 8) and saturates at 6.  A block that
// holds an infinity or a NaN has no such e: its scale byte is 255, which
// stands for NaN, so that it shows in every result that uses the block.
//
// Both kernels are bound by memory: one pass, 16 bytes a lane and load.
// Measured on one MI355X, 14336 x 4096 in bfloat16: quantised 25 us
// (5.9 TB/s; 31.5 with the values widened and multiplied by the inverse scale
// ahead of the conversion), back 24 us (6.2 TB/s).  Tried for the first and no
// faster: a lane per block, four pieces a lane.  Along columns the same matrix takes
// 76 us (2.0 TB/s; 55 us, 4.9 TB/s from 32 bits): neighbouring lanes read two bytes
// each, and store 16 bytes a row apart.
#pragma once

#include "expert_common.hpp"

namespace gemmf32 {

struct Mx4Args {
    const char *x;          // values (quantise: in, dequantise: out)
    u8 *codes;              // (rows, kp / 2): two codes a byte, the even column in the low half
    u8 *scales;             // (kp / 128, rows, 4)
    long long ld;           // elements from row to row (columns layout: from column to column)
    int rows, k, kp;
};

struct MxBlock {
    float scale;            // 2^e: the magnitudes are below 8 times it
    unsigned byte;          // 127 + e, or 255
};

// From the largest magnitude's bits (as an unsigned number a NaN is larger
// than an infinity, which is larger than any finite value).
__device__ __forceinline__ MxBlock mx_block(unsigned largest)
{
    const int field = (int)(largest >> 23);
    const int biased = max(field - 2, 0);                 // 127 + e
    MxBlock b;
    b.byte = field == 255 ? 255u : (unsigned)biased;
    // (2^-127 is below the normal numbers: a mantissa bit.)
    b.scale = __uint_as_float(max((unsigned)biased << 23, 0x00400000u));
    return b;
}

__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return (float)x; }

// Eight neighbouring values of a row, as they are loaded.  The conversion
// divides by the block's scale, rounds to nearest, ties to the even code, and
// saturates at 6 (checked for every bfloat16 value under every scale; the
// borders of the codes are in the tests).
template <class E>
struct Mx8;

template <>
struct Mx8<float> {
    float v[8];

    __device__ __forceinline__ void load(const float *p, int left)
    {
        const f32x4 a = __builtin_bit_cast(f32x4, load_chunk(p, left));
        const f32x4 b = __builtin_bit_cast(f32x4, load_chunk(p + 4, left - 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    }
    __device__ __forceinline__ void values(float (&out)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = v[i];
    }
    __device__ __forceinline__ unsigned largest() const
    {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[i]));
        return m;
    }
    __device__ __forceinline__ unsigned codes(float scale) const
    {
        unsigned w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
        return w;
    }
};

template <>
struct Mx8<__bf16> {
    i32x4 v;

    __device__ __forceinline__ void load(const __bf16 *p, int left) { v = load_chunk(p, left); }
    __device__ __forceinline__ void values(float (&out)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[2 * i] = __uint_as_float((unsigned)v[i] << 16);
            out[2 * i + 1] = __uint_as_float((unsigned)v[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ unsigned largest() const
    {
        typedef unsigned short Pair __attribute__((ext_vector_type(2)));
        Pair m = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(Pair, v[i] & 0x7fff7fff));
        return (unsigned)max(m[0], m[1]) << 16;
    }
    __device__ __forceinline__ unsigned codes(float scale) const
    {
        // (Each word by value: the bit cast of a vector's element read its first.)
        typedef __bf16 Pair __attribute__((ext_vector_type(2)));
        const int w0 = v[0], w1 = v[1], w2 = v[2], w3 = v[3];
        unsigned w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(Pair, w0), scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(Pair, w1), scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(Pair, w2), scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(Pair, w3), scale, 3);
        return w;
    }
};

// Eight values from p on, those at or past `left` zero.  Unaligned wide
// loads are in order here: rows of odd length start anywhere.
template <class E>
__device__ __forceinline__ void load8(const E *p, int left, float (&v)[8])
{
    struct __attribute__((packed, aligned(sizeof(E)))) Eight {
        E e[8];
    };
    if (left >= 8) {
        const Eight t = *reinterpret_cast<const Eight *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(t.e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
    }
}

// x of another lane: CTRL 0xb1 and 0x4e the neighbour and the other pair of
// four, 0x124 and 0x128 four and eight places on in the row of 16.
template <int CTRL>
__device__ __forceinline__ unsigned mx_lane(unsigned x)
{
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}

// Rows contiguous along k: four lanes hold a block, eight values each, and
// sixteen lanes the four blocks of a scale word.
template <class E>
__global__ __launch_bounds__(256) void mx4_quantize_rows_kernel(Mx4Args a)
{
    const int lane = threadIdx.x & 63;
    const int segments = (a.kp + 511) / 512;              // 512 columns a wavefront
    const unsigned unit = blockIdx.x * 4 + (threadIdx.x >> 6);      // (fits: the host checks)
    const long long row = unit / (unsigned)segments;
    if (row >= a.rows) return;
    const int col = (int)(unit % (unsigned)segments) * 512 + lane * 8;
    Mx8<E> x;
    x.load(reinterpret_cast<const E *>(a.x) + row * a.ld + col, a.k - col);
    unsigned largest = x.largest();
    largest = max(largest, mx_lane<0xb1>(largest));
    largest = max(largest, mx_lane<0x4e>(largest));
    const MxBlock b = mx_block(largest);
    const unsigned codes = b.byte == 255 ? 0u : x.codes(b.scale);
    unsigned word = b.byte << (8 * ((lane >> 2) & 3));
    word |= mx_lane<0x128>(word);
    word |= mx_lane<0x124>(word);
    if (col < a.kp) {
        *reinterpret_cast<unsigned *>(a.codes + row * (a.kp / 2) + col / 2) = codes;
        if ((lane & 15) == 0)
            *reinterpret_cast<unsigned *>(a.scales + ((long long)(col / 128) * a.rows + row) * 4) = word;
    }
}

// Rows contiguous along the other axis (x(r, c) = x[c * ld + r]): a lane
// takes one row's block, neighbouring lanes neighbouring rows; the four
// wavefronts take the four blocks of a scale word.
template <class E>
__global__ __launch_bounds__(256) void mx4_quantize_columns_kernel(Mx4Args a)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int strips = (a.rows + 63) / 64;
    const int kb = blockIdx.x / strips;
    const int row = blockIdx.x % strips * 64 + lane;
    if (row >= a.rows) return;
    const int col = kb * 128 + wave * 32;
    Mx8<float> x[4];
    const E *p = reinterpret_cast<const E *>(a.x) + (long long)col * a.ld + row;
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i / 8].v[i % 8] = col + i < a.k ? to_f32(p[(long long)i * a.ld]) : 0.0f;
    unsigned largest = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) largest = max(largest, x[i].largest());
    const MxBlock b = mx_block(largest);
    u32x4 codes = {};
    if (b.byte != 255)
#pragma unroll
        for (int i = 0; i < 4; ++i) codes[i] = x[i].codes(b.scale);
    *reinterpret_cast<u32x4 *>(a.codes + (long long)row * (a.kp / 2) + col / 2) = codes;
    a.scales[((long long)kb * a.rows + row) * 4 + wave] = (u8)b.byte;
}

// Codes and scales back to values: 16 bytes of them a lane and store, so that
// a wavefront's store is one run (32 bits: two runs of 256 columns; with eight
// neighbouring columns a lane the stores had gaps, 79 us at 8192 x 7168).  The
// scale byte 0 is 2^-127, below the normal numbers: set by its mantissa bit.
template <class E>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(Mx4Args a)
{
    constexpr int N = 16 / sizeof(E), RUNS = 8 / N;
    const int lane = threadIdx.x & 63;
    const int segments = (a.k + 511) / 512;
    const unsigned unit = blockIdx.x * 4 + (threadIdx.x >> 6);
    const long long row = unit / (unsigned)segments;
    if (row >= a.rows) return;
    struct __attribute__((packed, aligned(sizeof(E)))) Run {
        E e[N];
    } t[RUNS];
    int col[RUNS];
#pragma unroll
    for (int q = 0; q < RUNS; ++q) {
        col[q] = (int)(unit % (unsigned)segments) * 512 + q * 64 * N + lane * N;
        if (col[q] >= a.k) continue;
        const u8 *const p = a.codes + row * (a.kp / 2) + col[q] / 2;
        const unsigned codes = N == 8 ? *reinterpret_cast<const unsigned *>(p) : *reinterpret_cast<const unsigned short *>(p);
        const unsigned byte = a.scales[((long long)(col[q] / 128) * a.rows + row) * 4 + ((col[q] >> 5) & 3)];
        const float scale = byte == 255 ? __builtin_nanf("") : __uint_as_float(byte ? byte << 23 : 0x00400000u);
        // A code times a power of two is exact in 32 and in 16 bits.
        const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
        const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
        t[q].e[0] = (E)(v0.x * scale), t[q].e[1] = (E)(v0.y * scale);
        t[q].e[2] = (E)(v1.x * scale), t[q].e[3] = (E)(v1.y * scale);
        if constexpr (N == 8) {
            const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
            const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
            t[q].e[4] = (E)(v2.x * scale), t[q].e[5] = (E)(v2.y * scale);
            t[q].e[6] = (E)(v3.x * scale), t[q].e[7] = (E)(v3.y * scale);
        }
    }
    E *const out = reinterpret_cast<E *>(const_cast<char *>(a.x)) + row * a.ld;
#pragma unroll
    for (int q = 0; q < RUNS; ++q) {
        if (col[q] + N <= a.k) {
            *reinterpret_cast<Run *>(out + col[q]) = t[q];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (col[q] + i < a.k) out[col[q] + i] = t[q].e[i];
        }
    }
}

}  // namespace gemmf32
