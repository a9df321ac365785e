// MXFP4 (OCP Microscaling Formats v1.0): 4-bit E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
// their negatives) in blocks of 32 consecutive values along the contraction, each block with one
// E8M0 scale, a power of two 2^(byte - 127).
//
//   e    = clamp(floor(log2(max |x|)) - 2, -127, 125)        (2 = exponent of E2M1's largest, 6)
//   code = round to nearest even E2M1 of x 2^-e, at most 6
//
// With x in fp32 everything but that last rounding is exact: floor(log2) is the exponent field,
// and x 2^-e a multiplication by a normal power of two.  A block that holds an infinity or a NaN
// gets the NaN scale (255) and zero codes, so that whatever it is multiplied into is NaN.
//
// Layouts of an operand [rows, K]:
//   codes   [rows][ceil(K/32) * 16 bytes], the value of even k in the low half of a byte; values
//           past K are zero.
//   scales  tiles of 128 rows x 4 blocks, 512 bytes each, [ceil(rows/128)][ceil(K/128)]; in a
//           tile the byte of row r, block j is at (r % 32) * 16 + (r / 32) * 4 + j, which is what
//           tcgen05.cp 32x128b brings to tensor memory as the block-scaled MMA reads it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace tpmlp {
namespace mx {

// Byte of the scale of row `row`, block `blk` in the tiled layout with `k_tiles` = ceil(K/128).
__host__ __device__ __forceinline__ long long scale_offset(long long row, long long blk, long long k_tiles) {
    return ((row >> 7) * k_tiles + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// Scale byte of a block whose largest |x| has the bits amax (ordered: finite < 0x7F800000 <= infinity and NaN).
__device__ __forceinline__ uint32_t scale_of(uint32_t amax) {
    const uint32_t ex = amax >> 23;
    return amax >= 0x7F800000u ? 255u : (ex > 2u ? ex - 2u : 0u);
}
// 2^-e of scale byte s <= 252: a normal fp32 number (2^127 .. 2^-125); 0 for the NaN scale.
__device__ __forceinline__ float inverse_scale(uint32_t s) {
    return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}
// 2^e of scale byte s: subnormal for 0, NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : (s == 255u ? 0x7FFFFFFFu : s << 23));
}

// Eight values (already scaled) to eight codes, v[0] in the lowest half byte.
__device__ __forceinline__ uint32_t encode8(float v0, float v1, float v2, float v3, float v4, float v5, float v6,
                                            float v7) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v0), "f"(v1), "f"(v2), "f"(v3), "f"(v4), "f"(v5), "f"(v6), "f"(v7));
    return r;
}
// Eight codes to their values.
__device__ __forceinline__ void decode8(uint32_t c, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float amax3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The same of two bf16 pairs, each half by itself; the signs of the result mean nothing.
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (a, b) * s, two products in one instruction.
__device__ __forceinline__ void mul2(float& a, float& b, float s) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\t"
        "mov.b64 y, {%2, %2};\n\t"
        "mul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(s));
}

// One block of 32 fp32 values of this thread: 16 bytes of codes and the scale byte.  About 60
// instructions: 16 three-operand maxima, 16 paired products, 16 conversions of two values.
__device__ __forceinline__ uint32_t quantize32(const float (&v)[32], uint4& codes) {
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = amax3(v[i * 8], v[i * 8 + 1], v[i * 8 + 2]);
        a[i] = amax3(a[i], v[i * 8 + 3], v[i * 8 + 4]);
        a[i] = amax3(a[i], v[i * 8 + 5], v[i * 8 + 6]);
    }
    a[0] = amax3(a[0], v[7], v[15]);
    a[1] = amax3(a[1], v[23], v[31]);
    const uint32_t s = scale_of(__float_as_uint(amax3(amax3(a[0], a[1], a[2]), a[3], 0.0f)));
    const float inv = inverse_scale(s);
    uint32_t c[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[w * 8 + i];
#pragma unroll
        for (int i = 0; i < 8; i += 2) mul2(x[i], x[i + 1], inv);
        c[w] = encode8(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
    }
    codes = s == 255u ? make_uint4(0, 0, 0, 0) : make_uint4(c[0], c[1], c[2], c[3]);
    return s;
}

// Column sums of up to two fp32 arrays [rows][cols] of partial sums, rounded to the output's type.
struct SumsArgs {
    const float* in[2];
    void* out[2];
    int cols[2];
    int rows, f32;
    int items0, items;  // items of 8 columns of the first array, of both
};
// One item, a warp: four lanes share a column, each takes every fourth row.  The order is fixed and does not depend
// on who takes the item.
__device__ __forceinline__ void sum_columns(const SumsArgs& a, int item, int lane) {
    const int k = item >= a.items0, cols = a.cols[k];
    const int c = (item - (k ? a.items0 : 0)) * 8 + (lane & 7);
    float v = 0.0f;
    if (c < cols) {
        const float* src = a.in[k] + c;
#pragma unroll 8
        for (int r = lane >> 3; r < a.rows; r += 4) v += src[static_cast<long long>(r) * cols];
    }
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
    if (lane < 8 && c < cols) {
        if (a.f32) static_cast<float*>(a.out[k])[c] = v;
        else static_cast<__nv_bfloat16*>(a.out[k])[c] = __float2bfloat16_rn(v);
    }
}

}  // namespace mx
}  // namespace tpmlp
