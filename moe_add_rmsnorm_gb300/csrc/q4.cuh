// Device helpers of the products with 4-bit weights (q4_row.cu, q4_rows.cuh, q4_mma.cuh).
//
// The arithmetic.  A 4-bit word less its zero point is a small integer, exact in f16, and so is an int8 activation word; an f32
// activation is, in units of a power of two that its 32-value block shares, the sum of two f16 parts (22 significant bits
// of the block's largest value).  So a 32-value block's dot is a warp-wide f16 product with f32 sums over one or two
// columns, in which every product is exact; it is then multiplied by the weights' scale and the block's, in f32.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "ffn4.h"

namespace q8 {

enum { FORM_F32 = 0, FORM_ONE = 1, FORM_TWO = 2 };  // activations: f32, int8 words, words and low words

// The eight words of w less their zero point, as pairs of f16: values (0, 4), (1, 5), (2, 6), (3, 7).  A word placed in the
// low mantissa bits of 1024 is 1024 + word, one placed four bits higher 1024 + 16 word = 16 (64 + word): both exact.  (The
// conversion by 1024's mantissa bits is published: Kim, Henry, Fahim and Hassan Awadalla, "Who Says Elephants Can't Run:
// Bringing Large Scale MoE Models into Cloud Scale Production", 2022.)
// zc: 1024 + z twice; zf: -(64 + z) twice.
__device__ __forceinline__ void words_f16(uint32_t w, uint32_t zc, uint32_t zf, uint32_t (&h)[4]) {
    const __half2 sixteenth = __float2half2_rn(0.0625f);
    const __half2 c = *reinterpret_cast<const __half2*>(&zc), f = *reinterpret_cast<const __half2*>(&zf);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t lo, hi;
        asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(lo) : "r"(w));
        asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(hi) : "r"(w));
        const __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), c);
        const __half2 b = __hfma2(*reinterpret_cast<__half2*>(&hi), sixteenth, f);
        h[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
        h[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
        w >>= 8;
    }
}

// The two forms of a zero point that words_f16 takes, the second from the first.
__device__ __forceinline__ uint32_t zero_less(uint32_t zc) {
    const __half2 v = __hsub2(__float2half2_rn(960.f), *reinterpret_cast<__half2*>(&zc));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void zero_forms(uint32_t z, uint32_t& zc, uint32_t& zf) {
    zc = 0x64006400u | (z * 0x10001u);
    zf = zero_less(zc);
}

__device__ __forceinline__ float scale_f32(uint32_t bits, int bf16) {
    return bf16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half((unsigned short)bits));
}

// d += a b over 16 rows, 8 columns and 16 values (f16 in, f32 sums).
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pairs of f32, two operations an instruction.
__device__ __forceinline__ float2 pair_mul(float2 a, float2 b) {
    float2 d;
    asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ void pair_fma(float2& acc, float2 a, float bx, float by) {
    asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%0, %1}; fma.rn.f32x2 z, x, y, z; "
        "mov.b64 {%0, %1}, z;}"
        : "+f"(acc.x), "+f"(acc.y) : "f"(a.x), "f"(a.y), "f"(bx), "f"(by));
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight consecutive values of an activation row as f16 parts, in the order words_f16 gives the weights.
struct ActParts {
    uint4 hi, lo;
    float scale;
};

// The largest finite magnitude of eight values.
__device__ __forceinline__ float finite_max(const float (&x)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]) <= 3.402823466e38f ? fabsf(x[i]) : 0.f);
    return m;
}

// The parts of eight values that share a unit with others of which m is the largest magnitude.  The unit, 2^(e - 141), brings
// m into [2^14, 2^15): well inside f16, and a value's second part leaves f16's normal range only 2^18 below that.  e is held
// where both the unit and its inverse are normal numbers.
__device__ __forceinline__ ActParts split_values(const float (&x)[8], float m) {
    const unsigned e = max(__float_as_uint(m) >> 23, 15u);
    const float up = __uint_as_float((268u - e) << 23);
    float v[8], r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = x[i] * up;
        const float h = __half2float(__float2half_rn(v[i]));
        r[i] = fabsf(h) <= 65504.f ? v[i] - h : 0.f;  // (what is not finite stays in the first part)
    }
    ActParts p;
    p.hi = make_uint4(pack_f16(v[0], v[4]), pack_f16(v[1], v[5]), pack_f16(v[2], v[6]), pack_f16(v[3], v[7]));
    p.lo = make_uint4(pack_f16(r[0], r[4]), pack_f16(r[1], r[5]), pack_f16(r[2], r[6]), pack_f16(r[3], r[7]));
    p.scale = __uint_as_float((e - 14u) << 23);
    return p;
}

// Eight int8 words (and low words, in 128ths) as f16 parts.
__device__ __forceinline__ uint4 words_parts(uint2 w, float unit) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = unit * (float)(int8_t)(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xff);
    return make_uint4(pack_f16(v[0], v[4]), pack_f16(v[1], v[5]), pack_f16(v[2], v[6]), pack_f16(v[3], v[7]));
}

// Values 8 i .. 8 i + 7 of f32 activation row r (zeros from `cols` on).
__device__ __forceinline__ void act_values(const Q4Act& a, int64_t r, int i, int cols, float (&x)[8]) {
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
    if (8 * i < cols) {
        const float4* p = reinterpret_cast<const float4*>(a.x + r * a.stride + 8 * i);
        u = p[0], v = p[1];
    }
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
}

// Values 8 i .. 8 i + 7 of quantized activation row r (zeros from `cols` on).
__device__ __forceinline__ ActParts act_words(const Q4Act& a, int64_t r, int i, int cols) {
    ActParts p = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), 0.f};
    if (8 * i < cols) {
        const int64_t at = r * cols + 8 * i;
        p.hi = words_parts(*reinterpret_cast<const uint2*>(a.q + at), 1.f);
        if (a.lo) p.lo = words_parts(*reinterpret_cast<const uint2*>(a.lo + at), 0.0078125f);
        p.scale = a.s[at >> 5];
    }
    return p;
}

}  // namespace q8
