// fp4.cuh -- rows of the 4-bit cache: how they are quantised and what they stand for.
//
// A row (one token, one KV head, 128 values) is 128 E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a
// sign; two a byte, the even dimension in the low half), one E4M3 scale for every 16 of them and one
// exponent byte e, 1 .. 254 for 2^(e - 127), 255 for NaN.  It stands for code * scale * 2^(e - 127):
// 2 + 4 significant bits and a power of two, which bf16 and f16 hold without a rounding.
//
// Quantising x: 2^(e - 127) is the least power of two by which the row's largest magnitude is at
// most 6 * 448; with y = x / 2^(e - 127), exact, a group of 16 takes the scale E4M3(max|y| / 6) and
// the codes E2M1(y / scale), both rounded to the nearest, ties to even, and clamped to the largest.
// y and the scale have few enough bits that the fp32 quotients, correctly rounded, cross no midpoint:
// the codes of bf16 rows are those of exact arithmetic.  A group whose scale rounds to 0 (under
// 2^-10 * 6 * 2^(e - 127)) gets codes 0, a row that holds a NaN or an infinity the exponent 255.
#pragma once

#include "common.cuh"

namespace pa {

constexpr int kFp4Group = 16;                     // values under one scale
constexpr int kFp4Groups = kD / kFp4Group;        // scales of a row (8 bytes)
constexpr int kFp4RowCodes = kD / 2;              // bytes of a row's codes
constexpr uint32_t kFp4NanExp = 255;

// Largest magnitude of the row as bits (NaN sorts above infinity) -> its exponent byte.
__device__ __forceinline__ uint32_t fp4_row_exp(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return kFp4NanExp;
    if (amax_bits == 0) return 127;
    // amax = m 2^E <= 1.3125 * 2^11 * 2^n: n = E - 11, one more when m > 1.3125
    return (uint32_t)max((int)((amax_bits + 0x7fffffu - 0x280000u) >> 23) - 11, 1);
}

// 2^(127 - e), by which a row is divided by its power of two (e in 1 .. 244).
__device__ __forceinline__ float fp4_unit_inverse(uint32_t e) {
    return __uint_as_float((254u - min(e, 253u)) << 23);   // (anything will do for a row that is NaN)
}

// 2^(e - 127), NaN for 255 (e = 0, which no append writes, would be 2^-127; it counts as 0).
__device__ __forceinline__ float fp4_unit(uint32_t e) {
    return __uint_as_float(e == kFp4NanExp ? 0x7fc00000u : e << 23);
}

// The fp32 quotient a / b, correctly rounded, from r = 1 / b: a * r and one correction by the exact
// remainder (Markstein 1990, IBM J. Res. Dev. 34(1)); zeros keep a's sign.  For quotients far from overflow
// and for those so small that the code is 0 in any case.
__device__ __forceinline__ float fp4_quotient(float a, float b, float r) {
    const float p = __fmul_rn(a, r);
    return __fmaf_rn(__fmaf_rn(p, b, -a), -r, p);
}

// E4M3 scale of a group whose largest |y| is `top`.
__device__ __forceinline__ uint32_t fp4_group_scale(float top) {
    return f32x2_to_e4m3x2(fp4_quotient(top, 6.f, 1.f / 6.f), 0.f) & 0xffu;
}

// The value of an E4M3 scale byte.
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    float v;
    asm("{\n .reg .b16 a, l, h;\n .reg .b32 p;\n cvt.u16.u32 a, %1;\n cvt.rn.f16x2.e4m3x2 p, a;\n mov.b32 {l, h}, p;\n"
        " cvt.f32.f16 %0, l;\n}"
        : "=f"(v)
        : "r"(code));
    return v;
}

// Eight values -> eight E2M1 codes, value 0 in the lowest four bits; nearest, ties to even, beyond 6 to 6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&q)[8]) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

// Eight E2M1 codes -> four f16x2, exact: h[i] = {code 2i, code 2i + 1}.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// The codes of eight values y of a group with E4M3 scale byte `scale`.
__device__ __forceinline__ uint32_t fp4_codes(const float (&y)[8], uint32_t scale) {
    const float m = e4m3_value(scale);
    const float r = __frcp_rn(m);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {   // fp4_quotient, two at a time
        float p0, p1, d0, d1;
        ffma2(p0, p1, y[e], y[e + 1], r, r, -0.f, -0.f);
        ffma2(d0, d1, p0, p1, m, m, -y[e], -y[e + 1]);
        ffma2(q[e], q[e + 1], d0, d1, -r, -r, p0, p1);
    }
    return m > 0.f ? f32x8_to_e2m1x8(q) : 0u;
}

__device__ __forceinline__ uint32_t umax_xor(uint32_t x, int o) {
    return max(x, __shfl_xor_sync(0xffffffffu, x, o));
}

}  // namespace pa
