// The 4-bit format of a cache: e2m1 codes (sign and 0, 0.5, 1, 1.5, 2, 3, 4, 6), two in a byte
// (element 2i in the low half of byte i), and one e4m3 scale for 16 elements.  A scale has four
// significant bits and a code two, so their product is exact in bf16 and in fp16 (it is a
// multiple of 2^-10 and at most 2688): what a cache holds is taken into the matrix products
// as it is.
#pragma once

#include <cstdint>

namespace jfa {

// The eight codes of w as four fp16 pairs, (element 2i, element 2i + 1).
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 bytes as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(h) : "r"(two));
    return h;
}

// The e4m3 bytes nearest to a (low) and b (high), at most 448.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b) {
    uint32_t two;
    asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.u32.u16 %0, x;\n\t}" : "=r"(two) : "f"(a), "f"(b));
    return two;
}

// The e2m1 codes nearest to eight values, ties to even, at most 6.
__device__ __forceinline__ uint32_t to_e2m1(const float* v) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}

__device__ __forceinline__ uint32_t f16_mul2(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// An fp16 pair as floats.
__device__ __forceinline__ float2 f16_to_float(uint32_t h) {
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}

// (lo, hi) rounded to an fp16 pair.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
}

}  // namespace jfa
