// rc_paged4.cuh -- the 4-bit paged cache's numbers: E2M1 codes, and scale bytes
// with 5 bits of exponent and 3 of fraction (the top byte but the sign of an fp16
// number, so that a byte becomes one by a shift).  A code times a scale has at
// most 6 significant bits and lies between 2^-18 and 61,440: an exact fp16 and
// bf16 number.
#pragma once
#include "rc_paged.cuh"

namespace rc {

constexpr int kBlock4 = 16;              // dims of a scale
constexpr uint32_t kTopScale4 = 226u;    // 10,240: the largest scale that a row gets
constexpr uint32_t kFirstNan4 = 248u;    // infinity, and NaN above it
// Where a row's running maximum (in log2 units) is this large, scores are rounded before it is subtracted, and a maximum is
// kept as it is: its own weight is 1.  Below, a weight is exp2 of one multiply-add of the score with a maximum kept
// some units lower, where rounding moves the exponent by 2^-5 at most; far above, that would be more than fp16 weights allow.
constexpr float kLargeScore4 = 0x1p20f;
// That is looked at where a query row's largest value is 16 or more (its power of two in query_tile_f16 2^-10 then): of others
// no score is over 16 x 128 x 61,440 x log2(e) / sqrt(128) < 2^24, where the exponent moves by 2^-1 and weights still fit.
// (32 x 8,000 tokens with 16 rows: 81.4 us without the question, 82.4 so, 83.2 if all rows are asked; a prefill 489, 491 and
// 496, with queries of 64 times the size 556 without and 564 with it.)
constexpr float kLargeQuery4 = 0x1p-10f;

__device__ __forceinline__ float scale4_value(uint32_t b) { return __half2float(__ushort_as_half(static_cast<unsigned short>(b << 7))); }

// Scale bytes 0, 1 and 2, 3 of a word as pairs of fp16 numbers.
__device__ __forceinline__ uint32_t scales01(uint32_t w) { return __byte_perm(w, 0u, 0x1404) >> 1; }
__device__ __forceinline__ uint32_t scales23(uint32_t w) { return __byte_perm(w, 0u, 0x3424) >> 1; }
// Bytes `odd` and 2 + `odd` of a word (odd 0 or 1) as fp16 numbers.
__device__ __forceinline__ uint32_t scales_apart(uint32_t w, int odd) { return __byte_perm(w, 0u, 0x2404u + 0x1010u * odd) >> 1; }
// Not 0 if a byte of a word is 248 or more: no number.
__device__ __forceinline__ uint32_t nan_scales(uint32_t w) { return ((w & 0x78787878u) + 0x08080808u) & w & 0x80808080u; }

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Both numbers times the lower, or the upper, one of b.
__device__ __forceinline__ uint32_t half2_mul_lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {l, l};\n\tmul.rn.f16x2 %0, %1, t;\n\t}\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t half2_mul_hi(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {h, h};\n\tmul.rn.f16x2 %0, %1, t;\n\t}\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Eight codes of a word as four pairs of fp16 numbers, in order.
__device__ __forceinline__ void codes8_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
// Eight numbers as codes (nearest, ties to even, cut at 6), the first in the low bits.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}\n"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

}  // namespace rc
