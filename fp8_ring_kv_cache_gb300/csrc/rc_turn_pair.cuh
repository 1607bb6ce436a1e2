// rc_turn_pair.cuh -- the turn with twice the bits: (cos, sin) as sums of two fp32
// numbers and the products with bf16 numbers summed without loss, for codes that
// are those of the exact turn.
#pragma once
#include "rc_paged.cuh"

namespace rc {

// (cos, sin) of position * frequency as sums of two fp32 numbers each, to 2^-25.6
// at the worst (four roundings of sin's x^3 terms, under 0.081): the angle, exact
// in integers, is brought within an eighth of a turn and taken as two fp32
// numbers, and the Taylor series to x^11 and x^10 there are kept apart from their
// leading terms.
struct TurnPair {
    float2 hi, lo;  // (cos, sin)
};
__device__ __forceinline__ TurnPair turn_cos_sin_pair(int pos, uint64_t turns) {
    const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
    const uint32_t quad = static_cast<uint32_t>((frac + (1ull << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(frac - (static_cast<uint64_t>(quad) << 62));  // / 2^64 turns
    const float top = static_cast<float>(static_cast<int32_t>(rest >> 38)) * 0x1p-23f;      // eighths of a turn: exact
    const float low = static_cast<float>(static_cast<uint32_t>(rest >> 8) & 0x3fffffffu);
    constexpr float kH = 0.785398185253143310546875f, kL = -2.18556938e-8f;  // pi / 4
    const float x0 = __fmul_rn(top, kH);
    const float x1 = __fadd_rn(__fmaf_rn(top, kH, -x0), __fmaf_rn(top, kL, low * 8.71967125e-17f));  // 2 pi / 2^56
    const float x = __fadd_rn(x0, x1), xl = __fadd_rn(x1, -__fadd_rn(x, -x0));
    const float z = __fmul_rn(x, x), zl = __fmaf_rn(x, x, -z);
    const float S = fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.50521084e-8f, 2.75573192e-6f), -1.98412698e-4f), 8.33333333e-3f),
                         -1.66666667e-1f);
    const float sl = fmaf(x * z, S, fmaf(-0.5f * z, xl, xl));
    const float C = fmaf(z, fmaf(z, fmaf(z, -2.75573192e-7f, 2.48015873e-5f), -1.38888889e-3f), 4.16666667e-2f);
    const float c0 = __fadd_rn(1.f, -0.5f * z);
    const float cl = __fadd_rn(__fadd_rn(-0.5f * z, -__fadd_rn(c0, -1.f)), fmaf(z * z, C, -fmaf(x, xl, 0.5f * zl)));
    float2 s, c;  // (hi, lo)
    s.x = __fadd_rn(x, sl);
    s.y = __fadd_rn(sl, -__fadd_rn(s.x, -x));
    c.x = __fadd_rn(c0, cl);
    c.y = __fadd_rn(cl, -__fadd_rn(c.x, -c0));
    const float2 cc = (quad & 1u) ? s : c, ss = (quad & 1u) ? c : s;
    const float cf = (quad == 1u || quad == 2u) ? -1.f : 1.f, sf = (quad & 2u) ? -1.f : 1.f;
    TurnPair r;
    r.hi = make_float2(cf * cc.x, sf * ss.x);
    r.lo = make_float2(cf * cc.y, sf * ss.y);
    return r;
}

// a c + b s with c and s as sums of two numbers (a, b of 8 bits), rounded to odd:
// a later rounding to fewer bits takes it for the exact sum.
__device__ __forceinline__ float sum_exactly(float a, float c, float cl, float b, float s, float sl) {
    const float p = __fmul_rn(a, c), q = __fmul_rn(b, s), d = __fadd_rn(p, q), bb = __fadd_rn(d, -p);
    const float rest = __fadd_rn(__fadd_rn(p, -__fadd_rn(d, -bb)), __fadd_rn(q, -bb));
    const float low = __fadd_rn(__fadd_rn(rest, __fmaf_rn(a, c, -p)), __fadd_rn(__fmaf_rn(b, s, -q), fmaf(a, cl, b * sl)));
    const float y = __fadd_rn(d, low), off = __fadd_rn(low, -__fadd_rn(y, -d));
    const uint32_t u = __float_as_uint(y);
    if (off == 0.f || (u & 1u) || (u & 0x7fffffffu) == 0u) return y;
    return __uint_as_float(((off > 0.f) == (y > 0.f)) ? u | 1u : u - 1u);  // between y and its neighbour: the odd one
}

}  // namespace rc
