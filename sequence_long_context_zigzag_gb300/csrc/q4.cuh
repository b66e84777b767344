// q4.cuh -- the 4-bit format of a paged cache: what its writers and its readers share (not part of the ABI).
//
// A row of hd values is hd / 32 groups of 32, each with a scale byte b, s(b) = (8 + (b & 7)) 2^((b >> 3) - 23): an
// unsigned float of 5 exponent and 3 fraction bits, 2^-20 to 3840, without a zero. A code c in [-8, 7] stands for c s.
// Codes are two's complement, 8 to a 32-bit word: value e of the 8 is nibble e / 2 + 4 (e % 2), so (word >> 4 j) has the
// values 2 j and 2 j + 1 in the low nibbles of its halves, where an operand of the tensor cores has them.
//   c s has at most 7 significant bits (3 of the code, 4 of the scale): it is exact in bf16, and readers of every kind see
// the same values. A page of zero bytes holds zeros.
#pragma once

#include <stdint.h>

#include "usp_internal.cuh"

namespace usp {

constexpr int kQ4Group = 32;

// bytes of a row's codes and scales
__host__ __device__ constexpr int q4_code_bytes(int hd) { return hd / 2; }
__host__ __device__ constexpr int q4_scale_bytes(int hd) { return hd / kQ4Group; }

// 1 + f / 8 has the fraction field f << 20, and the exponent field of 2^(e - 20) is e + 107
__device__ __forceinline__ float q4_scale(uint32_t b) { return __uint_as_float((b << 20) + (107u << 23)); }

// The smallest b with 7.5 s(b) >= a (255 where there is none): every value of a group whose largest magnitude is a is then
// at most half a step from a code (7.5 s rounds to 8, and 7 is as near). The estimate is a rounded product; 7.5 s is
// exact, so the comparisons make it the definition's.
__device__ __forceinline__ uint32_t q4_scale_for(float a) {
    const uint32_t y = __float_as_uint(a * (1.0f / 7.5f));
    int b = (int)((y + 0xfffffu) >> 20) - (107 << 3);
    b = max(0, min(b, 255));
    if (b > 0 && 7.5f * q4_scale(b - 1) >= a) --b;
    else if (b < 255 && 7.5f * q4_scale(b) < a) ++b;
    return (uint32_t)b;
}

// min(7, max(-8, x / s to the nearest whole number, ties to even)) by the definition: x - r s is exact in fp32 for |x| <=
// 9 s (s has 4 significant bits), and tells on which side of the tie x lies. NaN gives 0.
static __device__ __noinline__ int q4_code_exact(float x, float s) {
    if (x != x) return 0;
    float r = rintf(fminf(fmaxf(x / s, -9.f), 9.f));
    if (fabsf(x) <= 9.f * s) {
        const float e = fmaf(-r, s, x), h = 0.5f * s;
        if (fabsf(e) > h || (fabsf(e) == h && ((int)r & 1))) r += copysignf(1.f, e);
    }
    return (int)fminf(fmaxf(r, -8.f), 7.f);
}

// The word of 8 values' codes, scale byte b. The codes come from the rounded product with 1 / s; where that lies so near
// a tie that its rounding may have decided (or a value is NaN or past the largest scale), all 8 are taken by the
// definition: x * inv is off by less than 2^-20 of a step.
__device__ __forceinline__ uint32_t q4_pack(const float (&x)[8], uint32_t b) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the rounded whole number
    const float s = q4_scale(b), inv = __frcp_rn(s);
    uint32_t w = 0;
    bool fine = b < 255;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = fmaf(x[e], inv, kMagic);
        fine = fine && fabsf(fmaf(x[e], inv, kMagic - y)) < 0.49999f;  // false for a NaN
        w |= (__float_as_uint(y) & 15u) << (4 * (e / 2 + 4 * (e % 2)));
    }
    if (!fine) {
        w = 0;
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
            float v = 0.f;  // (a selection: x stays in registers)
#pragma unroll
            for (int i = 0; i < 8; ++i) v = i == e ? x[i] : v;
            w |= ((uint32_t)q4_code_exact(v, s) & 15u) << (4 * (e / 2 + 4 * (e % 2)));
        }
    }
    return w;
}

int check_q4_dims(const usp_q4_dims &d);

}  // namespace usp
