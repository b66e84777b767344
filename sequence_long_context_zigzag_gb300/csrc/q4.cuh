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
// at most half a step from a code (7.5 s rounds to 8, and 7 is as near). The estimate's factor is below 1 / 7.5, so it is never
// too large; 7.5 s is exact, and the comparison makes it the definition's.
__device__ __forceinline__ uint32_t q4_scale_for(float a) {
    const uint32_t y = __float_as_uint(a * 0.133333325f);
    const int b = max((int)((y + 0xfffffu) >> 20) - (107 << 3), 0);
    return (uint32_t)min(b + (7.5f * q4_scale((uint32_t)b) < a ? 1 : 0), 255);
}

// min(7, max(-8, x / s to the nearest whole number, ties to even)) by the definition, inv being 1 / s nearly: x - r s is
// exact in fp32 for |x| <= 9 s (s has 4 significant bits), and tells on which side of the tie x lies. NaN gives 0.
__device__ __forceinline__ int q4_code_exact(float x, float s, float inv) {
    if (x != x) return 0;
    float r = rintf(fminf(fmaxf(x * inv, -9.f), 9.f));
    const float e = fmaf(-r, s, x), h = 0.5f * s;
    if (fabsf(x) <= 9.f * s && (fabsf(e) > h || (fabsf(e) == h && ((int)r & 1)))) r += copysignf(1.f, e);
    return (int)fminf(fmaxf(r, -8.f), 7.f);
}

// What the values of a group share: its scale byte, and 1 / s to 2^-23.
struct Q4Scale {
    uint32_t b;
    float inv;
    __device__ __forceinline__ explicit Q4Scale(float largest) : b(q4_scale_for(largest)) {
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(q4_scale(b)));
    }
};

// The word of 8 values' codes. x / s is taken to a grid of 2^-18 (48 + x / s, rounded: off by 2^-20 and half a grid step, less
// than a step), and that to a whole number. A quotient that is a tie lies on the grid and rounds to even; no other one
// crosses a tie, but one nearer than a grid step may land on it. kExact: the values are bf16 numbers X 2^i, whose quotients
// X 2^j / (8 .. 15) lie 2^-11 at least from a tie that they are not on. Otherwise all 8 are taken by the definition where one lies on
// a tie, and in any case where values may be past the largest scale.
// Codes are summed as digits of 16: y's low bits hold the whole number r, and what its upper bits add is a constant.
template <bool kExact> __device__ __forceinline__ uint32_t q4_pack(const float (&x)[8], const Q4Scale &s) {
    constexpr float kGrid = 48.f, kMagic = 12582912.f;  // 1.5 * 2^5, 1.5 * 2^23
    constexpr uint32_t kBits = 0x4b400000u, kOnes = 0x11111111u;
    uint32_t w = 0x88888888u - kBits * kOnes;  // digits r + 8 need no borrow
    uint32_t tie = 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = fminf(fmaf(x[e], s.inv, kGrid), kGrid + 7.f);
        const float y = q + (kMagic - kGrid);
        w += __float_as_uint(y) << (4 * (e / 2 + 4 * (e % 2)));
        if (!kExact) tie = min(tie, (__float_as_uint(q) & 0x3ffffu) ^ 0x20000u);
    }
    if (s.b < 255 && (kExact || tie != 0)) return w ^ 0x88888888u;
    w = 0;
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
        float v = 0.f;  // (a selection: x stays in registers)
#pragma unroll
        for (int i = 0; i < 8; ++i) v = i == e ? x[i] : v;
        w |= ((uint32_t)q4_code_exact(v, q4_scale(s.b), s.inv) & 15u) << (4 * (e / 2 + 4 * (e % 2)));
    }
    return w;
}

int check_q4_dims(const usp_q4_dims &d);

}  // namespace usp
