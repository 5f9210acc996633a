// The 4-bit cache type: groups of 16 values n * s, s an e4m3 scale and n in -7..7
// held as n + 8. A 32-bit word holds 8 values, value i at bits 4 (i / 2) + 16 (i mod 2),
// so that one shift and one mask leave two neighbours in the halves of a word.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dsrows {
namespace int4 {

constexpr int kGroup = 16;
constexpr uint8_t kNanScale = 0x7F;

// A group's scale s as the pair of factors of `widen`: (s, s) and (-136 s, -136 s)
// as bf16. Both are exact: s has 4 significant bits, 136 = 8 * 17, and 17 times
// 4 bits is 8 bits.
struct Factors {
    uint32_t s, c;
};

// The scales in the low two bytes of `b`.
__device__ __forceinline__ float2 scales2(uint32_t b) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(b & 0xFFFFu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// The factors of two scales, bytes `at` and `at` + 1 of `b`. A byte's exponent and mantissa
// in a bf16's places are s 2^-120 (the types' biases are 7 and 127; subnormals agree
// too), so one exact product gives s. The byte of NaN would give 480, bytes with a sign 512 and
// more: from 480 on, s (145/128) 2^119 is past the largest bf16, up to 448 it is not, and
// infinity times 0 makes it NaN.
template <int at>
__device__ __forceinline__ void factors2(uint32_t b, Factors& f0, Factors& f1) {
    constexpr uint32_t kScale = 0x7B807B80u, kFar = 0x7B117B11u, kMinus136 = 0xC308C308u;
    const uint32_t x = __byte_perm(b, 0, at == 0 ? 0x4140 : 0x4342) * 16u;
    uint32_t s = fma_bf16x2(x, kScale, 0x80008000u);
    s = fma_bf16x2(fma_bf16x2(s, kFar, 0x80008000u), 0u, s);
    const uint32_t c = fma_bf16x2(s, kMinus136, 0x80008000u);
    f0 = {__byte_perm(s, 0, 0x1010), __byte_perm(c, 0, 0x1010)};
    f1 = {__byte_perm(s, 0, 0x3232), __byte_perm(c, 0, 0x3232)};
}

// One word's 8 values as bf16 pairs: word j holds values 2 j and 2 j + 1. 0x4300 | (n + 8)
// is 128 + 8 + n in bf16, so (136 + n) s - 136 s is n s, which is exact in bf16. The mask
// and the exponent are one instruction (with both as constants it became two: 64 of the
// 311 ALU instructions of a key in the indexer).
__device__ __forceinline__ void widen(uint32_t word, Factors f, uint32_t* out) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t t;
        asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(t) : "r"(word >> (4 * j)), "r"(0x43004300u));
        out[j] = fma_bf16x2(t, f.s, f.c);
    }
}

// Quantise a group: 16 values to two words and the scale byte; `held` receives the
// values that the cache then stands for. The quotients are correctly rounded by
// Markstein's theorem (q0 = y r with r = 1 / s rounded to nearest, q = q0 + (y - q0 s) r
// with fused products), 3 FMA instructions instead of a division each; adding and
// taking away 1.5 * 2^23 rounds to the nearest integer, even on ties. Four values of a
// half word are packed as one sum below 2^16 in fp32.
__device__ __forceinline__ uint8_t quantise(const float (&y)[kGroup], uint32_t (&word)[2], float (&held)[kGroup]) {
    constexpr float kToInt = 12582912.0f;
    uint32_t top = 0;  // of the magnitudes as integers: infinity and NaN are the largest
#pragma unroll
    for (int i = 0; i < kGroup; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    const uint8_t byte = top < 0x7F800000u
                             ? (uint8_t)__nv_cvt_float_to_fp8(__uint_as_float(top) / 7.0f, __NV_SATFINITE, __NV_E4M3)
                             : kNanScale;
    const float s = scales2(byte).x;
    // s = 0: every n is 0. s = NaN: every n is -7 (what fmaxf makes of NaN), every value NaN.
    const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
    float n[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
        const float q0 = y[i] * r;
        n[i] = fmaf(fmaf(-q0, s, y[i]), r, q0);
    }
    // A normal s is at least 16/17 of top / 7, so |q| <= 7.44 rounds to 7 at most; a subnormal,
    // saturated or NaN one says nothing.
    if (byte < 0x08 || byte >= 0x7E)
#pragma unroll
        for (int i = 0; i < kGroup; ++i) n[i] = fminf(fmaxf(n[i], -7.0f), 7.0f);
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
        n[i] = (n[i] + kToInt) - kToInt;
        held[i] = n[i] * s;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float* c = n + 8 * k + h;
            // (n + 8) of values h, h + 2, h + 4, h + 6 at bits 0, 4, 8, 12: the eights sum to 0x8888.
            const float sum = fmaf(fmaf(fmaf(c[6], 16.0f, c[4]), 16.0f, c[2]), 16.0f, c[0]) + (float)0x8888;
            half[h] = __float_as_uint(sum + 8388608.0f);
        }
        word[k] = __byte_perm(half[0], half[1], 0x5410);
    }
    return byte;
}

}  // namespace int4
}  // namespace dsrows
