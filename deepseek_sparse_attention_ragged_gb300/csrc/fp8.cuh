// The 8-bit cache type: blocks of 128 values v * 2^e, v an e4m3 number of magnitude at
// most 448 and e the block's exponent, -100 .. 7, held as the byte e + 127. A power of two
// as the scale makes every cached value exact in bf16: the readers need no rounding of their own.
#pragma once

#include <cuda_fp8.h>

#include "int4.cuh"

namespace dsrows {
namespace fp8 {

constexpr int kBlock = 128;
constexpr uint32_t kMinByte = 27, kMaxByte = 134;  // e = -100 .. 7
constexpr uint32_t kNanByte = 255;

// A block's exponent byte as the factor of `widen`: 2^(e + 120) as a pair of bf16, NaN for a
// byte out of range.
__device__ __forceinline__ uint32_t factor(uint32_t byte) {
    return byte - kMinByte <= kMaxByte - kMinByte ? (byte + 120) * 0x00800080u : 0x7FC07FC0u;
}

// The 4 values of a word as bf16 pairs. A byte's exponent and mantissa in a bf16's places are
// v 2^-120 (the types' biases are 7 and 127; subnormals agree too), so one exact product gives
// v 2^e. There is no code for NaN: 0x7F is 480 (an append never writes it). Here as (v0, v2) and (v1, v3): three or four
// logical operations, and shifts to the left, which the FMA pipe does.
__device__ __forceinline__ void widen_apart(uint32_t word, uint32_t f, uint32_t& even, uint32_t& odd) {
    constexpr uint32_t kPlaces = 0x07F007F0u;
    const uint32_t signs = word & 0x80808080u;
    even = int4::fma_bf16x2((word * 16 & kPlaces) | (signs * 256 & ~kPlaces), f, 0x80008000u);
    odd = int4::fma_bf16x2((word >> 4 & kPlaces) | (signs & ~kPlaces), f, 0x80008000u);
}

// ... in order. (Two neighbouring bytes put in their places first take two operations more.)
__device__ __forceinline__ void widen(uint32_t word, uint32_t f, uint32_t* out) {
    uint32_t even, odd;
    widen_apart(word, f, even, odd);
    out[0] = __byte_perm(even, odd, 0x5410);
    out[1] = __byte_perm(even, odd, 0x7632);
}

// The exponent byte of a block from the largest magnitude's bits: the least e with top <= 448 2^e,
// within its range; 448 is 1.75 2^8. Infinity and NaN are the largest magnitudes.
__device__ __forceinline__ uint32_t exponent_byte(uint32_t top) {
    if (top >= 0x7F800000u) return kNanByte;
    const int b = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)min(max(b, (int)kMinByte), (int)kMaxByte);
}

// 16 values of a block to 4 words: v = y 2^-e to the nearest e4m3 (ties to even, saturating); zeros in a block
// that is stored as NaN. The product is exact: it can only lose bits far below e4m3's smallest step.
__device__ __forceinline__ void quantise(const float (&y)[16], uint32_t byte, uint32_t (&word)[4]) {
    const float down = __uint_as_float((254u - (byte == kNanByte ? 127u : byte)) << 23);  // 2^-e
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i] * down, y[4 * i + 1] * down), __NV_SATFINITE,
                                                     __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2] * down, y[4 * i + 3] * down),
                                                     __NV_SATFINITE, __NV_E4M3);
        word[i] = byte == kNanByte ? 0u : lo | hi << 16;
    }
}

}  // namespace fp8
}  // namespace dsrows
