// The angle of a rotary pair, shared by the rotation and append kernels.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace dsrows {

// Cosine and sine of `pos` * theta times m, where `turns` is theta / (2 pi) as a
// 64-bit fraction of a turn: the product modulo 2^64 is the angle's fraction of a
// turn exactly (far positions lose nothing), its high word, as a signed number,
// the angle in [-1/2, 1/2) turns. That word's rounding to fp32 moves the angle by
// 2^-25 of itself at most.
__device__ __forceinline__ float2 rope_turn(int32_t pos, uint64_t turns, float m, bool inverse) {
    const uint64_t phase = (uint64_t)(uint32_t)pos * turns;
    const float half_turns = (float)(int32_t)(phase >> 32) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * m, (inverse ? -s : s) * m);
}

// The rotation of a pair (x, y) in fp32, each element with one rounded and one fused
// product, so that every path gives the same bits.
__device__ __forceinline__ float rope_first(float x, float y, float2 cs) { return fmaf(x, cs.x, -__fmul_rn(y, cs.y)); }
__device__ __forceinline__ float rope_second(float x, float y, float2 cs) { return fmaf(x, cs.y, __fmul_rn(y, cs.x)); }
__device__ __forceinline__ void rope_pair(float& a, float& b, float2 cs) {
    const float x = a, y = b;
    a = rope_first(x, y, cs);
    b = rope_second(x, y, cs);
}

}  // namespace dsrows
