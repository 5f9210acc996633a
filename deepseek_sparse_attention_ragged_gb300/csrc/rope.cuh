// The angle of a rotary pair, shared by the rotation and append kernels.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace dsrows {

// Cosine and sine of `pos` * theta times m, where `turns` is theta / (2 pi) as a 64-bit
// fraction of a turn: the product modulo 2^64 is the angle's fraction of a turn, with no error
// but the table's half step of 2^-64 times the position. It is split into the nearest quarter
// turn and a remainder, exactly, whose 64 bits both words of r = [-pi/4, pi/4] are taken from:
// small angles keep their relative accuracy (with the high word alone the sine of 10^-4 was
// off by 10^-5 of itself). The Taylor polynomials of sine (to r^9, the next term is below
// 2e-9) and cosine (to r^8, 3e-8) give both: half the instructions of reducing and evaluating
// a general argument, which were a quarter of the append's.
__device__ __forceinline__ float2 rope_turn(int32_t pos, uint64_t turns, float m, bool inverse) {
    const uint64_t phase = (uint64_t)(uint32_t)pos * turns;
    const uint32_t high = (uint32_t)(phase >> 32);
    const uint32_t quarter = (high + 0x20000000u) >> 30;
    constexpr float kHigh = 1.4629180792671596e-9f, kLow = kHigh / 4294967296.0f;  // 2 pi / 2^32, 2 pi / 2^64
    const float r = fmaf((float)(int32_t)(high - (quarter << 30)), kHigh, (float)(uint32_t)phase * kLow);
    const float r2 = r * r;
    float s = fmaf(r2, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, -1/7!
    s = fmaf(r2, s, 8.3333333e-3f);                     // 1/5!
    s = fmaf(r2, s, -1.6666667e-1f);                    // -1/3!
    s = fmaf(r2 * r, s, r);
    float c = fmaf(r2, 2.4801587e-5f, -1.3888889e-3f);  // 1/8!, -1/6!
    c = fmaf(r2, c, 4.1666667e-2f);                     // 1/4!
    c = fmaf(r2, c, -0.5f);
    c = fmaf(r2, c, 1.0f);
    // A quarter turn on: (c, s) -> (-s, c).
    const float cq = quarter & 1 ? s : c, sq = quarter & 1 ? c : s;
    const float cm = (quarter + 1) & 2 ? -m : m, sm = (quarter >> 1 & 1) != (inverse ? 1u : 0u) ? -m : m;
    return make_float2(cq * cm, sq * sm);
}

// The rotation of a pair (x, y) in fp32, each element with one rounded and one fused
// product, so that every path gives the same bits: own * cos + other * (-+ sin).
__device__ __forceinline__ float rope_first(float x, float y, float2 cs) { return fmaf(x, cs.x, -__fmul_rn(y, cs.y)); }
__device__ __forceinline__ float rope_second(float x, float y, float2 cs) { return fmaf(y, cs.x, __fmul_rn(x, cs.y)); }
__device__ __forceinline__ void rope_pair(float& a, float& b, float2 cs) {
    const float x = a, y = b;
    a = rope_first(x, y, cs);
    b = rope_second(x, y, cs);
}

}  // namespace dsrows
