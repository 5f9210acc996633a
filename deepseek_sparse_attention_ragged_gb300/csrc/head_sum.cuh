// The indexer's epilogue arithmetic: a key's 64 head dot products to its score.
#pragma once

#include "common.cuh"

namespace dsrows {

__device__ __forceinline__ float relu_nan(float x) {
    // max(0, x) that keeps NaN (a NaN dot product must poison the score).
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
    return r;
}

// Two fp32 FMAs in one instruction (each rounded as fmaf): d = a * b + c lane-wise.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
          "l"(*reinterpret_cast<const uint64_t*>(&c)));
    return *reinterpret_cast<const float2*>(&d);
}

// sum_h w[h] relu(x[h]) over the 64 head dot products x of one key, with w in
// registers (wr) or shared memory (w_s): four chains (heads h = c mod 4, in
// head order), added pairwise.
__device__ __forceinline__ float head_sum(const uint32_t (&x)[64], const float* wr, const float* w_s) {
    if (wr) {
        // Weights in registers: chains 0 and 1 (heads h = 0, 1 mod 4) and chains
        // 2 and 3 advance in pairs, two FMAs per instruction.
        float2 s01 = make_float2(0.0f, 0.0f), s23 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int h = 0; h < kIdxHeads; h += 4) {
            const float2 r01 = make_float2(relu_nan(__uint_as_float(x[h])), relu_nan(__uint_as_float(x[h + 1])));
            const float2 r23 = make_float2(relu_nan(__uint_as_float(x[h + 2])), relu_nan(__uint_as_float(x[h + 3])));
            s01 = fma2(r01, make_float2(wr[h], wr[h + 1]), s01);
            s23 = fma2(r23, make_float2(wr[h + 2], wr[h + 3]), s23);
        }
        return (s01.x + s01.y) + (s23.x + s23.y);
    }
    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < kIdxHeads; h += 4) {
        const float4 w4 = *reinterpret_cast<const float4*>(w_s + h);
        s4[0] = fmaf(relu_nan(__uint_as_float(x[h])), w4.x, s4[0]);
        s4[1] = fmaf(relu_nan(__uint_as_float(x[h + 1])), w4.y, s4[1]);
        s4[2] = fmaf(relu_nan(__uint_as_float(x[h + 2])), w4.z, s4[2]);
        s4[3] = fmaf(relu_nan(__uint_as_float(x[h + 3])), w4.w, s4[3]);
    }
    return (s4[0] + s4[1]) + (s4[2] + s4[3]);
}

// The same sum, 32 heads at a time with the weights in shared memory. With kAdd, x + |x| =
// 2 max(0, x) takes the place of the maximum and w holds half the weights: the products and so
// the sums are the same, bit for bit, where the half weights are exact (halvable()) and no 2 x
// overflows. The addition runs on the FMA pipe, the maximum on the integer pipe at half its
// rate. An overflowing 2 x makes the total NaN or infinite where the maximum's may be finite: a
// total that is not finite says nothing, and is taken again without kAdd.
template <bool kAdd>
struct HeadSum {
    float2 s01 = {0.0f, 0.0f}, s23 = {0.0f, 0.0f};
    static __device__ __forceinline__ float relu(uint32_t bits) {
        const float x = __uint_as_float(bits);
        return kAdd ? x + fabsf(x) : relu_nan(x);
    }
    __device__ __forceinline__ void add(const uint32_t (&x)[32], const float* w_s) {
#pragma unroll
        for (int h = 0; h < 32; h += 4) {
            const float4 w4 = *reinterpret_cast<const float4*>(w_s + h);
            s01 = fma2(make_float2(relu(x[h]), relu(x[h + 1])), make_float2(w4.x, w4.y), s01);
            s23 = fma2(make_float2(relu(x[h + 2]), relu(x[h + 3])), make_float2(w4.z, w4.w), s23);
        }
    }
    __device__ __forceinline__ float total() const { return (s01.x + s01.y) + (s23.x + s23.y); }
};

// Whether half of a weight is exact: below 2^-125 the half may lose its last bit.
__device__ __forceinline__ bool halvable(float w) { return w == 0.0f || !(fabsf(w) < 0x1p-125f); }

// The score of a key from its 64 head dot products in TMEM (one lane, 64 columns).
template <bool kAdd>
__device__ __forceinline__ float head_sum_tmem(uint32_t taddr, const float* w_s) {
    HeadSum<kAdd> sum;
    uint32_t v[32];
    tmem_ld_x32(taddr, v);
    tmem_ld_wait();
    sum.add(v, w_s);
    tmem_ld_x32(taddr + 32, v);
    tmem_ld_wait();
    sum.add(v, w_s + 32);
    return sum.total();
}

}  // namespace dsrows
