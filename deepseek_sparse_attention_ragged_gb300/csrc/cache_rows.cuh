// Sixteen neighbouring elements of a cached row, in any page type.
#pragma once

#include "common.cuh"
#include "fp8.cuh"
#include "int4.cuh"
#include "kernels.h"

namespace dsrows {

// As they are held (bf16: 32 bytes, 8 bits: 16, 4 bits: 8), and the byte of their scale.
template <int kFormat>
struct Held16 {
    uint4 d[kFormat == DS_CACHE_BF16 ? 2 : 1];
    uint32_t sc;
};

// Elements 16 g .. 16 g + 15 of row `at` of page `id`.
template <int kDimOf, int kFormat>
__device__ __forceinline__ void load16(const PagedCache& cache, uint32_t id, uint32_t at, uint32_t g, Held16<kFormat>& h) {
    const uint32_t size = 1u << cache.page_shift;  // a page is below 2^20 bytes
    const uint8_t* page = cache.pages + ((size_t)id << cache.page_shift) * cache.row_bytes;
    if constexpr (kFormat == DS_CACHE_BF16) {
        const uint4* row = reinterpret_cast<const uint4*>(page + (at * kDimOf + 16 * g) * 2);
        h.d[0] = row[0];
        h.d[1] = row[1];
    } else if constexpr (kFormat == DS_CACHE_FP8) {
        h.d[0] = *reinterpret_cast<const uint4*>(page + (kDimOf == kDim ? at * kDimOf + 16 * g : (g * size + at) * 16));
        h.sc = page[size * kDimOf + at * (kDimOf / fp8::kBlock) + 16 * g / fp8::kBlock];
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(
            page + (kDimOf == kDim ? at * (kDim / 2 + kDim / int4::kGroup) + 8 * g : ((g / 2) * size + at) * 16 + (g % 2) * 8));
        h.d[0].x = v.x;
        h.d[0].y = v.y;
        h.sc = page[kDimOf == kDim ? at * (kDim / 2 + kDim / int4::kGroup) + kDim / 2 + g
                                   : size * (kDimOf / 2) + at * (kDimOf / int4::kGroup) + g];
    }
}

// ... as 8 bf16 pairs, exactly.
template <int kFormat>
__device__ __forceinline__ void widen16(const Held16<kFormat>& h, uint32_t (&w)[8]) {
    const uint32_t v[4] = {h.d[0].x, h.d[0].y, h.d[0].z, h.d[0].w};
    if constexpr (kFormat == DS_CACHE_BF16) {
        const uint32_t more[4] = {h.d[1].x, h.d[1].y, h.d[1].z, h.d[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = v[i], w[4 + i] = more[i];
    } else if constexpr (kFormat == DS_CACHE_FP8) {
        const uint32_t f = fp8::factor(h.sc);
#pragma unroll
        for (int i = 0; i < 4; ++i) fp8::widen(v[i], f, w + 2 * i);
    } else {
        int4::Factors f, unused;
        int4::factors2<0>(h.sc, f, unused);
        int4::widen(v[0], f, w);
        int4::widen(v[1], f, w + 4);
    }
}

__device__ __forceinline__ void st_global_v8(void* to, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

}  // namespace dsrows
