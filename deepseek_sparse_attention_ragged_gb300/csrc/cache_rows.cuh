// Eight neighbouring elements of a cached row, in any page type.
#pragma once

#include "common.cuh"
#include "fp8.cuh"
#include "int4.cuh"
#include "kernels.h"

namespace dsrows {

// As they are held, and the byte of their scale.
struct Held8 {
    uint4 d;
    uint32_t sc;
};

// Elements 8 g .. 8 g + 7 of row `at` of page `id`.
template <int kDimOf, int kFormat>
__device__ __forceinline__ Held8 load8(const PagedCache& cache, uint32_t id, size_t at, uint32_t g) {
    const uint8_t* page = cache.pages + ((size_t)id << cache.page_shift) * cache.row_bytes;
    const size_t size = (size_t)1 << cache.page_shift;
    Held8 h = {};
    if constexpr (kFormat == DS_CACHE_BF16) {
        h.d = *reinterpret_cast<const uint4*>(page + (at * kDimOf + 8 * g) * 2);
    } else if constexpr (kFormat == DS_CACHE_FP8) {
        const uint2 v = *reinterpret_cast<const uint2*>(
            kDimOf == kDim ? page + at * kDimOf + 8 * g : page + (size_t)(g / 2) * (16 * size) + at * 16 + (g % 2) * 8);
        h.d.x = v.x;
        h.d.y = v.y;
        h.sc = page[size * kDimOf + at * (kDimOf / fp8::kBlock) + 8 * g / fp8::kBlock];
    } else if constexpr (kDimOf == kDim) {
        const uint8_t* row = page + at * cache.row_bytes;
        h.d.x = *reinterpret_cast<const uint32_t*>(row + 4 * g);
        h.sc = row[kDimOf / 2 + g / 2];
    } else {
        h.d.x = *reinterpret_cast<const uint32_t*>(page + (size_t)(g / 4) * (16 * size) + at * 16 + (g % 4) * 4);
        h.sc = page[size * (kDimOf / 2) + at * (kDimOf / int4::kGroup) + g / 2];
    }
    return h;
}

// ... as 4 bf16 pairs, exactly.
template <int kFormat>
__device__ __forceinline__ void widen8(const Held8& h, uint32_t (&w)[4]) {
    if constexpr (kFormat == DS_CACHE_BF16) {
        w[0] = h.d.x, w[1] = h.d.y, w[2] = h.d.z, w[3] = h.d.w;
    } else if constexpr (kFormat == DS_CACHE_FP8) {
        const uint32_t f = fp8::factor(h.sc);
        fp8::widen(h.d.x, f, w);
        fp8::widen(h.d.y, f, w + 2);
    } else {
        int4::Factors f, unused;
        int4::factors2<0>(h.sc, f, unused);
        int4::widen(h.d.x, f, w);
    }
}

}  // namespace dsrows
