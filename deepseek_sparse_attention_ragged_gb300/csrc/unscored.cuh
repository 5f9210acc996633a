// What a scoring thread leaves when a wait gives up (compiled for the host too, where it is tested).
#pragma once

#include <math.h>
#include <stdint.h>

namespace dsrows {

// -inf for the thread's keys of tiles it, it + tiles, ... below `mine`: key j in the first,
// `keys` more in each next, those below kv_len.
__host__ __device__ inline void unscored(float* out, uint32_t it, uint32_t mine, uint32_t tiles, uint32_t j, uint32_t keys,
                                         uint32_t kv_len) {
#pragma unroll 1
    for (; it < mine; it += tiles, j += keys)
        if (j < kv_len) out[j] = -INFINITY;
}

}  // namespace dsrows
