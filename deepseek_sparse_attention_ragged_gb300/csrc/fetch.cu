// Rows read back from a paged cache: row slot[i] of entry seq[i], widened exactly and rounded
// once to the output's type.
//
// Bound by the bytes read and written (for a few rows: by the launch and three dependent loads, the
// indices, the page id and the row). A thread has 16 neighbouring elements, a group of the 4-bit type and 16 bytes of the
// 8-bit one, and stores them by 32 bytes; the indices of its rows are looked up two steps ahead and their page
// ids one step, so that a row's load waits for neither.
//
// 37 4-bit rows 1.5 us. 262144 8-bit keys into bf16 (34 MB read, 67 MB written: 15.3 us at the measured copy bandwidth)
// 19.3 us; 20001 8-bit rows of 512 into 32 bits (51 MB: 7.4 us) 9.1 us. Two rows a thread in flight made no difference;
// with each row's look-ups in front of it, and stores of 16 bytes, the two took 29.4 and 13.7 us. Waits for loads are the largest
// stall; the widening uses half of the integer pipe.

#include "cache_rows.cuh"
#include "kernels.h"

namespace dsrows {

namespace {

constexpr int kFetchThreads = 256;
constexpr int kFetchBlocks = 6;  // of a multiprocessor

// 16 elements from 8 bf16 pairs; `aligned`: to 32 bytes, 16 bytes or the type (2, 1, 0).
__device__ __forceinline__ float element(const uint32_t (&w)[8], int i) {
    return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}
__device__ __forceinline__ void put_words(void* out, const uint32_t (&w)[8], uint32_t aligned) {
    if (aligned == 2) {
        st_global_v8(out, w);
    } else if (aligned == 1) {
        static_cast<uint4*>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) static_cast<uint16_t*>(out)[i] = (uint16_t)(w[i / 2] >> 16 * (i % 2));
    }
}
__device__ __forceinline__ void put16(__nv_bfloat16* out, const uint32_t (&w)[8], uint32_t aligned) {
    put_words(out, w, aligned);
}
__device__ __forceinline__ void put16(__half* out, const uint32_t (&w)[8], uint32_t aligned) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2 two = __floats2half2_rn(element(w, 2 * i), element(w, 2 * i + 1));
        h[i] = *reinterpret_cast<const uint32_t*>(&two);
    }
    put_words(out, h, aligned);
}
__device__ __forceinline__ void put16(float* out, const uint32_t (&w)[8], uint32_t aligned) {
    if (aligned == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) out[i] = element(w, i);
        return;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __float_as_uint(element(w, 8 * k + i));
        put_words(out + 8 * k, f, aligned);
    }
}

}  // namespace

template <typename T, int kDimOf, int kFormat>
__global__ void __launch_bounds__(kFetchThreads) fetch_kernel(const __grid_constant__ FetchCall p) {
    constexpr int LANES = kDimOf / 16;  // threads of a row
    constexpr int ROWS = kFetchThreads / LANES;
    pdl_trigger();
    const int r = threadIdx.x / LANES, g = threadIdx.x % LANES;
    const uint32_t shift = p.cache.page_shift;
    const uint64_t step = (uint64_t)gridDim.x * ROWS;
    struct Place {
        int32_t seq, slot;
    };
    auto look = [&](uint64_t token) {
        return token < p.tokens ? Place{p.seq[token], p.slot[token]} : Place{-1, 0};
    };
    auto page_of = [&](const Place& at) -> int32_t {
        const uint32_t page_no = (uint32_t)at.slot >> shift;
        const bool in = at.seq >= 0 && (uint32_t)at.seq < p.cache.entries && at.slot >= 0 && page_no < p.cache.table_stride;
        return in ? p.cache.table[(uint64_t)at.seq * p.cache.table_stride + page_no] : -1;
    };
    pdl_wait();
    uint64_t token = (uint64_t)blockIdx.x * ROWS + r;
    Place now = look(token), next = look(token + step);
    int32_t id = page_of(now);
#pragma unroll 1
    for (; token < p.tokens; token += step) {
        Held16<kFormat> held;
        const bool there = id >= 0 && (uint32_t)id < p.cache.num_pages;
        if (there)
            load16<kDimOf, kFormat>(p.cache, (uint32_t)id, (uint32_t)now.slot & ((1u << shift) - 1), g, held);
        id = page_of(next);
        const Place then = look(token + 2 * step);
        if (g == 0 && p.invalid) p.invalid[token] = now.seq != -1 && !there ? 1u : 0u;
        if (now.seq != -1) {
            uint32_t w[8];
            if (there) {
                widen16(held, w);
            } else {  // no page: NaN
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = 0x7FC07FC0u;
            }
            put16(static_cast<T*>(p.out) + token * p.out_stride + 16 * g, w, p.aligned);
        }
        now = next;
        next = then;
    }
}

template <typename T, int kDimOf>
static cudaError_t launch_rows(const FetchCall& p, int format, int num_sms, cudaStream_t stream, bool pdl) {
    constexpr uint64_t rows = kFetchThreads / (kDimOf / 16);
    // Blocks with the same number of steps each.
    const uint64_t work = (p.tokens + rows - 1) / rows, most = (uint64_t)num_sms * kFetchBlocks;
    const uint64_t steps = (work + most - 1) / most;
    const dim3 grid((uint32_t)((work + steps - 1) / steps));
    auto launch = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kFetchThreads), 0, stream, pdl, p); };
    if (format == DS_CACHE_INT4) return launch(fetch_kernel<T, kDimOf, DS_CACHE_INT4>);
    if (format == DS_CACHE_FP8) return launch(fetch_kernel<T, kDimOf, DS_CACHE_FP8>);
    return launch(fetch_kernel<T, kDimOf, DS_CACHE_BF16>);
}

template <typename T>
static cudaError_t launch_type(const FetchCall& p, uint32_t dim, int format, int num_sms, cudaStream_t stream, bool pdl) {
    return dim == kDim ? launch_rows<T, kDim>(p, format, num_sms, stream, pdl)
                       : launch_rows<T, kIdxDim>(p, format, num_sms, stream, pdl);
}

cudaError_t launch_fetch(const FetchCall& p, int dtype, uint32_t dim, int format, int num_sms, cudaStream_t stream,
                         bool pdl) {
    if (p.tokens == 0) return cudaSuccess;
    if (dtype == DS_F32) return launch_type<float>(p, dim, format, num_sms, stream, pdl);
    if (dtype == DS_F16) return launch_type<__half>(p, dim, format, num_sms, stream, pdl);
    return launch_type<__nv_bfloat16>(p, dim, format, num_sms, stream, pdl);
}

}  // namespace dsrows
