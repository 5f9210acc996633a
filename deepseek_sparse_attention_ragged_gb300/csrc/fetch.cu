// Rows read back from a paged cache: row slot[i] of entry seq[i], widened exactly and rounded
// once to the output's type.
//
// Bound by the bytes read and written (for a few rows: by the launch and three dependent loads, the
// indices, the page id and the row). A thread has 8 neighbouring elements of kUnroll rows, so that
// neighbours store 16 bytes (32 for fp32) each without a gap, and the loads of its rows are in
// flight together.

#include "cache_rows.cuh"
#include "kernels.h"

namespace dsrows {

namespace {

constexpr int kFetchThreads = 256;
constexpr int kFetchUnroll = 2;
constexpr int kFetchBlocks = 6;  // of a multiprocessor

// 8 elements from 4 bf16 pairs.
__device__ __forceinline__ void put8(__nv_bfloat16* out, const uint32_t (&w)[4], bool wide) {
    if (wide) {
        *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)(w[i / 2] >> 16 * (i % 2));
}
__device__ __forceinline__ float element(const uint32_t (&w)[4], int i) {
    return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}
__device__ __forceinline__ void put8(float* out, const uint32_t (&w)[4], bool wide) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<float4*>(out)[i] = make_float4(element(w, 4 * i), element(w, 4 * i + 1),
                                                            element(w, 4 * i + 2), element(w, 4 * i + 3));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = element(w, i);
}
__device__ __forceinline__ void put8(__half* out, const uint32_t (&w)[4], bool wide) {
    __align__(16) __half h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = __float2half_rn(element(w, i));
    if (wide) {
        *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(h);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = h[i];
}

}  // namespace

template <typename T, int kDimOf, int kFormat>
__global__ void __launch_bounds__(kFetchThreads) fetch_kernel(const __grid_constant__ FetchCall p) {
    constexpr int LANES = kDimOf / 8;  // threads of a row
    constexpr int ROWS = kFetchThreads / LANES;
    pdl_trigger();
    const int r = threadIdx.x / LANES, g = threadIdx.x % LANES;
    const uint32_t shift = p.cache.page_shift;
    const uint64_t step = (uint64_t)gridDim.x * (ROWS * kFetchUnroll);
    struct Place {
        int32_t seq[kFetchUnroll], slot[kFetchUnroll];
    };
    auto look = [&](uint64_t first, Place& at) {
#pragma unroll
        for (int u = 0; u < kFetchUnroll; ++u) {
            const uint64_t token = first + u * ROWS;
            at.seq[u] = token < p.tokens ? p.seq[token] : -1;
            at.slot[u] = token < p.tokens ? p.slot[token] : 0;
        }
    };
    auto page_of = [&](const Place& at, int32_t (&id)[kFetchUnroll]) {
#pragma unroll
        for (int u = 0; u < kFetchUnroll; ++u) {
            const uint32_t page_no = (uint32_t)at.slot[u] >> shift;
            const bool in = at.seq[u] >= 0 && (uint32_t)at.seq[u] < p.cache.entries && at.slot[u] >= 0 &&
                            page_no < p.cache.table_stride;
            id[u] = in ? p.cache.table[(uint64_t)at.seq[u] * p.cache.table_stride + page_no] : -1;
        }
    };
    pdl_wait();
    // The indices are looked up two steps ahead, the page ids one.
    uint64_t first = (uint64_t)blockIdx.x * (ROWS * kFetchUnroll) + r;
    Place now, next;
    int32_t id[kFetchUnroll];
    look(first, now);
    look(first + step, next);
    page_of(now, id);
#pragma unroll 1
    for (; first < p.tokens; first += step) {
        Held8 held[kFetchUnroll];
#pragma unroll
        for (int u = 0; u < kFetchUnroll; ++u) {
            if ((uint32_t)id[u] >= p.cache.num_pages) id[u] = -1;
            if (id[u] >= 0)
                held[u] = load8<kDimOf, kFormat>(p.cache, (uint32_t)id[u], (uint32_t)now.slot[u] & ((1u << shift) - 1), g);
        }
        int32_t next_id[kFetchUnroll];
        Place then;
        page_of(next, next_id);
        look(first + 2 * step, then);
#pragma unroll
        for (int u = 0; u < kFetchUnroll; ++u) {
            const uint64_t token = first + u * ROWS;
            const bool row = now.seq[u] != -1;  // also false past the last token
            if (g == 0 && p.invalid && token < p.tokens) p.invalid[token] = row && id[u] < 0 ? 1u : 0u;
            if (row) {
                uint32_t w[4] = {0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};  // no page: NaN
                if (id[u] >= 0) widen8<kFormat>(held[u], w);
                put8(static_cast<T*>(p.out) + token * p.out_stride + 8 * g, w, p.wide != 0);
            }
            id[u] = next_id[u];
        }
        now = next;
        next = then;
    }
}

template <typename T, int kDimOf>
static cudaError_t launch_rows(const FetchCall& p, int format, int num_sms, cudaStream_t stream, bool pdl) {
    constexpr uint64_t rows = kFetchThreads / (kDimOf / 8) * kFetchUnroll;
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
