// Append rows to a paged cache: rotate (optional), round to the cache's type,
// store into the row's page.
//
// Bound by the bytes of the rows read and written (and, for a few rows, by the
// launch). A lane owns 16 consecutive elements, which is one group of the 4-bit
// type, so its scale needs no exchange: a warp holds one 512-wide row or four
// 128-wide ones. The lanes of a row share its sines and cosines through shared
// memory (each takes rot / 2 / lanes of them); in the half layout a pair's other
// element comes from its lane by a shuffle where the halves are whole groups, and is
// read again where they are not. The row is fetched while its place is looked up
// (index, page id, page: three dependent loads).
//
// Eight 512-wide rows: 2.5 us. Long runs, over three sets of inputs (most of them in L2) and over
// sets of 300 MB and more, with the bytes' time at the measured copy bandwidth:
//   32768 x 128, bf16 into 4-bit pages, half of each rotated, and the values   7.6 / 10.2 us (2.9)
//   32768 x 128, bf16 into bf16 pages                                          6.2 /  8.9 us (2.5)
//   8191 x 512, bf16 into 4-bit pages, and the values                          6.3 /  8.9 us (2.8)
//   8191 x 512, fp32 into bf16 pages                                           6.2 /  8.2 us (3.7)
// Waits for loads are the largest stall in all of them (half of the issue slots are used on 4-bit
// keys, a quarter on fp32 rows): a warp's one set of rows waits for its dependent look-ups, which only
// other warps hide, and a lane's 16-byte accesses lie 32 or 64 bytes apart from its neighbour's.
// The instructions count next: 14.3 us on the keys with divisions for quotients and per-element
// index arithmetic. More blocks on an SM than the 48 registers allow made it slower (8.9 us at 40
// registers, 11.2 us at 32, against 8.4).

#include "int4.cuh"
#include "rope.cuh"

namespace dsrows {

namespace {

constexpr int kAppendThreads = 128;

template <typename T>
__device__ __forceinline__ float widen_f(T v) {
    return (float)v;
}

}  // namespace

template <typename T, int kDimOf, bool kInt4>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendCall p) {
    constexpr int G = int4::kGroup;
    constexpr int LANES = kDimOf / G;  // lanes of a row
    constexpr int ROWS = kAppendThreads / LANES;
    // Pair i of a row at [i mod 16][i / 16], padded: lanes read with strides of 8 or 16 pairs, and
    // the rows of a warp lie in different banks.
    constexpr int W = kDimOf / 32 + 1;
    constexpr int PAD = LANES == 32 ? 0 : 4;
    __shared__ float2 trig_s[ROWS][16 * W + PAD];
    auto pair_at = [](uint32_t i) { return (i % 16) * W + i / 16; };
    pdl_trigger();
    const int r = threadIdx.x / LANES, g = threadIdx.x % LANES;
    const uint64_t token = (uint64_t)blockIdx.x * ROWS + r;
    const bool there = token < p.tokens;
    pdl_wait();
    // The row is fetched while its place is looked up.
    float y[G];
    const T* x = static_cast<const T*>(p.x) + token * p.x_stride + g * G;
    if (there) {
        if (p.wide) {
            __align__(16) T v[G];
#pragma unroll
            for (int i = 0; i < (int)(G * sizeof(T) / 16); ++i)
                reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(x)[i];
#pragma unroll
            for (int i = 0; i < G; ++i) y[i] = widen_f(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < G; ++i) y[i] = widen_f(x[i]);
        }
    }
    // The row's place. The checks are uniform over its lanes.
    const int32_t seq = there ? p.seq[token] : -1;
    bool ok = false;
    size_t page = 0;
    uint32_t at = 0;
    int32_t pos = 0;
    if (there && seq != -1) {
        const int32_t slot = p.slot[token];
        const uint32_t page_no = (uint32_t)slot >> p.cache.page_shift;
        ok = seq >= 0 && (uint32_t)seq < p.cache.entries && slot >= 0 && page_no < p.cache.table_stride;
        if (ok) {
            const int32_t id = p.cache.table[(uint64_t)seq * p.cache.table_stride + page_no];
            ok = id >= 0 && (uint32_t)id < p.cache.num_pages;
            page = (size_t)(uint32_t)id;
            at = (uint32_t)slot & ((1u << p.cache.page_shift) - 1);
        }
        if (p.rope.rot) {
            pos = p.positions[token];
            ok = ok && pos >= 0;
        }
    }
    if (there && g == 0 && p.invalid) p.invalid[token] = seq != -1 && !ok ? 1u : 0u;

    if (p.rope.rot) {
        const uint32_t pairs = p.rope.rot / 2;
        if (ok)
            for (uint32_t i0 = g; i0 < pairs; i0 += 4 * LANES) {
                uint64_t turns[4];  // four pairs' loads together
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i0 + k * LANES < pairs) turns[k] = p.rope.turns[i0 + k * LANES];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i0 + k * LANES < pairs)
                        trig_s[r][pair_at(i0 + k * LANES)] = rope_turn(pos, turns[k], p.rope.magnitude, false);
            }
        __syncwarp();
        const uint32_t e0 = g * G - p.rope.first;  // this lane's elements within the range, modulo 2^32
        const bool inside = e0 < p.rope.rot, low = e0 < pairs;
        if (p.whole) {
            // The range begins and ends with lanes' groups, and so do its halves.
            if (p.half) {
                const int other = (threadIdx.x & 31) + (!inside ? 0 : low ? (int)pairs / G : -((int)pairs / G));
                const float2* trig = &trig_s[r][pair_at(!inside ? 0 : low ? e0 : e0 - pairs)];
                const uint32_t flip = low ? 0x80000000u : 0u;
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const float z = __shfl_sync(0xFFFFFFFFu, y[i], other);
                    if (inside && ok) {
                        // rope_first or rope_second, by the sine's sign.
                        const float2 cs = trig[i * W];
                        y[i] = fmaf(y[i], cs.x, __fmul_rn(z, __uint_as_float(__float_as_uint(cs.y) ^ flip)));
                    }
                }
            } else if (inside && ok) {
                const float2* trig = &trig_s[r][pair_at(e0 / 2)];
#pragma unroll
                for (int i = 0; i < G; i += 2) rope_pair(y[i], y[i + 1], trig[i / 2 * W]);
            }
        } else if (ok && p.half) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const uint32_t e = e0 + i;
                if (e < p.rope.rot) {
                    const bool first = e < pairs;
                    const float z = widen_f(x[first ? i + (int)pairs : i - (int)pairs]);
                    float a = first ? y[i] : z, b = first ? z : y[i];
                    rope_pair(a, b, trig_s[r][pair_at(first ? e : e - pairs)]);
                    y[i] = first ? a : b;
                }
            }
        } else if (ok) {
#pragma unroll
            for (int i = 0; i < G; i += 2)  // first is even: a pair lies in one lane
                if (e0 + i < p.rope.rot) rope_pair(y[i], y[i + 1], trig_s[r][pair_at((e0 + i) / 2)]);
        }
    }
    if (!ok) return;
    uint8_t* base = p.cache.pages + (page << p.cache.page_shift) * p.cache.row_bytes;
    __nv_bfloat16* held_out = p.values ? p.values + token * kDimOf + g * G : nullptr;
    __align__(16) __nv_bfloat16 held[G];
    if constexpr (kInt4) {
        uint32_t word[2];
        float h[G];
        const uint8_t scale = int4::quantise(y, word, h);
        if constexpr (kDimOf == kDim) {
            uint8_t* row = base + (size_t)at * p.cache.row_bytes;
            *reinterpret_cast<uint2*>(row + 8 * g) = make_uint2(word[0], word[1]);
            row[kDimOf / 2 + g] = scale;
        } else {
            // Plane g / 2 holds 32 values of each row; then the scales.
            const size_t size = (size_t)1 << p.cache.page_shift;
            *reinterpret_cast<uint2*>(base + (g / 2) * size * 16 + at * 16 + (g & 1) * 8) =
                make_uint2(word[0], word[1]);
            base[size * (kDimOf / 2) + at * (kDimOf / G) + g] = scale;
        }
        if (!held_out) return;
#pragma unroll
        for (int i = 0; i < G; ++i) held[i] = __float2bfloat16_rn(h[i]);
    } else {
#pragma unroll
        for (int i = 0; i < G; ++i) held[i] = __float2bfloat16_rn(y[i]);
        uint4* row = reinterpret_cast<uint4*>(base + (size_t)at * p.cache.row_bytes + g * G * 2);
        row[0] = reinterpret_cast<const uint4*>(held)[0];
        row[1] = reinterpret_cast<const uint4*>(held)[1];
        if (!held_out) return;
    }
    reinterpret_cast<uint4*>(held_out)[0] = reinterpret_cast<const uint4*>(held)[0];
    reinterpret_cast<uint4*>(held_out)[1] = reinterpret_cast<const uint4*>(held)[1];
}

template <typename T, int kDimOf>
static cudaError_t launch_rows(const AppendCall& p, int format, cudaStream_t stream, bool pdl) {
    constexpr uint64_t rows = kAppendThreads / (kDimOf / int4::kGroup);
    const dim3 grid((uint32_t)((p.tokens + rows - 1) / rows));
    if (format == DS_CACHE_INT4)
        return launch_kernel(append_kernel<T, kDimOf, true>, grid, dim3(kAppendThreads), 0, stream, pdl, p);
    return launch_kernel(append_kernel<T, kDimOf, false>, grid, dim3(kAppendThreads), 0, stream, pdl, p);
}

template <typename T>
static cudaError_t launch_type(const AppendCall& p, uint32_t dim, int format, cudaStream_t stream, bool pdl) {
    return dim == kDim ? launch_rows<T, kDim>(p, format, stream, pdl) : launch_rows<T, kIdxDim>(p, format, stream, pdl);
}

cudaError_t launch_append(const AppendCall& p, int dtype, uint32_t dim, int format, cudaStream_t stream, bool pdl) {
    if (p.tokens == 0) return cudaSuccess;
    if (dtype == DS_F32) return launch_type<float>(p, dim, format, stream, pdl);
    if (dtype == DS_F16) return launch_type<__half>(p, dim, format, stream, pdl);
    return launch_type<__nv_bfloat16>(p, dim, format, stream, pdl);
}

}  // namespace dsrows
