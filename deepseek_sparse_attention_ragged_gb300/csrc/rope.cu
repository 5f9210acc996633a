// Rotary positions: pair (a, b) of a row at position t becomes
//   m (a cos x - b sin x), m (a sin x + b cos x),  x = t theta_i
// (x negated for the inverse, which is the transpose).
//
// Bound by the bytes moved: 2 (in place: 2 rot / dim) of the rows.
//
// Out of place (rope_rows_kernel) a thread moves the same 16 bytes of up to 16 heads of a
// token and its neighbours the rest of those rows, so that an access of a warp covers whole
// lines; the heads of a group are interleaved over the block, so that its rows at one time
// lie side by side. The angles of a thread's pairs stay in its registers, and in the half
// layout a pair's other element comes by shuffles. 4096 x 64 bf16 rows of 128, half of each
// rotated (134 MB, nothing in L2): 23.6 us, where a plain copy of them takes 21.1 us; 23.9
// with 8 heads a thread, 28.9 with 4. A thread per pair of halves took 27.0 us (each access
// 64 bytes of a line), the angles shared through shared memory 44 us (a barrier).
//
// In place (rope_kernel) a thread owns one unit of a row's rotated range, 16 bytes of
// interleaved pairs or 16 bytes from each half, for up to 8 heads: nobody else reads what
// it writes. 1021 x 64 fp32 rows of 512, 64 rotated: 4.2 us (33 MB, partly in L2); eight tokens of 64
// heads: 1.7 us. The same kernel serves half layouts whose range crosses a warp of
// rope_rows_kernel (rows of 12 or 24 pieces, say), and moves rows whose address, stride or
// range is not a multiple of 16 bytes element by element, one pair a unit; threads of
// their own then copy what is not rotated (the two cases above with rows off by one
// element: 38.5 us, each access a fraction of a line, and 6.6 us).

#include "rope.cuh"

namespace dsrows {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeThreadsMax = 544;   // one row a block: 1024 / 2 units and one more, in whole warps
constexpr uint32_t kGroupMax = 8;      // heads of a thread, at most: in place
constexpr uint32_t kRowsGroupMax = 16; // ... and out of place
constexpr uint32_t kFull = 512;        // threads an SM keeps busy with

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// N elements of a row: 16 bytes in one access, or element by element. kStream: what goes
// by once (out of place) is the first to leave the L2.
template <typename T, int N>
struct Piece {
    T v[N];
};
template <typename T, int N, bool kWide, bool kStream>
__device__ __forceinline__ Piece<T, N> get(const T* p) {
    Piece<T, N> r;
    if constexpr (kWide) {
        static_assert(N * sizeof(T) == 16, "16 bytes");
        const uint4* q = reinterpret_cast<const uint4*>(p);
        *reinterpret_cast<uint4*>(r.v) = kStream ? __ldcs(q) : *q;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r.v[i] = p[i];
    }
    return r;
}
template <typename T, int N, bool kWide, bool kStream>
__device__ __forceinline__ void put(T* p, const Piece<T, N>& r) {
    if constexpr (kWide) {
        uint4* q = reinterpret_cast<uint4*>(p);
        if constexpr (kStream) __stcs(q, *reinterpret_cast<const uint4*>(r.v));
        else *q = *reinterpret_cast<const uint4*>(r.v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = r.v[i];
    }
}

// Heads h, h + step, ... (H of them) of a token: one or two pieces of each row.
template <typename T, int N, int H, bool kWide>
struct Step {
    Piece<T, N> a[H], b[H];
    __device__ __forceinline__ void load(const T* x, uint64_t stride, uint32_t h, uint32_t h1, uint32_t step,
                                         uint32_t fa, uint32_t fb, bool two) {
#pragma unroll
        for (int k = 0; k < H; ++k)
            if (h + k * step < h1) {
                const T* row = x + (uint64_t)(h + k * step) * stride;
                a[k] = get<T, N, kWide, false>(row + fa);
                if (two) b[k] = get<T, N, kWide, false>(row + fb);
            }
    }
    __device__ __forceinline__ void store(T* out, uint64_t stride, uint32_t h, uint32_t h1, uint32_t step,
                                          uint32_t fa, uint32_t fb, bool two) const {
#pragma unroll
        for (int k = 0; k < H; ++k)
            if (h + k * step < h1) {
                T* row = out + (uint64_t)(h + k * step) * stride;
                put<T, N, kWide, false>(row + fa, a[k]);
                if (two) put<T, N, kWide, false>(row + fb, b[k]);
            }
    }
};

// Elements of one access: with kWide 16 bytes; else one pair (interleaved) or one
// element of each half.
template <typename T, bool kHalf, bool kWide>
constexpr int piece_len() {
    return kWide ? 16 / (int)sizeof(T) : (kHalf ? 1 : 2);
}

}  // namespace

template <typename T, bool kHalf, bool kWide>
__global__ void __launch_bounds__(kRopeThreadsMax) rope_kernel(const __grid_constant__ RopeCall p) {
    constexpr int N = piece_len<T, kHalf, kWide>();
    constexpr int M = kWide ? N : 1;  // a piece outside the range
    constexpr int PAIRS = kHalf ? N : N / 2;
    // Heads of a step: four pieces of 16 bytes a thread. With two heads the interleaved rotation
    // of 1021 x 64 fp32 rows in place took 5.7 us instead of 4.2.
    constexpr int H = kHalf ? 2 : 4;
    pdl_trigger();
    const uint32_t units = p.units + p.copies;
    const uint32_t u = threadIdx.x % units;
    const uint64_t item = (uint64_t)blockIdx.x * p.slots + threadIdx.x / units;
    const uint64_t token = item / p.groups;
    if (token >= p.tokens) return;
    // Heads h0, h0 + step, ...: the rows that a block's threads move at one time lie side by side.
    const uint32_t h0 = (uint32_t)(item - token * p.groups), h1 = p.heads, step = p.groups;
    pdl_wait();
    const T* x = static_cast<const T*>(p.x) + token * p.x_token;
    T* out = static_cast<T*>(p.out) + token * p.out_token;
    // A thread's heads go by in steps of H, whose loads are in flight together; the first step's loads are issued before
    // the angles are taken.
    if (u >= p.units) {
        // Pieces q and q + copies of the elements outside the range.
        const uint32_t before = p.rope.first / M, skip = p.rope.rot / M, pieces = p.dim / M - skip;
        const uint32_t q = u - p.units, q2 = q + p.copies;
        const bool two = q2 < pieces;
        const uint32_t fa = (q < before ? q : q + skip) * M, fb = two ? (q2 < before ? q2 : q2 + skip) * M : fa;
        Step<T, M, H, kWide> now;
        now.load(x, p.x_head, h0, h1, step, fa, fb, two);
        if (p.positions[token] < 0) return;
        for (uint32_t h = h0; h < h1; h += H * step) {
            now.store(out, p.out_head, h, h1, step, fa, fb, two);
            now.load(x, p.x_head, h + H * step, h1, step, fa, fb, two);
        }
        return;
    }
    const uint32_t fa = p.rope.first + u * N;
    const uint32_t fb = fa + p.rope.rot / 2;
    Step<T, N, H, kWide> now;  // b: the second half's piece (kHalf)
    now.load(x, p.x_head, h0, h1, step, fa, fb, kHalf);
    const int32_t pos = p.positions[token];
    if (pos < 0) return;
    float2 cs[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i)
        cs[i] = rope_turn(pos, p.rope.turns[u * PAIRS + i], p.rope.magnitude, p.inverse != 0);
    for (uint32_t h = h0; h < h1; h += H * step) {
#pragma unroll
        for (int k = 0; k < H; ++k)
            if (h + k * step < h1) {
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    T& ta = kHalf ? now.a[k].v[i] : now.a[k].v[(2 * i) % N];
                    T& tb = kHalf ? now.b[k].v[i] : now.a[k].v[(2 * i + 1) % N];
                    float va = to_f(ta), vb = to_f(tb);
                    rope_pair(va, vb, cs[i]);
                    ta = from_f<T>(va);
                    tb = from_f<T>(vb);
                }
            }
        now.store(out, p.out_head, h, h1, step, fa, fb, kHalf);
        now.load(x, p.x_head, h + H * step, h1, step, fa, fb, kHalf);
    }
}

// Out of place, rows, strides and ranges in pieces of 16 bytes: a thread moves piece v of
// p.group heads of a token, so that an access of a warp covers whole lines. In the half
// layout a pair's other element comes from its lane by shuffles: the launcher sees to it
// that a row's range lies in one warp.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const __grid_constant__ RopeCall p) {
    constexpr int N = 16 / (int)sizeof(T);
    constexpr int PAIRS = kHalf ? N : N / 2;
    constexpr int H = 4;  // heads whose loads are in flight together
    pdl_trigger();
    const uint32_t v = threadIdx.x % p.units, pairs = p.rope.rot / 2;
    const uint64_t item = (uint64_t)blockIdx.x * p.slots + threadIdx.x / p.units;
    const uint64_t token = item / p.groups;
    const bool there = token < p.tokens;
    const uint32_t step = p.groups, h0 = there ? (uint32_t)(item - token * p.groups) : 0u, h1 = there ? p.heads : 0u;
    const uint32_t f = v * N, e = f - p.rope.first;  // e: within the range, modulo 2^32
    const bool turns = e < p.rope.rot, low = e < pairs;
    const T* x = static_cast<const T*>(p.x) + (there ? token : 0) * p.x_token + f;
    T* out = static_cast<T*>(p.out) + (there ? token : 0) * p.out_token + f;
    pdl_wait();
    Piece<T, N> a[H];
    auto load = [&](uint32_t h) {
#pragma unroll
        for (int k = 0; k < H; ++k)
            if (h + k * step < h1) a[k] = get<T, N, true, true>(x + (uint64_t)(h + k * step) * p.x_head);
    };
    load(h0);
    const int32_t pos = there ? p.positions[token] : -1;
    float2 cs[PAIRS];
    if (turns) {
        const uint64_t* t = p.rope.turns + (!kHalf ? e / 2 : low ? e : e - pairs);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) cs[i] = rope_turn(pos, t[i], p.rope.magnitude, p.inverse != 0);
    }
    const int lane = threadIdx.x & 31;
    const int other = lane + (!turns ? 0 : low ? (int)(pairs / N) : -(int)(pairs / N));
    const uint32_t flip = low ? 0x80000000u : 0u;
    // Every lane of the warp goes round as often (the shuffles), by the same count of heads.
    for (uint32_t n = 0; n < p.group; n += H) {
        const uint32_t h = h0 + n * step;
#pragma unroll
        for (int k = 0; k < H; ++k) {
            if constexpr (kHalf) {
                Piece<T, N> b;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<uint32_t*>(b.v)[i] =
                        __shfl_sync(0xFFFFFFFFu, reinterpret_cast<const uint32_t*>(a[k].v)[i], other);
                if (turns)
#pragma unroll
                    for (int i = 0; i < N; ++i)  // rope_first or rope_second, by the sine's sign
                        a[k].v[i] = from_f<T>(fmaf(to_f(a[k].v[i]), cs[i].x,
                                                   __fmul_rn(to_f(b.v[i]), __uint_as_float(__float_as_uint(cs[i].y) ^ flip))));
            } else if (turns) {
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    float va = to_f(a[k].v[2 * i]), vb = to_f(a[k].v[2 * i + 1]);
                    rope_pair(va, vb, cs[i]);
                    a[k].v[2 * i] = from_f<T>(va);
                    a[k].v[2 * i + 1] = from_f<T>(vb);
                }
            }
            if (h + k * step < h1 && pos >= 0) put<T, N, true, true>(out + (uint64_t)(h + k * step) * p.out_head, a[k]);
        }
        load(h + H * step);
    }
}

template <typename T, bool kHalf>
static cudaError_t launch_rows(RopeCall& p, int num_sms, cudaStream_t stream, bool pdl) {
    p.units = p.dim / (16 / (uint32_t)sizeof(T));
    p.slots = kRopeThreads / p.units;
    uint32_t group = 1;
    while (group < kRowsGroupMax && group < p.heads &&
           p.tokens * ((p.heads + 2 * group - 1) / (2 * group)) * p.units >= (uint64_t)kFull * num_sms)
        group *= 2;
    p.group = group;
    p.groups = (p.heads + group - 1) / group;
    const uint64_t blocks = (p.tokens * p.groups + p.slots - 1) / p.slots;
    if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
    return launch_kernel(rope_rows_kernel<T, kHalf>, dim3((uint32_t)blocks), dim3(p.units * p.slots), 0, stream, pdl, p);
}

// Whether rope_rows_kernel takes the half layout of these rows: whole rows in a warp, or the
// range within one warp of a row of whole warps.
template <typename T>
static bool range_in_a_warp(const RopeCall& p) {
    constexpr uint32_t n = 16 / sizeof(T);
    const uint32_t pieces = p.dim / n, first = p.rope.first / n, last = first + p.rope.rot / n - 1;
    return 32 % pieces == 0 || (pieces % 32 == 0 && first / 32 == last / 32);
}

template <typename T, bool kHalf, bool kWide>
static cudaError_t launch(RopeCall& p, int num_sms, cudaStream_t stream, bool pdl) {
    constexpr int N = piece_len<T, kHalf, kWide>();
    constexpr int M = kWide ? N : 1;
    p.units = p.rope.rot / (kHalf ? 2 * N : N);
    p.copies = p.inplace ? 0 : (p.dim / M - p.rope.rot / M + 1) / 2;
    const uint32_t units = p.units + p.copies;  // at most dim / 2 + 1
    // Heads per thread: as many as leave kFull threads for every SM, at most kGroupMax.
    uint32_t group = 1;
    while (group < kGroupMax && group < p.heads &&
           p.tokens * ((p.heads + 2 * group - 1) / (2 * group)) * units >= (uint64_t)kFull * num_sms)
        group *= 2;
    p.group = group;
    p.groups = (p.heads + group - 1) / group;
    p.slots = units >= kRopeThreads ? 1 : kRopeThreads / units;
    const uint64_t items = p.tokens * p.groups;
    const uint64_t blocks = (items + p.slots - 1) / p.slots;
    if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
    return launch_kernel(rope_kernel<T, kHalf, kWide>, dim3((uint32_t)blocks), dim3(units * p.slots), 0, stream, pdl,
                         p);
}

template <typename T>
static cudaError_t launch_type(RopeCall& p, int layout, int num_sms, cudaStream_t stream, bool pdl) {
    constexpr uint64_t n = 16 / sizeof(T);
    const uint64_t strides = p.x_token | p.x_head | p.out_token | p.out_head;
    const uint64_t range = p.rope.first | (layout == DS_ROPE_HALF ? p.rope.rot / 2 : p.rope.rot) | (p.inplace ? 0 : p.dim);
    const bool wide = ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) & 15) == 0 &&
                      ((strides | range) & (n - 1)) == 0;
    if (wide && !p.inplace) {
        if (layout == DS_ROPE_INTERLEAVED) return launch_rows<T, false>(p, num_sms, stream, pdl);
        if (range_in_a_warp<T>(p)) return launch_rows<T, true>(p, num_sms, stream, pdl);
    }
    if (layout == DS_ROPE_HALF)
        return wide ? launch<T, true, true>(p, num_sms, stream, pdl) : launch<T, true, false>(p, num_sms, stream, pdl);
    return wide ? launch<T, false, true>(p, num_sms, stream, pdl) : launch<T, false, false>(p, num_sms, stream, pdl);
}

cudaError_t launch_rope(RopeCall p, int dtype, int layout, int num_sms, cudaStream_t stream, bool pdl) {
    if (p.tokens == 0) return cudaSuccess;
    if (dtype == DS_F32) return launch_type<float>(p, layout, num_sms, stream, pdl);
    if (dtype == DS_F16) return launch_type<__half>(p, layout, num_sms, stream, pdl);
    return launch_type<__nv_bfloat16>(p, layout, num_sms, stream, pdl);
}

}  // namespace dsrows
