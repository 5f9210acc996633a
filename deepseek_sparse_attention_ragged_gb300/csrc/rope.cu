// Rotary positions: pair (a, b) of a row at position t becomes
//   m (a cos x - b sin x), m (a sin x + b cos x),  x = t theta_i
// (x negated for the inverse, which is the transpose).
//
// Bound by the bytes moved: 2 (in place: 2 rot / dim) of the rows. A thread owns
// one unit of a row's rotated range: 16 bytes of interleaved pairs, or 16 bytes
// from each half, with their angles in registers, and rotates that unit of a
// group of heads of one token, so sine and cosine are taken once per group; out of
// place, threads of their own copy two pieces each of what is not rotated. The
// heads of a group are interleaved over the block, so that its accesses at one time
// cover whole rows side by side. 4096 x 64 bf16 rows of 128, half of each rotated, out
// of place (134 MB): 27.3 us with inputs that are not in L2, 22.4 us replayed on the same
// ones (a plain copy of them: 21.1 us); replayed, with consecutive heads per thread
// 27.6 us, without the streaming hints 24.5 us, with the copies in the rotating threads
// 31.5 us. What is left is that an access takes 64 bytes of a line (23.3 us if it took
// all 128); threads that read whole lines and share the angles through shared memory
// needed a barrier and twice the loads, and took 44 us. Eight rows of 64 heads in
// place: 1.6 us; 1021 x 64 fp32 rows in place 4.2 us.
// A row whose address, stride or range is not a multiple of 16 bytes is moved
// by elements, one pair a unit.

#include "rope.cuh"

namespace dsrows {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeThreadsMax = 544;   // one row a block: 1024 / 2 units and one more, in whole warps
constexpr uint32_t kGroupMax = 8;
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

// N elements of a row: 16 bytes in one access, or element by element. kStream: the rows
// go by once (out of place), so they are the first to leave the L2.
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
template <typename T, int N, int H, bool kWide, bool kStream>
struct Step {
    Piece<T, N> a[H], b[H];
    __device__ __forceinline__ void load(const T* x, uint64_t stride, uint32_t h, uint32_t h1, uint32_t step,
                                         uint32_t fa, uint32_t fb, bool two) {
#pragma unroll
        for (int k = 0; k < H; ++k)
            if (h + k * step < h1) {
                const T* row = x + (uint64_t)(h + k * step) * stride;
                a[k] = get<T, N, kWide, kStream>(row + fa);
                if (two) b[k] = get<T, N, kWide, kStream>(row + fb);
            }
    }
    __device__ __forceinline__ void store(T* out, uint64_t stride, uint32_t h, uint32_t h1, uint32_t step,
                                          uint32_t fa, uint32_t fb, bool two) const {
#pragma unroll
        for (int k = 0; k < H; ++k)
            if (h + k * step < h1) {
                T* row = out + (uint64_t)(h + k * step) * stride;
                put<T, N, kWide, kStream>(row + fa, a[k]);
                if (two) put<T, N, kWide, kStream>(row + fb, b[k]);
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

template <typename T, bool kHalf, bool kWide, bool kStream>
__global__ void __launch_bounds__(kRopeThreadsMax) rope_kernel(const __grid_constant__ RopeCall p) {
    constexpr int N = piece_len<T, kHalf, kWide>();
    constexpr int M = kWide ? N : 1;  // a piece outside the range
    constexpr int PAIRS = kHalf ? N : N / 2;
    // Heads of a step: four pieces of 16 bytes a thread. With two heads the interleaved rotation
    // of 1021 x 64 fp32 rows in place took 5.7 us instead of 4.2; with four the half layout's
    // 4096 x 64 bf16 rows out of place 24.5 us instead of 22.4.
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
        Step<T, M, H, kWide, kStream> now;
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
    Step<T, N, H, kWide, kStream> now;  // b: the second half's piece (kHalf)
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

template <typename T, bool kHalf, bool kWide, bool kStream>
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
    return launch_kernel(rope_kernel<T, kHalf, kWide, kStream>, dim3((uint32_t)blocks), dim3(units * p.slots), 0, stream, pdl,
                         p);
}

template <typename T>
static cudaError_t launch_type(RopeCall& p, int layout, int num_sms, cudaStream_t stream, bool pdl) {
    constexpr uint64_t n = 16 / sizeof(T);
    const uint64_t strides = p.x_token | p.x_head | p.out_token | p.out_head;
    const uint64_t range = p.rope.first | (layout == DS_ROPE_HALF ? p.rope.rot / 2 : p.rope.rot) | (p.inplace ? 0 : p.dim);
    const bool wide = ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) & 15) == 0 &&
                      ((strides | range) & (n - 1)) == 0;
    if (layout == DS_ROPE_HALF)
        return !wide ? launch<T, true, false, false>(p, num_sms, stream, pdl)
               : p.inplace ? launch<T, true, true, false>(p, num_sms, stream, pdl)
                           : launch<T, true, true, true>(p, num_sms, stream, pdl);
    return !wide ? launch<T, false, false, false>(p, num_sms, stream, pdl)
           : p.inplace ? launch<T, false, true, false>(p, num_sms, stream, pdl)
                       : launch<T, false, true, true>(p, num_sms, stream, pdl);
}

cudaError_t launch_rope(RopeCall p, int dtype, int layout, int num_sms, cudaStream_t stream, bool pdl) {
    if (p.tokens == 0) return cudaSuccess;
    if (dtype == DS_F32) return launch_type<float>(p, layout, num_sms, stream, pdl);
    if (dtype == DS_F16) return launch_type<__half>(p, layout, num_sms, stream, pdl);
    return launch_type<__nv_bfloat16>(p, layout, num_sms, stream, pdl);
}

}  // namespace dsrows
