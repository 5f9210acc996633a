// Sink-softmax attention over every cached row, for rows that share a prefix: per row r and head h,
// over the slots j < kv_len[r] (the first prefix_len of them the same rows for every r),
//   l_j = scale * q_h . g_j,  m = max(sink_h, max l_j),
//   out_h = sum_j exp(l_j - m) g_j / (exp(sink_h - m) + sum_j exp(l_j - m)),
// with g_j the 512-wide cache row (keys and values are the same).
//
// The work is a list of segments: the prefix once for every two rows of the batch, then what each
// row has behind it. A segment is a run of tiles of 128 slots, and the tiles of all segments are
// dealt out to pairs of CTAs (2-CTA clusters on neighbouring SMs) in equal runs. A pair's run within one
// segment is a part: it carries the running maximum and sum of the softmax and the accumulated output
// through its tiles, and leaves them in the workspace. A second kernel joins each row's
// parts, in their order, with the sink.
//
// A pair works on 2 x 64 query vectors (CTA c holds the 64 heads of the segment's row c) with
// cta_group::2 MMAs of M = 128:
//   S[128 heads x 128 slots] = Q . G^T      (K = 512; CTA c brings slots 64 c .. 64 c + 63)
//   O[128 heads x 512 dims] += P . G        (K = 128 slots; CTA c brings dims 256 j + 128 c .. + 127)
// O of 64 heads takes 256 TMEM columns in this layout, which leaves room for four S; with one CTA and M = 128 it would
// fill TMEM alone. A CTA has the 64 slots of the K form and the 256 dims of the V form that it brings, half of
// what one CTA by itself would read. Each keeps its own softmax: its 64 heads see every slot of the tile, so
// nothing but the operands crosses the pair.
//
// Warp roles: 0 looks up the tiles' rows, 1 issues S and 2 P . G (in the pair's first CTA), 3 loads the queries, 4 to 11
// do the softmax, two sets on alternate tiles (a thread has 64 slots of one head), and the others bring the
// operands. The K form (the CTA's 64 slots, 128 dims a unit) and the V form (64 slots and 128 of the CTA's dims a unit) of the
// rows have rings of their own, of 16 KB units: a tile of S comes ahead of P . G of the one before. bf16 rows come by TMA, in boxes of rows of one
// page; packed rows are widened in registers on their way to shared memory, or, where enough rows of the batch share
// them, once for all by a kernel beforehand.
// Rows past a segment's end and rows without a page are zeros with probability 0.
//
// In a captured graph, all launches of a call (the time that its operations or its bytes alone would take):
//   3 rows, 300 shared and up to 40 more, bf16 pages           11.2 us (0.1)
//   1 row of 131073, bf16                                      37.1 us (19.9, bytes)
//   8 rows, 65536 shared and up to 999 more, bf16              54.0 us (36.3, operations)
//   5 rows, 40007 shared and up to 1000 more, 4 bits           39.3 us (13.9, operations)
//   63 rows, 20001 shared and up to 311 more, 8 bits           117 us (87.5, operations)
// A tile takes a pair 1.3 us on bf16 rows (its MMAs 1.0): the tensor cores are busy for 65% of the attention kernel at
// eight rows and 75% at 63. No unit is full; a ring unit's way round (commit, wait, 16 KB by TMA, wait, MMAs) takes about
// 2,000 cycles and the rings hold seven eighths of a tile, which is what shared memory has room for. Taken out one by
// one, at 63 rows (then 119 us): the loads 109, seven of eight S MMAs 112, half of P . G 115, a quarter of the bytes 117,
// the exponentials 119; 8 KB units 143, one P buffer 153, three K and four V units 128. The rest is fixed: some 10 us of
// launches, first loads, the parts (2 us: a multiprocessor stores 32 bytes a cycle, by bulk copies too) and their join,
// which a short call or a single row sees most. Packed rows widened as they are used take 2.7 us (8 bits) or 2.5 us (4
// bits) a tile: every value passes registers. A single long row of bf16 takes 1.7 us a tile, which is 5.9 TB/s of DRAM.

#include <float.h>

#include <algorithm>

#include "cache_rows.cuh"
#include "common.cuh"
#include "fp8.cuh"
#include "int4.cuh"
#include "kernels.h"

namespace dsrows {

namespace {

constexpr int kTile = kPrefixTile;            // slots of a tile
constexpr int kUnitBytes = 16384;             // a ring unit: [64 slots][128 dims], two blocks of 64 dims
constexpr int kQBytes = kHeads * kDim * 2;    // the CTA's query row, 8 blocks [64 heads][64 dims]
constexpr int kPBytes = kHeads * kTile * 2;   // P of a tile: 2 blocks [64 heads][64 slots]
constexpr int kBoxRows = kPrefixBoxRows;      // most rows of a TMA box
constexpr int kPlaceBufs = 4;                 // tiles whose rows are looked up
// A kernel's source of rows: the pages of a format, or bf16 rows widened beforehand.
constexpr int kWidened = -1;
template <int kFormat>
constexpr bool kByTma = kFormat == DS_CACHE_BF16 || kFormat == kWidened;
constexpr int kSoftmaxWarp = 4, kBuildWarp = 12;  // two sets of four softmax warps
// Units of the K form, which hold a tile, and of the V form. Where the rows come by TMA, three units of the V form are
// enough, and P is held for two tiles (P of the next tile is written while P G of this one runs); widening
// sets another pace, and has four, and one P.
constexpr uint32_t kKUnits = 4;
template <int kFormat>
constexpr uint32_t kVUnits = kByTma<kFormat> ? 3 : 4;
template <int kFormat>
constexpr uint32_t kPBufs = kByTma<kFormat> ? 2 : 1;
constexpr uint32_t kUnitsMax = 8;
// Warps that bring operands, those of them that fill a unit, and those that read a tile's places for a form.
template <int kFormat>
constexpr int kBuildWarps = kByTma<kFormat> ? kKUnits + kVUnits<kFormat> : 16;
template <int kFormat>
constexpr int kFillers = kByTma<kFormat> ? 1 : 8;
template <int kFormat>
constexpr int kReaders = kByTma<kFormat> ? 4 : 16;
template <int kFormat>
constexpr int kThreads = 32 * (kBuildWarp + kBuildWarps<kFormat>);
constexpr uint32_t kOCol = 128;               // TMEM: two S of 64 columns, O, two more S
constexpr uint32_t kSBufs = 4;
// A set's warps meet once a tile, so a warp may write its largest logits of the set's next tile before another
// has read those of this one, but not those of the one after.
constexpr uint32_t kRedBufs = 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint16_t kBoth = 3;                 // the CTAs of a pair
// The running maximum is raised only when a tile's exceeds it by more than this (in units of ln 2): the
// accumulated output is then scaled, and the weights stay below 2^8.
constexpr float kSlack = 8.0f;

// Tiles whose weights' products with the rows are summed in TMEM, at most: a longer run is folded into its part in the
// workspace piece by piece. The tensor cores cut a product off at 2^-25 of the sum that it is added to (seen where a run of
// ones stopped at 2^26), so the 16 of a step take up to 2^-21 of the sum and the 4096 steps of a piece 2^-9 of it, if all cuts
// were largest; and no wait for a piece lasts for seconds. A piece costs less than 10 us, beside some
// 900 of its tiles (64 rows over 155000 bf16 rows).
constexpr uint32_t kPieceTiles = 512;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kNoRow = -1, kBadRow = -2;
constexpr uint32_t kMasked = 1;     // some slot of the tile has no row
constexpr uint32_t kByThreads = 2;  // the tile is not whole boxes of rows of one page each

template <int kFormat>
struct Layout {
    static constexpr size_t ring = 0;  // K units, then V units
    static constexpr size_t q = ring + (size_t)(kKUnits + kVUnits<kFormat>) * kUnitBytes;
    static constexpr size_t p = q + kQBytes;
    static constexpr size_t place = p + kPBufs<kFormat> * (size_t)kPBytes;  // i32 [kPlaceBufs][128]
    static constexpr size_t red = place + kPlaceBufs * kTile * 4;          // f32 [2][kRedBufs][128]
    static constexpr size_t maxima = red + 2 * kRedBufs * 128 * 4;         // f32 [2][128]
    static constexpr size_t bars = maxima + 2 * 128 * 4;
};

struct __align__(8) Bars {
    // In the pair's first CTA, from both:
    uint64_t full[kUnitsMax];
    uint64_t q_full, p_full[2], s_free[kSBufs], o_read;
    // In each CTA:
    uint64_t empty[kUnitsMax];
    uint64_t q_free, s_full[kSBufs], pv_done[2], m_ready[2], drained;
    uint64_t place_full[kPlaceBufs], place_free[kPlaceBufs];
    uint32_t form[kPlaceBufs];     // of the tile: kMasked, kByThreads
    uint32_t tmem_base;
};

template <int kFormat>
constexpr size_t kSmem = Layout<kFormat>::bars + sizeof(Bars) + 1024;
static_assert(kSmem<DS_CACHE_BF16> <= 227 * 1024 && kSmem<DS_CACHE_INT4> <= 227 * 1024, "shared memory");

// ---- the pair's tcgen05 forms and barriers ---------------------------------------------------

__device__ __forceinline__ void umma2_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on `bar` of both CTAs when the MMAs issued so far complete.
__device__ __forceinline__ void umma2_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(kBoth)
        : "memory");
}
// Arrive on the first CTA's barrier. What an arrival announces is this CTA's own shared memory (through the
// async proxy, after a proxy fence) or TMEM, which its own tensor core reads: the order within the CTA is
// what counts. (With cluster scope an arrival takes 323 cycles instead of 8, and waits for every load in flight.)
__device__ __forceinline__ void arrive_first_cta(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(smem_u32(bar), 0))
                 : "memory");
}
__device__ __forceinline__ void arrive_first_cta_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cluster.b64 _, [%0], %1;" ::"r"(
                     cluster_addr(smem_u32(bar), 0)),
                 "r"(bytes)
                 : "memory");
}
// A tile of a tensor map into this CTA's shared memory, its bytes counted on the first CTA's barrier.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(dst),
        "l"(map), "r"(cluster_addr(smem_u32(bar), 0)), "r"(x), "r"(y)
        : "memory");
}
// A bounded wait of a whole warp (its lanes go on or give up together), whose first tries read no timer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t* status) {
    bool ok = false;
    for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
    if (!ok) ok = mbar_wait(bar, parity, status);
    return __all_sync(0xFFFFFFFFu, ok);
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// Byte offset of 16-byte chunk `ch` of row `row` in a 128-byte-swizzled block of 128-byte rows.
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t ch) { return row * 128 + ((ch ^ (row & 7)) << 4); }

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
    return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
    return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
          "l"(*reinterpret_cast<const uint64_t*>(&c)));
    return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void sync_softmax(uint32_t set) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");
}

// ---- the operands ------------------------------------------------------------------------------

// The dim of a row that dim d of CTA `rank`'s half of it is (V form).
__device__ __forceinline__ uint32_t v_dim(uint32_t d, uint32_t rank) { return 256 * (d >> 7) + 128 * rank + (d & 127); }

// A lane's values of a step of a packed unit, eight rows of 128 dims: a 16-byte piece of one row (4 bits) or
// two (8 bits). Eight lanes, whose 16-byte accesses are one turn of the load and store unit, have two rows by
// four pieces (8 bits) or four by two (4 bits): few cache lines a turn, and chunks that the swizzle puts into
// different banks. (With eight rows to eight lanes a load took 27 cycles, 3,500 a tile on 8 bits.)
template <int kFormat>
struct Piece {
    static constexpr uint32_t kValues = kFormat == DS_CACHE_FP8 ? 16 : 32;  // of 16 bytes
    static constexpr uint32_t kN = kFormat == DS_CACHE_FP8 ? 2 : 1;         // the second is 64 dims on
    uint4 d[kN];
    uint32_t sc;

    static __device__ __forceinline__ uint32_t row(uint32_t lane) {
        return kFormat == DS_CACHE_FP8 ? 2 * (lane >> 3) + (lane & 1) : 4 * (lane >> 3 & 1) + (lane & 3);
    }
    static __device__ __forceinline__ uint32_t first(uint32_t lane) {
        return kValues * (kFormat == DS_CACHE_FP8 ? lane >> 1 & 3 : 2 * (lane >> 4) + (lane >> 2 & 1));
    }
    // The pieces at dims dim and dim + 64 of the row at `place`; zeros without one.
    __device__ __forceinline__ void load(const PagedCache& cache, int32_t place, uint32_t dim) {
        const uint32_t where = (uint32_t)max(place, 0);
        if constexpr (kFormat == DS_CACHE_FP8) {
            const uint32_t shift = cache.page_shift, in_page = where & ((1u << shift) - 1);
            const uint8_t* page = cache.pages + (size_t)(where - in_page) * (kDim + kDim / fp8::kBlock);
            const uint8_t* row = page + (size_t)in_page * kDim + dim;
            d[0] = d[1] = make_uint4(0, 0, 0, 0);
            sc = 127;
            if (place >= 0) {
                d[0] = __ldcg(reinterpret_cast<const uint4*>(row));
                d[1] = __ldcg(reinterpret_cast<const uint4*>(row + 64));
                sc = __ldcg(page + ((size_t)kDim << shift) + in_page * (kDim / fp8::kBlock) + dim / fp8::kBlock);
            }
        } else {
            const uint8_t* row = cache.pages + (size_t)where * (kDim / 2 + kDim / int4::kGroup);
            d[0] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
            sc = 0;
            if (place >= 0) {
                d[0] = __ldcg(reinterpret_cast<const uint4*>(row + dim / 2));
                sc = __ldcg(reinterpret_cast<const uint16_t*>(row + kDim / 2 + dim / int4::kGroup));
            }
        }
    }
    // Widened into the unit: dst(ch) is the shared address of its row's dims 8 ch .. 8 ch + 7.
    template <class Dst>
    __device__ __forceinline__ void store(uint32_t first_dim, Dst dst) const {
#pragma unroll
        for (uint32_t n = 0; n < kN; ++n) {
            const uint32_t words[4] = {d[n].x, d[n].y, d[n].z, d[n].w};
            const uint32_t ch = (first_dim + 64 * n) / 8;
            if constexpr (kFormat == DS_CACHE_FP8) {
                const uint32_t f = fp8::factor(sc);
#pragma unroll
                for (uint32_t c = 0; c < 2; ++c) {
                    uint32_t o[4];
                    fp8::widen(words[2 * c], f, o);
                    fp8::widen(words[2 * c + 1], f, o + 2);
                    st_shared_v4(dst(ch + c), o[0], o[1], o[2], o[3]);
                }
            } else {
                int4::Factors f[2];
                int4::factors2<0>(sc, f[0], f[1]);
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) {
                    uint32_t o[4];
                    int4::widen(words[c], f[c >> 1], o);
                    st_shared_v4(dst(ch + c), o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The TMEM columns of S of tile `it`.
__device__ __forceinline__ uint32_t s_col(uint32_t it) { return (it & 1) * 64 + (it & 2) * 192; }

// ---- the pair's tiles --------------------------------------------------------------------------

// A run of a pair's tiles within one segment, or a piece of it.
struct Part {
    uint32_t seg;
    uint32_t start;   // its first tile's first slot
    uint32_t end;     // the segment's last slot + 1
    uint32_t tiles;
    bool more;        // a piece behind the run's first
};

// The parts of pair k in order, by pieces: for (Walk w(p, k); w.next(part);). What is dealt out in equal runs
// (pair k's begins at floor(line k / pairs)) is a line on which a segment's tiles follow p.seg_cost units for its set-up.
struct Walk {
    const PrefixParams& p;
    uint32_t t, end, seg, had;  // had: the last part's segment + 1
    __device__ __forceinline__ Walk(const PrefixParams& params, uint32_t pair) : p(params) {
        t = p.run * pair + p.rest * pair / p.pairs;
        end = p.run * (pair + 1) + p.rest * (pair + 1) / p.pairs;
        seg = had = 0;
        while (t < end && p.begin[seg + 1] <= t) ++seg;
    }
    __device__ __forceinline__ bool next(Part& part) {
        while (t < end) {
            while (p.begin[seg + 1] <= t) ++seg;  // t is below the last bound
            const uint32_t first = p.begin[seg] + p.seg_cost, stop = min(end, p.begin[seg + 1]);
            t = max(t, first);
            if (t < stop) {
                const bool shared = seg < p.groups;
                part.seg = seg;
                part.start = (shared ? 0u : p.prefix_len) + (t - first) * kTile;
                part.end = shared ? p.prefix_len : p.kv_len[seg - p.groups];
                part.tiles = min(stop - t, kPieceTiles);
                part.more = had == seg + 1;
                had = seg + 1;
                t += part.tiles;
                return true;
            }
            t = max(t, stop);
        }
        return false;
    }
};

}  // namespace

template <int kFormat>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<kFormat>, 1)
    prefix_attn_kernel(const __grid_constant__ PrefixParams p) {
    using L = Layout<kFormat>;
    constexpr uint32_t kV = kVUnits<kFormat>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Bars* bar = reinterpret_cast<Bars*>(smem + L::bars);
    int32_t* place_s = reinterpret_cast<int32_t*>(smem + L::place);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1, pair = blockIdx.x >> 1;
    const uint32_t ring = smem_u32(smem + L::ring);

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kKUnits + kV; ++i) {
            mbar_init(&bar->full[i], 2 * kFillers<kFormat>);
            mbar_init(&bar->empty[i], 1);
        }
        mbar_init(&bar->q_full, 2);
        mbar_init(&bar->o_read, 16);
        mbar_init(&bar->q_free, 1);
        mbar_init(&bar->drained, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar->p_full[i], 8);
            mbar_init(&bar->pv_done[i], 1);
            mbar_init(&bar->m_ready[i], 4);
        }
        for (uint32_t i = 0; i < kSBufs; ++i) {
            mbar_init(&bar->s_free[i], 8);
            mbar_init(&bar->s_full[i], 1);
        }
        for (int i = 0; i < kPlaceBufs; ++i) {
            mbar_init(&bar->place_full[i], 1);
            mbar_init(&bar->place_free[i], 2 * kReaders<kFormat> + 4);  // K form, V form, softmax
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bar->tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive_release();  // both CTAs' barriers are set before either arrives on the other's
    cluster_wait_acquire();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem_base, 0);
    // The pair's tiles. (What depends on the parameters alone comes before the wait for the kernel before this one.)
    const Walk all(p, pair);
    Part part;
    uint32_t n = 0;
    for (Walk w = all; w.next(part);) n += part.tiles;
    if (threadIdx.x == 32 * 3) {
        tma_prefetch_map(&p.qmap);
        if (kByTma<kFormat>) tma_prefetch_map(&p.kvmap);
    }
    // The first part's query and page ids into L2 (the kernel before may yet write them: nothing is read here).
    Walk ahead = all;
    if (ahead.next(part)) {
        const uint32_t r = part.seg < p.groups ? min(2 * part.seg + rank, p.rows - 1) : part.seg - p.groups;
        if (threadIdx.x < kQBytes / 128)
            prefetch_l2(reinterpret_cast<const uint8_t*>(p.q) + (size_t)p.q_row[r] * kQBytes + threadIdx.x * 128);
        else if (kFormat != kWidened && warp == 16 && lane < 2)
            prefetch_l2(p.cache.table + (part.seg < p.groups ? 0 : (size_t)(part.seg - p.groups) * p.cache.table_stride) +
                        (min(part.start + (kTile - 1) * lane, part.end - 1) >> p.cache.page_shift));
    }
    pdl_wait();
    pdl_trigger();
    // The first block starts first; a wait that gives up reports seconds later.
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

    uint32_t it = 0;  // the tiles so far
    if (warp == 0) {
        // ---- the tiles' rows: places in the pool ----------------------------------------------
        bool ok = true;
        for (Walk w = all; ok && w.next(part);) {
            const uint32_t entry = part.seg < p.groups ? 0 : part.seg - p.groups;
            const int32_t* table = p.cache.table + (size_t)entry * p.cache.table_stride;
            const uint32_t shift = p.cache.page_shift;
            // Widened rows: the part's first one.
            const uint32_t wide = part.seg < p.groups ? part.start : p.wide_begin[entry] * kTile + part.start - p.prefix_len;
            for (uint32_t i = 0; i < part.tiles; ++i, ++it) {
                const uint32_t buf = it % kPlaceBufs;
                int32_t id[4], at[4];
                bool all = true;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t j = part.start + i * kTile + lane + 32 * k;
                    id[k] = kFormat != kWidened && j < part.end ? table[j >> shift] : -1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t j = part.start + i * kTile + lane + 32 * k;
                    if (j >= part.end) at[k] = kNoRow;
                    else if (kFormat == kWidened) at[k] = (int32_t)(wide + i * kTile + lane + 32 * k);
                    else if (id[k] < 0 || (uint32_t)id[k] >= p.cache.num_pages) at[k] = kBadRow;
                    else at[k] = (int32_t)(((uint32_t)id[k] << shift) + (j & ((1u << shift) - 1)));
                    all = all && at[k] >= 0;
                }
                all = __all_sync(0xFFFFFFFFu, all);
                if (!wait_warp(&bar->place_free[buf], (it / kPlaceBufs & 1) ^ 1, p.status)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) place_s[buf * kTile + lane + 32 * k] = at[k];
                const uint32_t box = min(1u << shift, (uint32_t)kBoxRows);
                if (lane == 0) bar->form[buf] = (all ? 0u : kMasked) | (all && part.start % box == 0 ? 0u : kByThreads);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->place_full[buf]);
            }
        }
    } else if (warp <= 2) {
        // ---- the MMAs, issued in the first CTA for both: warp 1 S = Q G^T, warp 2 O += P G. (One warp for both took
        // 3,900 cycles a tile, twice the MMAs' time: waits of 100 to 200 cycles and 20 or so an MMA, one after another.)
        if (rank == 0) {
            // Unit u of a form, the lanes looking at all the form's units together: lane i at `full` in phase `parity`. Bits
            // are the units known to be full; lane u + units and later ones look at a barrier before its time.
            auto unit_full = [&](uint64_t* full, uint32_t parity, uint32_t u, uint32_t units, uint32_t& bits) -> bool {
                uint64_t start = 0;
                for (uint32_t tries = 1; !(bits >> u & 1); ++tries) {
                    bits = __ballot_sync(0xFFFFFFFFu, mbar_try_wait(full, parity)) & 15 & ((1u << (u + units)) - 1);
                    if (tries % 64 == 0) {
                        const uint64_t now = __shfl_sync(0xFFFFFFFFu, global_timer_ns(), 0);
                        if (start == 0) start = now;
                        if (now - start > kWaitBudgetNs) {
                            if (lane == 0) atomicOr(p.status, kStatusWaitTimeout);
                            return false;
                        }
                    }
                }
                return true;
            };
            uint32_t n_part = 0;
            bool ok = true;
            if (warp == 1) {
                constexpr uint32_t idesc = idesc_bf16_f32(128, 128);
                const uint64_t a_desc = smem_desc_sw128_kmajor(smem_u32(smem + L::q));
                for (Walk w = all; ok && w.next(part); ++n_part)
                    for (uint32_t i = 0; i < part.tiles; ++i, ++it) {
                        ok = i != 0 || wait_warp(&bar->q_full, n_part & 1, p.status);
                        ok = ok && wait_warp(&bar->s_free[it % kSBufs], (it / kSBufs & 1) ^ 1, p.status);
                        const uint32_t d = tmem + s_col(it);
                        uint32_t full = 0;
#pragma unroll
                        for (uint32_t u = 0; u < 4; ++u) {
                            ok = ok && unit_full(&bar->full[lane & 3], it & 1, u, kKUnits, full);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t b_desc = smem_desc_sw128_kmajor(ring + u * kUnitBytes);
                            if (elect_one()) {
#pragma unroll
                                for (uint32_t ks = 0; ks < 8; ++ks) {
                                    const uint32_t at = ((ks >> 2) * 8192 + (ks & 3) * 32) >> 4;
                                    umma2_bf16(d, a_desc + (u * kUnitBytes >> 4) + at, b_desc + at, idesc,
                                               u == 0 && ks == 0 ? 0u : 1u);
                                }
                                umma2_commit(&bar->empty[u]);
                                if (u == 3) {
                                    umma2_commit(&bar->s_full[it % kSBufs]);
                                    if (i + 1 == part.tiles) umma2_commit(&bar->q_free);
                                }
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
            } else {
                constexpr uint32_t idesc = idesc_bf16_f32(128, 256) | 1u << 16;  // B is MN-major
                for (Walk w = all; ok && w.next(part); ++n_part)
                    for (uint32_t i = 0; i < part.tiles; ++i, ++it) {
                        ok = wait_warp(&bar->p_full[it & 1], it >> 1 & 1, p.status);
                        // A part begins O anew, once the part before has been read.
                        ok = ok && (i != 0 || n_part == 0 || wait_warp(&bar->o_read, (n_part - 1) & 1, p.status));
                        const uint64_t a_desc = smem_desc_sw128_kmajor(smem_u32(smem + L::p) + it % kPBufs<kFormat> * kPBytes);
                        // The lane's unit of all. The last tile's lie in the units of the K form, which it has done with.
                        const uint32_t mine = 4 * it + (lane & 3);
                        const bool in_k = kByTma<kFormat> && it + 1 == n;
                        uint64_t* bars = &bar->full[in_k ? lane & 3 : kKUnits + mine % kV];
                        const uint32_t parity = (in_k ? n : mine / kV) & 1;
                        uint32_t full = 0;
#pragma unroll
                        for (uint32_t v = 0; v < 4; ++v) {
                            ok = ok && unit_full(bars, parity, v, in_k ? kKUnits : kV, full);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t slot = in_k ? v : kKUnits + (4 * it + v) % kV;
                            const uint64_t b_desc = smem_desc_sw128_mnmajor(ring + slot * kUnitBytes, 8192, 1024);
                            if (elect_one()) {
#pragma unroll
                                for (uint32_t ks = 0; ks < 4; ++ks)
                                    umma2_bf16(tmem + kOCol + 128 * (v & 1), a_desc + (((v >> 1) * 8192 + ks * 32) >> 4),
                                               b_desc + (ks * 2048 >> 4), idesc, i == 0 && v < 2 && ks == 0 ? 0u : 1u);
                                umma2_commit(&bar->empty[slot]);
                                if (v == 3) umma2_commit(&bar->pv_done[it & 1]);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
            }
            // Whatever was issued is done before the CTAs leave.
            if (elect_one()) umma2_commit(&bar->drained);
            __syncwarp();
            (void)wait_warp(&bar->drained, 0, p.status);
        }
    } else if (warp >= kSoftmaxWarp && warp < kBuildWarp) {
        // ---- softmax: two sets of four warps, each every second tile; thread = TMEM lane = (head, half of the
        // tile's slots). A set passes the running maxima on before it takes its exponentials.
        const uint32_t set = (warp - kSoftmaxWarp) >> 2;
        const uint32_t row = (threadIdx.x - 32 * kSoftmaxWarp) & 127, head = row & 63, half = row >> 6;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float* red_s = reinterpret_cast<float*>(smem + L::red) + 128 * kRedBufs * set;
        float* m_s = reinterpret_cast<float*>(smem + L::maxima);  // [2][128]
        const uint32_t p_row = smem_u32(smem + L::p) + set % kPBufs<kFormat> * kPBytes + half * 8192;
        const float scale = p.scale_log2;
        const float2 scale2 = make_float2(scale, scale);
        uint32_t met = 0;  // a set's warps meet once a tile
        float m_run = 0.0f;  // the maximum that the run's pieces so far refer to
        bool ok = true;
        for (Walk w = all; ok && w.next(part);) {
            float m = -INFINITY, sum = 0.0f;  // the maximum that the sum refers to, before the scale
            uint32_t bad = 0;
            const uint32_t begin = it;
            for (const uint32_t stop = it + part.tiles; it < stop; ++it) {
                if ((it & 1) != set) continue;
                const uint32_t pbuf = it % kPlaceBufs;
                const uint32_t sbuf = it % kSBufs, s_cols = lanes + s_col(it);
                if (!(ok = wait_warp(&bar->place_full[pbuf], it / kPlaceBufs & 1, p.status))) break;
                const bool masked = bar->form[pbuf] & kMasked;
                if (!(ok = wait_warp(&bar->s_full[sbuf], it / kSBufs & 1, p.status))) break;
                tc_fence_after();
                const ::int4* at = reinterpret_cast<const ::int4*>(place_s + pbuf * kTile + half * 64);
                // The largest S (the scale is positive). 0 * S * scale is NaN exactly where a logit is not finite.
                float top = -INFINITY;
                float2 odd = make_float2(0.0f, 0.0f);
#pragma unroll 1
                for (uint32_t h = 0; h < 2; ++h) {
                    uint32_t v[32];
                    tmem_ld_x32(s_cols + 32 * h, v);
                    tmem_ld_wait();
                    float2 t[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        t[c] = make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
                        odd = fma2(mul2(t[c], scale2), make_float2(0.0f, 0.0f), odd);
                    }
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const ::int4 a = at[8 * h + c];
                            if (a.x == kBadRow || a.y == kBadRow || a.z == kBadRow || a.w == kBadRow) bad = 1;
                            if (a.x < 0) t[2 * c].x = -INFINITY;
                            if (a.y < 0) t[2 * c].y = -INFINITY;
                            if (a.z < 0) t[2 * c + 1].x = -INFINITY;
                            if (a.w < 0) t[2 * c + 1].y = -INFINITY;
                        }
                    }
                    float tops[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tops[c] = fmaxf(t[c].x, t[c].y);
#pragma unroll
                    for (int c = 4; c < 16; ++c) tops[c & 3] = fmaxf(tops[c & 3], fmaxf(t[c].x, t[c].y));
                    top = fmaxf(top, fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
                }
                if (!(odd.x + odd.y == 0.0f)) bad = 1;
                float* red = red_s + 128 * (it / 2 % kRedBufs);
                red[row] = top;
                sync_softmax(set);
                ++met;
                top = fmaxf(top, red[row ^ 64]);
                // The running maximum of the tile before, and this tile's. A head's two threads decide alike.
                if (it > 0 && !(ok = wait_warp(&bar->m_ready[set ^ 1], (it - 1) >> 1 & 1, p.status))) break;
                float f = 1.0f;  // of O
                if (it == begin) {
                    m = finite_f(top) ? top : 0.0f;
                } else {
                    const float before = m_s[128 * (set ^ 1) + row];
                    float now = before;
                    if ((top - before) * scale > kSlack && finite_f(top)) {
                        now = top;
                        f = exp2_fast((before - now) * scale);
                    }
                    if (now != m) sum *= exp2_fast((m - now) * scale);  // the set's sum, of its own tiles
                    m = now;
                }
                m_s[128 * set + row] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->m_ready[set]);
                const bool moved = __any_sync(0xFFFFFFFFu, f != 1.0f);
                // The weights, from S again: 64 logits and 64 weights at once are more registers than there are. S less the
                // maximum, then scaled: a product with the scale less a rounded maximum would be off by up to half a
                // step of the maximum, which is past any weight for logits from 2^31 on. The product with the rows takes them
                // rounded to bf16, 2^-8 of a weight at most (the sums are of the weights themselves): against 64 bits the
                // output is off by 2.0e-3 (2-norm) where a row has some hundred slots and by 1.7e-3 where it has many,
                // 1.7e-3 of both being its own rounding. Their low parts would be as many MMAs again.
                const float2 minus = make_float2(-m, -m);
                float2 s2[2] = {};
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    uint32_t v[32], w16[16];
                    tmem_ld_x32(s_cols + 32 * h, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 x =
                            mul2(add2(make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), minus), scale2);
                        float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                        if (masked) {
                            const int2 a = reinterpret_cast<const int2*>(at)[16 * h + c];
                            e = make_float2(a.x < 0 ? 0.0f : e.x, a.y < 0 ? 0.0f : e.y);
                        }
                        s2[c & 1] = add2(s2[c & 1], e);
                        w16[c] = pack_bf16(e.x, e.y);
                    }
                    if (h == 0) {
                        // P G of the tile that had this P is done.
                        const uint32_t had = it - kPBufs<kFormat>;
                        if (it >= kPBufs<kFormat> && !(ok = wait_warp(&bar->pv_done[had & 1], had >> 1 & 1, p.status))) break;
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            arrive_first_cta(&bar->s_free[sbuf]);
                            mbar_arrive(&bar->place_free[pbuf]);
                        }
                    }
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c)
                        st_shared_v4(p_row + swizzled(head, 4 * h + c), w16[4 * c], w16[4 * c + 1], w16[4 * c + 2],
                                     w16[4 * c + 3]);
                }
                if (!ok) break;
                s2[0] = add2(s2[0], s2[1]);
                sum += s2[0].x + s2[0].y;
                if (moved) {
                    // So is that of the tile before this one: O may be scaled. (Its barrier's phase before this one is
                    // known to be over: P G of the tiles is done in their order.)
                    if (!(ok = wait_warp(&bar->pv_done[set ^ 1], (it - 1) >> 1 & 1, p.status))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (uint32_t c = 0; c < 256; c += 32) {
                        uint32_t o[32];
                        tmem_ld_x32(lanes + kOCol + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st_x32(lanes + kOCol + c, o);
                    }
                    tmem_st_wait();
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_first_cta(&bar->p_full[set]);
            }
            if (!ok) break;
            // ---- the part's state: the maximum that O refers to, each set's sum, and O -------------------
            const uint32_t last = it - 1;
            const uint32_t r = part.seg < p.groups ? 2 * part.seg + rank : rank == 0 ? part.seg - p.groups : p.rows;
            const bool mine = r < p.rows;  // the pair's second CTA may have no row
            float* out = p.parts + ((size_t)(pair + part.seg) * 2 + rank) * kPrefixPartFloats;
            if ((last & 1) != set) {
                if (!(ok = wait_warp(&bar->m_ready[set ^ 1], last >> 1 & 1, p.status))) break;
                const float now = m_s[128 * (set ^ 1) + row];
                if (now != m) sum *= exp2_fast((m - now) * scale);
                m = now;
            }
            // What the run's pieces before left here and this one, by a common maximum. (A thread reads only what it wrote.)
            const float top = part.more ? fmaxf(m_run, m) : m;
            const float f_run = part.more ? exp2_fast((m_run - top) * scale) : 0.0f, f = exp2_fast((m - top) * scale);
            m_run = top;
            if (mine) {
                float* to_sum = out + kHeads + 4 * head + 2 * set + half;
                if (bad) sum = __int_as_float(0x7FC00000);  // a flag is NaN
                *to_sum = part.more ? fmaf(*to_sum, f_run, sum * f) : sum;
                if (half == 0 && (last & 1) == set) out[head] = m_run * scale;
            }
            // The set that did not have the last tile waits for its own first, so that the other barrier is in that phase.
            if (kPBufs<kFormat> == 2 && (last & 1) != set && last > 0 &&
                !(ok = wait_warp(&bar->pv_done[set], (last - 1) >> 1 & 1, p.status)))
                break;
            if (!(ok = wait_warp(&bar->pv_done[last & 1], last >> 1 & 1, p.status))) break;
            tc_fence_after();
            float4* to = reinterpret_cast<float4*>(out + kPrefixHeadFloats) + 32 * set * 128 + row;
#pragma unroll 1
            for (uint32_t c = 0; c < 128; c += 32) {  // each set a half of the columns
                uint32_t o[32];
                tmem_ld_x32(lanes + kOCol + 128 * set + c, o);
                tmem_ld_wait();
                if (mine) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float4 v = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                               __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                        float4* at = to + (c / 4 + k) * 128;
                        if (part.more) {
                            const float4 was = *at;
                            v = make_float4(fmaf(was.x, f_run, v.x * f), fmaf(was.y, f_run, v.y * f),
                                            fmaf(was.z, f_run, v.z * f), fmaf(was.w, f_run, v.w * f));
                        }
                        *at = v;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_first_cta(&bar->o_read);
        }
        // A warp that gave up still meets the others.
        for (; met < (n + 1 - set) / 2; ++met) sync_softmax(set);
    } else if (warp == 3) {
        // ---- each part's query, once the MMAs of the part before have read theirs --------------
        uint32_t n_part = 0;
        for (Walk w = all; w.next(part); ++n_part) {
            if (n_part > 0 && !wait_warp(&bar->q_free, (n_part - 1) & 1, p.status)) break;
            const uint32_t r = part.seg < p.groups ? min(2 * part.seg + rank, p.rows - 1) : part.seg - p.groups;
            if (lane == 0) arrive_first_cta_expect(&bar->q_full, kQBytes);
            __syncwarp();
            if (lane < 8)
                tma_load_pair(smem_u32(smem + L::q) + lane * 8192, &p.qmap, &bar->q_full, 64 * lane,
                              (int)(p.q_row[r] * kHeads));
        }
    } else if (warp >= kBuildWarp) {
        // ---- operands -----------------------------------------------------------------------------
        auto looked_up = [&](uint32_t of) {
            return wait_warp(&bar->place_full[of % kPlaceBufs], of / kPlaceBufs & 1, p.status);
        };
        auto read = [&](uint32_t of) {  // this warp has read the tile's places
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->place_free[of % kPlaceBufs]);
        };
        if constexpr (kByTma<kFormat>) {
            // Warp b fills unit b: of the K form one of every tile and then, when S of the last tile is done, one of its
            // V form; of the other tiles' V form every kV-th.
            const uint32_t slot = warp - kBuildWarp, dst = ring + slot * kUnitBytes;
            const uint32_t box = kFormat == kWidened ? kBoxRows : min(1u << p.cache.page_shift, (uint32_t)kBoxRows);
            for (uint32_t lap = 0;; ++lap) {
                const bool v_unit = slot >= kKUnits;
                const uint32_t g = v_unit ? slot - kKUnits + lap * kV : 4 * min(lap, n - 1) + slot, of = g / 4, u = g % 4;
                if (n == 0 || (v_unit ? of + 1 >= n : lap > n)) break;
                const bool v_form = v_unit || lap == n;
                if (!looked_up(of)) break;
                // Boxes of rows: lane = (64 dims, row group).
                const uint32_t first = v_form ? 64 * (u >> 1) : 64 * rank, row = lane % (64 / box) * box, dims = lane / (64 / box);
                const bool boxes = kFormat == kWidened || !(bar->form[of % kPlaceBufs] & kByThreads);
                const int32_t* at = place_s + of % kPlaceBufs * kTile;
                // Widened runs end with zeros up to a whole tile.
                const int32_t y = kFormat == kWidened ? at[0] + (int32_t)(first + row) : at[first + row];
                if (!wait_warp(&bar->empty[slot], (lap & 1) ^ 1, p.status)) break;
                if (boxes) {
                    if (lane == 0) arrive_first_cta_expect(&bar->full[slot], kUnitBytes);
                    __syncwarp();
                    if (dims < 2)
                        tma_load_pair(dst + dims * 8192 + row * 128, &p.kvmap, &bar->full[slot],
                                      (int)(v_form ? v_dim(128 * (u & 1) + 64 * dims, rank) : 128 * u + 64 * dims), y);
                    read(of);
                } else {
                    // Rows by 16 bytes, zeros for those that are missing.
#pragma unroll 8
                    for (uint32_t k = lane; k < kUnitBytes / 16; k += 32) {
                        const uint32_t row = k >> 4, ch = k & 15;  // 8 dims
                        const int32_t place = at[first + row];
                        const uint32_t dim = v_form ? v_dim(128 * (u & 1) + 8 * ch, rank) : 128 * u + 8 * ch;
                        cp_async16_or_zero(dst + (ch >> 3) * 8192 + swizzled(row, ch & 7),
                                           p.cache.pages + (size_t)max(place, 0) * (2 * kDim) + 2 * dim, place >= 0);
                    }
                    read(of);
                    cp_async_commit_group();
                    cp_async_wait_group<0>();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_first_cta(&bar->full[slot]);
                }
            }
        } else {
            // Packed rows are widened by two teams of eight warps: team t fills units t and t + 2 of each form, warp s
            // of it the unit's step s, eight rows of 128 dims. The loads of a form are issued as the form before it is stored. (Two warps to a unit, four
            // steps each, took 4000 cycles from a free unit to a full one, and the ring holds no more than a tile.)
            const uint32_t team = (warp - kBuildWarp) >> 3, s = warp - kBuildWarp & 7;
            Piece<kFormat> held[2];
            // The forms in the order in which the MMAs take them: K(0), K(1), V(0), K(2), V(1), .., K(n - 1), V(n - 2),
            // V(n - 1). Form f's tile and kind.
            auto tile_of = [&](uint32_t f) { return f == 0 ? 0 : f == 2 * n - 1 ? n - 1 : f & 1 ? (f + 1) / 2 : f / 2 - 1; };
            auto v_form_of = [&](uint32_t f) { return f == 2 * n - 1 || (f > 0 && !(f & 1)); };
            auto fetch = [&](uint32_t f, uint32_t k) {
                const uint32_t of = tile_of(f), u = team + 2 * k, d = Piece<kFormat>::first(lane);
                const int32_t* at = place_s + of % kPlaceBufs * kTile + Piece<kFormat>::row(lane);
                if (v_form_of(f)) held[k].load(p.cache, at[64 * (u >> 1) + 8 * s], v_dim(128 * (u & 1), rank) + d);
                else held[k].load(p.cache, at[64 * rank + 8 * s], 128 * u + d);
            };
            bool ok = n > 0 && looked_up(0);
            if (ok) {
                fetch(0, 0);
                fetch(0, 1);
                read(0);
            }
            for (uint32_t f = 0; ok && f < 2 * n; ++f) {
                const bool v_form = v_form_of(f), then = f + 1 < 2 * n;
                const uint32_t row = 8 * s + Piece<kFormat>::row(lane);
                ok = !then || looked_up(tile_of(f + 1));
#pragma unroll
                for (uint32_t k = 0; k < 2; ++k) {
                    const uint32_t slot = (v_form ? kKUnits : 0) + team + 2 * k;
                    ok = ok && wait_warp(&bar->empty[slot], (tile_of(f) & 1) ^ 1, p.status);
                    if (!ok) break;
                    const uint32_t unit = ring + slot * kUnitBytes;
                    held[k].store(Piece<kFormat>::first(lane),
                                  [&](uint32_t ch) { return unit + (ch >> 3) * 8192 + swizzled(row, ch & 7); });
                    if (then) fetch(f + 1, k);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_first_cta(&bar->full[slot]);
                }
                if (ok && then) read(tile_of(f + 1));
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    // Neither CTA leaves while the other's MMAs or arrivals may reach it, for what lies there next would have them. The commits
    // arrive in both CTAs by themselves, the last of each issuing warp's on `drained` (the first CTA has waited for its
    // own). The threads' arrivals in the first CTA, the last ones of which nobody waits for, are performed before the
    // release.
    if (warp == 1) (void)wait_warp(&bar->drained, 0, p.status);
    cluster_arrive_release();
    cluster_wait_acquire();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ---- rows widened beforehand ---------------------------------------------------------------------

namespace {
constexpr int kWidenThreads = 256;
constexpr int kWidenUnroll = 2;                                             // rows of a thread, in flight together
constexpr int kWidenRows = kWidenThreads / (kDim / 16) * kWidenUnroll;      // of a block
}  // namespace

// The rows that a call attends to as bf16, each once: the prefix, then each entry's own, every run filled up with
// zeros to a whole tile. A row without a page is NaN, which zeroes the heads that see it. Bound by the
// bytes (1 KB written a row); an attention over many rows then reads them as it reads bf16 pages.
template <int kFormat>
__global__ void __launch_bounds__(kWidenThreads) prefix_widen_kernel(const __grid_constant__ PrefixParams p) {
    pdl_trigger();
    constexpr uint32_t kLanes = kDim / 16, kRows = kWidenThreads / kLanes;
    const uint32_t g = threadIdx.x % kLanes, shift = p.cache.page_shift;
    const uint32_t tile = blockIdx.x / (kTile / kWidenRows);
    const uint32_t in_tile = blockIdx.x % (kTile / kWidenRows) * kWidenRows + threadIdx.x / kLanes;
    // The run: its entry (the last one that begins at the tile or before it), first slot, first tile and end.
    uint32_t entry = 0, first = 0, begin = 0, end = p.prefix_len;
    if (tile >= p.wide_begin[0]) {
        for (uint32_t step = kPrefixRowsMax / 2; step > 0; step /= 2)
            if (entry + step < p.rows && p.wide_begin[entry + step] <= tile) entry += step;
        first = p.prefix_len;
        begin = p.wide_begin[entry];
        end = p.kv_len[entry];
    }
    const int32_t* table = p.cache.table + (size_t)entry * p.cache.table_stride;
    const uint32_t slot = first + (tile - begin) * kTile + in_tile;
    pdl_wait();
    Held16<kFormat> held[kWidenUnroll];
    int32_t id[kWidenUnroll];
#pragma unroll
    for (uint32_t k = 0; k < kWidenUnroll; ++k) {
        const uint32_t j = slot + kRows * k;
        id[k] = j < end ? table[j >> shift] : kNoRow;
        if (j < end && (uint32_t)id[k] >= p.cache.num_pages) id[k] = kBadRow;
    }
#pragma unroll
    for (uint32_t k = 0; k < kWidenUnroll; ++k)
        if (id[k] >= 0)
            load16<kDim, kFormat>(p.cache, (uint32_t)id[k], (slot + kRows * k) & ((1u << shift) - 1), g, held[k]);
#pragma unroll
    for (uint32_t k = 0; k < kWidenUnroll; ++k) {
        uint32_t w[8];
        if (id[k] >= 0) {
            widen16(held[k], w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = id[k] == kBadRow ? 0x7FC07FC0u : 0u;
        }
        st_global_v8(p.wide + ((size_t)tile * kTile + in_tile + kRows * k) * kDim + 16 * g, w);
    }
}

// ---- the join of a row's parts -------------------------------------------------------------------

namespace {
constexpr int kJoinThreads = 512;
constexpr int kJoinWays = kJoinThreads / kHeads;
constexpr uint32_t kJoinParts = kPrefixPairsMax + 2;  // a row's, at most: its segments lie on one line of runs
static_assert(kJoinParts <= 10 * kJoinWays, "parts that a thread holds");

// A row's parts in their order: those of its group's prefix, then its own.
struct RowParts {
    const float *shared, *own;  // of the first part of each
    uint32_t n0, count;
    static constexpr size_t kStep = 2 * kPrefixPartFloats;  // from one pair's to the next pair's
    static __host__ __device__ __forceinline__ uint32_t runs(const PrefixParams& p, uint32_t seg, uint32_t& first) {
        const uint32_t begin = p.begin[seg], end = p.begin[seg + 1];
        auto pair_of = [&](uint32_t t) { return (uint32_t)(((uint64_t)(t + 1) * p.pairs - 1) / p.line); };
        first = begin < end ? pair_of(begin + p.seg_cost) : 0;
        return begin < end ? pair_of(end - 1) - first + 1 : 0;
    }
    __host__ __device__ __forceinline__ RowParts(const PrefixParams& p, uint32_t r) {
        uint32_t a, b;
        n0 = runs(p, r / 2, a);
        count = n0 + runs(p, p.groups + r, b);
        shared = p.parts + (a + r / 2) * kStep + (r & 1) * kPrefixPartFloats;
        own = p.parts + (b + p.groups + r) * kStep;
    }
    __device__ __forceinline__ const float* at(uint32_t i) const { return i < n0 ? shared + i * kStep : own + (i - n0) * kStep; }
};
}  // namespace

// What a row's parts come to, once their maxima (with the sink's: `top`) and sums are known.
struct Joined {
    bool zero;
    float inv;
    __device__ __forceinline__ Joined(uint32_t stopped, float sink, float top, float den)  // a flagged part's sum is NaN
        : zero(stopped || !finite_f(sink) || !finite_f(top) || !finite_f(den) || !(den > 0.0f)), inv(1.0f / den) {}
    // Column `col` of the O layout, TMEM lane `lane`: four dims of a head.
    __device__ __forceinline__ void store(const PrefixParams& p, size_t at, uint32_t col, uint32_t lane, float4 acc) const {
        const uint32_t dim = 256 * (col >> 5) + 128 * (lane >> 6) + 4 * (col & 31);
        const float x[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
        __align__(8) __nv_bfloat16 y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = __float2bfloat16_rn(!zero && finite_f(x[k]) ? x[k] : 0.0f);
        *reinterpret_cast<uint2*>(p.out + at * kDim + dim) = *reinterpret_cast<const uint2*>(y);
    }
};
__device__ __forceinline__ float finite_sink2(float sink) {  // a finite sink stays finite
    return fminf(fmaxf(sink * kLog2e, -FLT_MAX), FLT_MAX);
}
__device__ __forceinline__ void add_scaled(float4& acc, const float4& o, float f) {
    acc.x = fmaf(o.x, f, acc.x);
    acc.y = fmaf(o.y, f, acc.y);
    acc.z = fmaf(o.z, f, acc.z);
    acc.w = fmaf(o.w, f, acc.w);
}

// Up to eight rows with many parts each, or two: a block joins `units` halves of a column of the O layout (4 dims of 64
// heads) of one row. Eight threads have every eighth part each, up to kHeld of them, whose maxima, sums and first half
// column are all in flight together.
template <int kHeld>
__global__ void __launch_bounds__(kJoinThreads, kHeld > 4 ? 1 : 2) prefix_join_split_kernel(const __grid_constant__ PrefixParams p,
                                                                                            uint32_t units) {
    __shared__ float m_s[kJoinWays][kHeads], l_s[kJoinWays][kHeads];
    __shared__ float4 acc_s[2][kJoinWays - 1][kHeads];
    pdl_trigger();
    const uint32_t r = blockIdx.x, way = threadIdx.x / kHeads, head = threadIdx.x % kHeads;
    const RowParts parts(p, r);
    const size_t at = (size_t)p.q_row[r] * kHeads + head;
    const uint32_t unit0 = blockIdx.y * units;
    float m[kHeld], f[kHeld];
    float4 sums[kHeld], o[kHeld];
    auto load = [&](uint32_t unit) {
        const size_t o_at = kPrefixHeadFloats + ((unit >> 1) * 128 + (unit & 1) * 64 + head) * 4;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (way + kJoinWays * k < parts.count)
                o[k] = __ldcg(reinterpret_cast<const float4*>(parts.at(way + kJoinWays * k) + o_at));
        }
    };
    pdl_wait();
    const float sink = p.sinks[(size_t)p.q_row[r] * p.sinks_row_stride + head];
    const uint32_t stopped = *p.status;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        m[k] = -INFINITY;
        sums[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (way + kJoinWays * k < parts.count) {
            const float* part = parts.at(way + kJoinWays * k);
            m[k] = __ldcg(part + head);
            sums[k] = __ldcg(reinterpret_cast<const float4*>(part + kHeads) + head);
        }
    }
    load(unit0);
    float top = m[0];
#pragma unroll
    for (int k = 1; k < kHeld; ++k) top = fmaxf(top, m[k]);
    m_s[way][head] = top;
    __syncthreads();
    const float sink2 = finite_sink2(sink);
    top = sink2;
#pragma unroll
    for (int k = 0; k < kJoinWays; ++k) top = fmaxf(top, m_s[k][head]);
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        f[k] = exp2f(m[k] - top);
        l = fmaf((sums[k].x + sums[k].y) + (sums[k].z + sums[k].w), f[k], l);
    }
    l_s[way][head] = l;
#pragma unroll 1
    for (uint32_t u = 0; u < units; ++u) {
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) add_scaled(acc, o[k], f[k]);
        if (way > 0) acc_s[u & 1][way - 1][head] = acc;
        if (u + 1 < units) load(unit0 + u + 1);
        __syncthreads();
        if (way == 0) {
            float den = exp2f(sink2 - top);
#pragma unroll
            for (int k = 0; k < kJoinWays; ++k) den += l_s[k][head];
            const Joined joined(stopped, sink, top, den);
            if (p.invalid && unit0 + u == 0) p.invalid[at] = joined.zero ? 1u : 0u;
#pragma unroll
            for (int k = 0; k < kJoinWays - 1; ++k) add_scaled(acc, acc_s[u & 1][k][head], 1.0f);
            joined.store(p, at, (unit0 + u) >> 1, ((unit0 + u) & 1) * 64 + head, acc);
        }
    }
}

// Many rows, or few parts each: a block joins `units` units of four columns of the O layout of one row, a thread to a lane
// of each. The factors exp(m_i - m) of the parts come first, for every head. Bound by the parts' bytes in L2. (With three
// parts ahead and two blocks on a multiprocessor 16 rows of 2000 took 17.6 us instead of 18.3, but 24 rows 19.7 instead of 19.2.)
constexpr uint32_t kJoinAhead = 2;
__global__ void __launch_bounds__(kJoinThreads, 3) prefix_join_kernel(const __grid_constant__ PrefixParams p, uint32_t units) {
    __shared__ float fac_s[kJoinParts][kHeads], sum_s[kJoinParts][kHeads];
    __shared__ float m_s[kJoinWays][kHeads], l_s[kJoinWays][kHeads];
    pdl_trigger();
    const uint32_t r = blockIdx.x, head = threadIdx.x & 63, head_way = threadIdx.x >> 6;
    const RowParts parts(p, r);
    const size_t at = (size_t)p.q_row[r] * kHeads + head;
    // Of the unit: column and lane, and its first two parts, whose loads need not wait for the factors.
    const uint32_t lane = threadIdx.x & 127, unit0 = blockIdx.y * units;
    auto o_at = [&](uint32_t unit) { return kPrefixHeadFloats + ((4 * unit + (threadIdx.x >> 7)) * 128 + lane) * 4; };
    float4 o[kJoinAhead];
    auto load = [&](uint32_t unit) {
#pragma unroll
        for (uint32_t i = 0; i < kJoinAhead; ++i) {
            o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < parts.count) o[i] = __ldcg(reinterpret_cast<const float4*>(parts.at(i) + o_at(unit)));
        }
    };
    pdl_wait();
    const float sink = p.sinks[(size_t)p.q_row[r] * p.sinks_row_stride + head];
    const uint32_t stopped = *p.status;
    load(unit0);
    float m = -INFINITY;
#pragma unroll 4
    for (uint32_t i = head_way; i < parts.count; i += kJoinWays) {
        const float* part = parts.at(i);
        const float x = __ldcg(part + head);
        const float4 sums = __ldcg(reinterpret_cast<const float4*>(part + kHeads) + head);
        fac_s[i][head] = x;
        sum_s[i][head] = (sums.x + sums.y) + (sums.z + sums.w);
        m = fmaxf(m, x);
    }
    m_s[head_way][head] = m;
    __syncthreads();
    const float sink2 = finite_sink2(sink);
    float top = sink2;
#pragma unroll
    for (int k = 0; k < kJoinWays; ++k) top = fmaxf(top, m_s[k][head]);
    float l = 0.0f;
#pragma unroll 4
    for (uint32_t i = head_way; i < parts.count; i += kJoinWays) {
        const float f = exp2f(fac_s[i][head] - top);
        fac_s[i][head] = f;
        l = fmaf(sum_s[i][head], f, l);
    }
    l_s[head_way][head] = l;
    __syncthreads();
    float den = exp2f(sink2 - top);
#pragma unroll
    for (int k = 0; k < kJoinWays; ++k) den += l_s[k][head];
    const Joined joined(stopped, sink, top, den);
    if (p.invalid && blockIdx.y == 0 && threadIdx.x < 64) p.invalid[at] = joined.zero ? 1u : 0u;
#pragma unroll 1
    for (uint32_t unit = unit0; unit < unit0 + units; ++unit) {
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (uint32_t i = 0; i < kJoinAhead; ++i)
            if (i < parts.count) add_scaled(acc, o[i], fac_s[i][head]);
        if (unit + 1 < unit0 + units) load(unit + 1);
#pragma unroll 2
        for (uint32_t i = kJoinAhead; i < parts.count; ++i)
            add_scaled(acc, __ldcg(reinterpret_cast<const float4*>(parts.at(i) + o_at(unit))), fac_s[i][head]);
        joined.store(p, at, 4 * unit + (threadIdx.x >> 7), lane, acc);
    }
}

template <int kFormat>
static cudaError_t launch(const PrefixParams& p, cudaStream_t stream, bool pdl) {
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t err = set_smem_limit_once(prefix_attn_kernel<kFormat>, kSmem<kFormat>, smem_set);
    if (err != cudaSuccess) return err;
    err = launch_kernel(prefix_attn_kernel<kFormat>, dim3(2 * p.pairs), dim3(kThreads<kFormat>), kSmem<kFormat>, stream, pdl, p);
    if (err != cudaSuccess) return err;
    uint32_t most = 0;  // parts of a row
    for (uint32_t r = 0; r < p.rows; ++r) most = std::max(most, RowParts(p, r).count);
    uint32_t units = 1;
    // (us, this kernel / the other: one row of 1216, 8 parts, 10.7 / 12.8; two rows of 500, 5 parts, 11.1 / 11.8; but three rows of 300,
    // 4 parts, 12.0 / 11.5; eight of 500, 5 parts, 15.2 / 12.8; 20 of 40000, 9 parts, 80 / 74.)
    const bool split = p.rows <= 2 || (p.rows <= 8 && most > 8);
    const uint32_t all = split ? 128 : 16, sms = 2 * kPrefixPairsMax, held = most <= 4 * kJoinWays ? 4 : 10;
    // Blocks that run together; of the other kernel about four for each multiprocessor (two were up to 8 us slower).
    while (units < all && p.rows * (all / units) > (!split ? 4 : held == 4 ? 2 : 1) * sms) units *= 2;
    const dim3 grid(p.rows, all / units), block(kJoinThreads);
    if (!split) return launch_kernel(prefix_join_kernel, grid, block, 0, stream, true, p, units);
    if (held == 4) return launch_kernel(prefix_join_split_kernel<4>, grid, block, 0, stream, true, p, units);
    return launch_kernel(prefix_join_split_kernel<10>, grid, block, 0, stream, true, p, units);
}

template <int kFormat>
static cudaError_t launch_packed(const PrefixParams& p, cudaStream_t stream, bool pdl) {
    if (!p.wide) return launch<kFormat>(p, stream, pdl);
    const cudaError_t err = launch_kernel(prefix_widen_kernel<kFormat>, dim3(p.wide_tiles * (kTile / kWidenRows)),
                                          dim3(kWidenThreads), 0, stream, pdl, p);
    return err == cudaSuccess ? launch<kWidened>(p, stream, true) : err;
}

cudaError_t launch_prefix_attn(const PrefixParams& p, int format, cudaStream_t stream, bool pdl) {
    if (format == DS_CACHE_INT4) return launch_packed<DS_CACHE_INT4>(p, stream, pdl);
    if (format == DS_CACHE_FP8) return launch_packed<DS_CACHE_FP8>(p, stream, pdl);
    return launch<DS_CACHE_BF16>(p, stream, pdl);
}

}  // namespace dsrows
