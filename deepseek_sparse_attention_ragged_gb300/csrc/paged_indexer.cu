// Indexer scores over a paged key cache, one query per entry:
//   s[j] = sum_h w[h] max(0, q_h . k_j)   (64 heads, 128 dims)
//
// The work is a stream of 128-key tiles; the CTAs are split over the entries in
// proportion to their tiles, and an entry's CTAs take every n-th of its tiles, so
// a CTA keeps one query for its whole life. Per tile one tcgen05.mma chain
// computes D[128 keys x 64 heads] = K_tile . Q^T (K = 128 as 8 steps of 16); the
// query lies in shared memory in the 128-byte-swizzled K-major layout, and the
// epilogue gives each thread one key (a TMEM lane) and its head sum, in the same
// order as the contiguous indexer, so a score depends on the key and the query alone.
//
// bf16 pages: bound by the key stream. TMA tiles of min(page_size, 128) rows go
// straight into the swizzled operand layout.
//
// 4-bit pages: 72 bytes a key instead of 256, so the tile's work in the SM counts
// more than the stream. Bulk copies bring whole pages (or a page's 128-row
// slices) into a ring; a thread reads one key's values and scales, widens them to
// bf16 (a shift, a mask and a packed FMA for two values, exact) and stores them
// into TMEM, where they are the A operand of the MMAs: the widened key never
// passes through shared memory, whose bandwidth (32 KB written and 32 KB read
// again a tile) would be the bound otherwise. 8 x 131072 keys take 20.8 us (22.8 us
// when nothing is in L2), of which the loads alone are 14.6 us (75.5 MB: 11.1 us at
// the measured copy bandwidth); it is 17.0 us without the head sums, and the MMAs
// hardly count (21.1 us with one of eight). No unit is full: 2.3 of 4 instructions
// issued a cycle, integer and FMA pipes at 41% and 39%, tensor pipe 31%, and the
// largest stall is one role waiting on another's results (TMEM loads, barriers); the
// first page comes only after the query's copy and a block barrier. Steps, in us: one
// issuing thread 34.7; the issuer's warp kept uniform 26.6
// (a divergent thread took 80 cycles an MMA, a uniform warp 25); four widening sets
// and two issuers 25.3; the mask and exponent of a value in one instruction 23.1;
// the polling loads 21.5; shared-space pointers and running indexes 20.8.
//
// Warp roles: 0 loads, the next kIssuers issue the MMAs (warp 1 owns TMEM), then
// kEpiSets epilogue sets of four warps and (4-bit pages) kWideSets widening sets.

#include "common.cuh"
#include "head_sum.cuh"
#include "int4.cuh"
#include "kernels.h"
#include "unscored.cuh"

namespace dsrows {

namespace {

constexpr int kTileKeys = 128;
constexpr int kHalfBytes = kTileKeys * 64 * 2;     // one 64-column SW128 block of a bf16 tile
constexpr int kBf16Tile = 2 * kHalfBytes;
constexpr int kQHalf = kIdxHeads * 64 * 2;         // one 64-column block of the query
constexpr int kInt4Row = kIdxDim / 2 + kIdxDim / int4::kGroup;  // 72 bytes
constexpr int kInt4Tile = kTileKeys * kInt4Row;
constexpr int kKeyWords = kIdxDim / 2;             // TMEM columns of a widened key (bf16 pairs)
constexpr int kIssuers = 2;   // warps that issue MMAs, each every second tile
constexpr int kEpiSets = 2;   // of four epilogue warps, each every second tile
constexpr int kWideSets = 4;  // of four widening warps, each every fourth tile
constexpr int kBufs = 4;      // accumulators, and widened tiles

template <bool kInt4>
struct Shape {
    static constexpr int kStages = kInt4 ? 12 : 4;
    static constexpr int kLap = 4;  // tiles whose loads are in the lanes' hands
    static constexpr int kStageBytes = kInt4 ? kInt4Tile : kBf16Tile;
    static constexpr int kThreads = 32 * (1 + kIssuers) + 128 * (kEpiSets + (kInt4 ? kWideSets : 0));
    static constexpr uint32_t kAccCols = kIdxHeads;
    static constexpr uint32_t kKeyCol = kBufs * kAccCols;  // widened keys: kBufs * kKeyWords columns
    static constexpr uint32_t kTmemCols = kInt4 ? 512 : 256;
    static constexpr size_t keys = 0;
    static constexpr size_t q = keys + (size_t)kStages * kStageBytes;
    static constexpr size_t w = q + 2 * (size_t)kQHalf;
    static constexpr size_t bars = w + 2 * kIdxHeads * 4;  // behind the weights and their halves
};
// The tiles of a buffer belong to one issuer and one set of each kind, and those of a stage to
// one lane of the loading warp, one issuer and one widening set: a wait for a parity is then
// never more than one phase ahead of its barrier.
static_assert(Shape<true>::kStages % Shape<true>::kLap == 0 && Shape<false>::kStages % Shape<false>::kLap == 0, "phases");
static_assert(kBufs % kIssuers == 0 && kBufs % kEpiSets == 0 && kBufs % kWideSets == 0, "phases");
static_assert(Shape<true>::kStages % kWideSets == 0 && Shape<true>::kStages % kIssuers == 0 &&
                  Shape<false>::kStages % kIssuers == 0,
              "phases");
static_assert(Shape<true>::kKeyCol + kBufs * kKeyWords <= 512, "TMEM columns");
static_assert(Shape<true>::q % 1024 == 0 && Shape<false>::q % 1024 == 0, "the swizzled query is 1-KiB aligned");

template <bool kInt4>
struct __align__(8) Bars {
    uint64_t full[Shape<kInt4>::kStages];
    uint64_t empty[Shape<kInt4>::kStages];
    uint64_t key_full[kBufs];   // a widened tile is in TMEM
    uint64_t key_empty[kBufs];  // its MMAs are done
    uint64_t acc_full[kBufs];
    uint64_t acc_empty[kBufs];
    uint32_t bad[Shape<kInt4>::kStages];  // sub-pages of the tile without a page
    uint32_t tmem_base;
};

template <bool kInt4>
constexpr size_t smem_bytes() {
    return Shape<kInt4>::bars + sizeof(Bars<kInt4>) + 1024;
}
static_assert(smem_bytes<true>() <= 227 * 1024 && smem_bytes<false>() <= 227 * 1024, "shared memory");

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_wait whose first tries read no timer, for waits of a few hundred cycles.
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, nullptr);
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T: A's rows are the TMEM lanes, two bf16 a column.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

}  // namespace

// A wait that gives up ends its role, so every later wait on its work gives up too, and the
// epilogue writes -inf for the keys that it has no sums for: the caller's buffer never keeps
// another call's scores.
template <bool kInt4>
__global__ void __launch_bounds__(Shape<kInt4>::kThreads, 1)
    paged_indexer_kernel(const __grid_constant__ PagedIndexerParams p) {
    using S = Shape<kInt4>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // Aligned by an offset, so that the pointers stay in the shared address space.
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* keys_s = smem + S::keys;
    uint8_t* q_s = smem + S::q;
    float* w_s = reinterpret_cast<float*>(smem + S::w);
    Bars<kInt4>* bar = reinterpret_cast<Bars<kInt4>*>(smem + S::bars);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);  // known to be uniform
    const int lane = threadIdx.x & 31;

    // This CTA's entry and tiles: first, first + step, ... below n_tiles.
    int e = 0;
    for (int i = 1; i < (int)p.rows; ++i)
        if (blockIdx.x >= p.cta_begin[i]) e = i;
    const uint32_t first = blockIdx.x - p.cta_begin[e];
    const uint32_t step = p.cta_begin[e + 1] - p.cta_begin[e];
    const uint32_t kv_len = p.kv_len[e];
    const uint32_t n_tiles = (kv_len + kTileKeys - 1) / kTileKeys;
    const uint32_t mine = first < n_tiles ? (n_tiles - first + step - 1) / step : 0;  // tiles of this CTA
    // A tile is `subs` pages of `sub_rows` keys, or a 128-row slice of one page.
    const uint32_t shift = p.cache.page_shift;
    const uint32_t sub_rows = shift < 7 ? 1u << shift : (uint32_t)kTileKeys;
    const uint32_t subs = kTileKeys / sub_rows;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], kInt4 ? 4 : 1);
            bar->bad[s] = 0;
        }
        for (int a = 0; a < kBufs; ++a) {
            mbar_init(&bar->key_full[a], 4);
            mbar_init(&bar->key_empty[a], 1);
            mbar_init(&bar->acc_full[a], 1);
            mbar_init(&bar->acc_empty[a], 4);
        }
        fence_barrier_init();
        if (!kInt4) tma_prefetch_map(&p.kmap);
    }
    if (warp == 1) {
        tmem_alloc(&bar->tmem_base, S::kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();  // the cache, the page table and the query may come from the previous kernel
    pdl_trigger();
    // The query, 16 bytes a thread, into the swizzled layout of two 64-column blocks.
    {
        const uint4* q = reinterpret_cast<const uint4*>(p.q + (size_t)p.q_row[e] * kIdxHeads * kIdxDim);
        for (int i = threadIdx.x; i < kIdxHeads * kIdxDim / 8; i += S::kThreads) {
            const int h = i >> 4, ch = i & 15;
            *reinterpret_cast<uint4*>(q_s + (ch >> 3) * kQHalf + h * 128 + (((ch & 7) ^ (h & 7)) << 4)) = q[i];
        }
        if (threadIdx.x < kIdxHeads) {
            const float w = p.w[(size_t)p.q_row[e] * kIdxHeads + threadIdx.x];
            w_s[threadIdx.x] = w;
            w_s[kIdxHeads + threadIdx.x] = 0.5f * w;
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem_base, 0);

    if (warp == 0) {
        // ---- loads: a lane owns one sub-page of every lap-th tile: it holds that page's id, issues
        // its copy as soon as the tile's stage is free, and goes on to its next tile, whose id it
        // fetched a lap before. The lanes poll together (one tile at a time, this loop took 680
        // cycles a tile and set the kernel's pace). A lap divides the stages, so the tile that
        // used a lane's stage last was the lane's own, and no wait is more than one phase ahead.
        constexpr uint32_t lap = S::kLap;  // tiles of up to 8 sub-pages each: 32 lanes
        const uint32_t my_tile = lane / subs, my_sub = lane % subs;
        const uint32_t group = ((1u << subs) - 1) << (my_tile * subs);  // the tile's lanes; subs <= 8
        const uint32_t sub_bytes = sub_rows * (kInt4 ? kInt4Row : kIdxDim * 2);
        const int32_t* table = p.cache.table + (size_t)e * p.cache.table_stride;
        const uint64_t policy = l2_policy_evict_first();
        const uint32_t tiles = my_tile < lap ? mine : 0;  // the other lanes have none
        auto first_key = [&](uint32_t it) { return (first + it * step) * kTileKeys + my_sub * sub_rows; };
        auto wants = [&](uint32_t it) { return it < tiles && first_key(it) < kv_len; };
        auto page_id = [&](uint32_t it) -> int32_t { return wants(it) ? table[first_key(it) >> shift] : -1; };
        uint32_t it = my_tile, s = my_tile, parity = 1;
        int32_t id = page_id(it), next = page_id(it + lap);
        uint64_t start = 0;
        bool ok = true;
        for (uint32_t tries = 0; ok && __any_sync(0xFFFFFFFFu, it < tiles); ++tries) {
            const bool want = wants(it);
            const bool have = want && id >= 0 && (uint32_t)id < p.cache.num_pages;
            const bool ready = it < tiles && mbar_try_wait(&bar->empty[s], parity);
            const uint32_t have_bits = __ballot_sync(0xFFFFFFFFu, have) & group;
            const uint32_t bad_bits = __ballot_sync(0xFFFFFFFFu, want && !have) & group;
            if ((__ballot_sync(0xFFFFFFFFu, ready) & group) == group) {
                if (my_sub == 0) {
                    bar->bad[s] = bad_bits >> (my_tile * subs);
                    mbar_arrive_expect_tx(&bar->full[s], __popc(have_bits) * sub_bytes);
                }
                if (have) {
                    uint8_t* dst = keys_s + s * S::kStageBytes + my_sub * (kInt4 ? sub_bytes : sub_rows * 128);
                    const uint32_t in_page = shift <= 7 ? 0u : first_key(it) & ((1u << shift) - 1);
                    if (!kInt4) {
                        const int y = (int)(((uint32_t)id << shift) + in_page);
                        tma_load_2d(dst, &p.kmap, &bar->full[s], 0, y, policy);
                        tma_load_2d(dst + kHalfBytes, &p.kmap, &bar->full[s], 64, y, policy);
                    } else {
                        const uint8_t* page = p.cache.pages + ((size_t)(uint32_t)id << shift) * p.cache.row_bytes;
                        if (shift <= 7) {
                            bulk_copy_g2s(dst, page, sub_bytes, &bar->full[s]);
                        } else {
                            // A 128-row slice of each plane, and its scales.
                            for (uint32_t c = 0; c < 5; ++c)
                                bulk_copy_g2s(dst + c * kTileKeys * 16,
                                              page + ((size_t)c << shift) * 16 + (size_t)in_page * (c < 4 ? 16 : 8),
                                              kTileKeys * (c < 4 ? 16 : 8), &bar->full[s]);
                        }
                    }
                }
                it += lap;
                if ((s += lap) >= S::kStages) s -= S::kStages, parity ^= 1;
                id = next;
                next = page_id(it + lap);
                start = 0;
            }
            if ((tries & 63) == 63) {  // bounded, as every wait
                const uint64_t now = global_timer_ns();
                if (start == 0) start = now;
                ok = !__any_sync(0xFFFFFFFFu, it < tiles && now - start > kWaitBudgetNs);
            }
            __syncwarp();
        }
        // Every load has landed before the CTA exits: each lane waits for its last tile of each stage.
        for (uint32_t k = 0; k < S::kStages / lap && it >= lap && my_tile < lap; ++k) {
            it -= lap;
            s = it % S::kStages;
            (void)mbar_wait(&bar->full[s], (it / S::kStages) & 1, nullptr);
        }
    } else if (warp <= kIssuers) {
        // ---- MMA issuer: the whole warp runs the loop, so that addresses and descriptors
        // stay in uniform registers, and one elected lane executes each MMA -----------------
        constexpr uint32_t idesc = idesc_bf16_f32(kTileKeys, kIdxHeads);
        const uint32_t b_base = smem_u32(q_s);
        uint32_t it = warp - 1, a = it, s = it, ph = 0, sph = 0;  // tile, buffer, stage, their phases
        for (; it < mine; it += kIssuers) {
            if (!wait_short(&bar->acc_empty[a], ph ^ 1)) break;
            if (kInt4) {
                if (!wait_short(&bar->key_full[a], ph)) break;
            } else {
                if (!wait_short(&bar->full[s], sph)) break;
            }
            tc_fence_after();
            const uint32_t d_tmem = tmem + a * S::kAccCols;
            const uint32_t a_base = smem_u32(keys_s + (size_t)s * S::kStageBytes);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kIdxDim / 16; ++kk) {
                    const uint32_t koff = (uint32_t)(kk & 3) * 32;  // 16 bf16 inside the 128-byte row
                    const uint64_t bdesc = smem_desc_sw128_kmajor(b_base + (kk >> 2) * kQHalf + koff);
                    if (kInt4)
                        umma_bf16_ta(d_tmem, tmem + S::kKeyCol + a * kKeyWords + kk * 8, bdesc, idesc, kk > 0);
                    else
                        umma_bf16(d_tmem, smem_desc_sw128_kmajor(a_base + (kk >> 2) * kHalfBytes + koff), bdesc, idesc,
                                  kk > 0);
                }
                umma_commit(kInt4 ? &bar->key_empty[a] : &bar->empty[s]);
                umma_commit(&bar->acc_full[a]);
            }
            __syncwarp();
            if ((a += kIssuers) >= kBufs) a -= kBufs, ph ^= 1;
            if ((s += kIssuers) >= S::kStages) s -= S::kStages, sph ^= 1;
        }
        // The MMAs issued are done before TMEM is freed.
        for (uint32_t k = it > kBufs ? it - kBufs : warp - 1; k < it; k += kIssuers)
            (void)mbar_wait(&bar->acc_full[k % kBufs], (k / kBufs) & 1, nullptr);
    } else if (warp < 1 + kIssuers + 4 * kEpiSets) {
        // ---- epilogue: one key per thread, alternate tiles per set -----------------------
        const int set = (warp - 1 - kIssuers) >> 2;
        const int quarter = warp & 3;
        const uint64_t keep = l2_policy_evict_last();  // the top-k reads the scores next
        float* out = p.scores + (size_t)e * p.score_stride;
        const bool halves = __all_sync(0xFFFFFFFFu, halvable(w_s[lane]) && halvable(w_s[lane + 32]));
        uint32_t a = set, ph = 0;  // buffer and its phase
        uint32_t j = (first + set * step) * kTileKeys + quarter * 32 + lane;
        for (uint32_t it = set; it < mine; it += kEpiSets, j += kEpiSets * step * kTileKeys) {
            // A bf16 key without a page is left out here (a widened one is NaN).
            bool have = true;
            if (!kInt4 && j < kv_len) {
                const int32_t id = p.cache.table[(size_t)e * p.cache.table_stride + (j >> shift)];
                have = id >= 0 && (uint32_t)id < p.cache.num_pages;
            }
            if (!wait_short(&bar->acc_full[a], ph)) {
                unscored(out, it, mine, kEpiSets, j, kEpiSets * step * kTileKeys, kv_len);
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + a * S::kAccCols;
            float sc = INFINITY;
            if (halves) sc = head_sum_tmem<true>(taddr, w_s + kIdxHeads);
            if (__any_sync(0xFFFFFFFFu, !finite_f(sc))) {
                const float again = head_sum_tmem<false>(taddr, w_s);
                sc = finite_f(sc) ? sc : again;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->acc_empty[a]);
            if (j < kv_len) st_global_hint(out + j, finite_f(sc) && have ? sc : -INFINITY, keep);
            if ((a += kEpiSets) >= kBufs) a -= kBufs, ph ^= 1;
        }
    } else {
        // ---- widening: one key per thread, alternate tiles per set ----------------------
        const int set = (warp - 1 - kIssuers - 4 * kEpiSets) >> 2;
        const int quarter = warp & 3;
        const uint32_t key = quarter * 32 + lane;
        const uint32_t sub = key / sub_rows, row = key % sub_rows;
        const uint8_t* row_s = keys_s + sub * sub_rows * kInt4Row + row * 16;
        const uint8_t* scale_s = keys_s + (sub * kInt4Row + kIdxDim / 2) * sub_rows + row * 8;
        const uint32_t tcol = tmem + ((uint32_t)(quarter * 32) << 16) + S::kKeyCol;
        uint32_t a = set, s = set, ph = 0, sph = 0;  // buffer, stage, their phases
        for (uint32_t it = set; it < mine; it += kWideSets) {
            const uint32_t taddr = tcol + a * kKeyWords;
            if (!wait_short(&bar->full[s], sph)) break;
            uint4 d[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                d[c] = *reinterpret_cast<const uint4*>(row_s + s * S::kStageBytes + c * sub_rows * 16);
            uint2 sc = *reinterpret_cast<const uint2*>(scale_s + s * S::kStageBytes);
            // A key without a page becomes NaN (its score -inf).
            if ((bar->bad[s] >> sub) & 1) sc.x = sc.y = 0x7F7F7F7Fu;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->empty[s]);
            if (!wait_short(&bar->key_empty[a], ph ^ 1)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                int4::Factors f0, f1;  // two groups a plane
                const uint32_t b = c < 2 ? sc.x : sc.y;
                if (c % 2 == 0) int4::factors2<0>(b, f0, f1);
                else int4::factors2<2>(b, f0, f1);
                uint32_t r[16];
                int4::widen(d[c].x, f0, r);
                int4::widen(d[c].y, f0, r + 4);
                int4::widen(d[c].z, f1, r + 8);
                int4::widen(d[c].w, f1, r + 12);
                tmem_st_x16(taddr + c * 16, r);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->key_full[a]);
            if ((a += kWideSets) >= kBufs) a -= kBufs, ph ^= 1;
            if ((s += kWideSets) >= S::kStages) s -= S::kStages, sph ^= 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmemCols);
    }
}

template <bool kInt4>
static cudaError_t launch(const PagedIndexerParams& p, int num_sms, cudaStream_t stream, bool pdl) {
    static std::atomic<uint64_t> smem_set{0};
    constexpr size_t bytes = smem_bytes<kInt4>();
    const cudaError_t err = set_smem_limit_once(paged_indexer_kernel<kInt4>, bytes, smem_set);
    if (err != cudaSuccess) return err;
    const uint32_t grid = p.total_tiles < (uint32_t)num_sms ? p.total_tiles : (uint32_t)num_sms;
    return launch_kernel(paged_indexer_kernel<kInt4>, dim3(grid), dim3(Shape<kInt4>::kThreads), bytes, stream, pdl, p);
}

cudaError_t launch_paged_indexer(const PagedIndexerParams& p, int format, int num_sms, cudaStream_t stream, bool pdl) {
    return format == DS_CACHE_INT4 ? launch<true>(p, num_sms, stream, pdl) : launch<false>(p, num_sms, stream, pdl);
}

}  // namespace dsrows
