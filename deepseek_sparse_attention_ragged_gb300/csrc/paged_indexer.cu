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
// as much as the stream. Bulk copies bring whole pages (or a page's 128-row
// slices) into a ring; a thread reads one key's values and scales, widens them to
// bf16 (one shift, one mask and one packed FMA for two values, exact) and stores
// them into TMEM, where they are the A operand of the MMAs: the widened key never
// passes through shared memory, whose bandwidth (32 KB written and 32 KB read
// again a tile) would be the bound otherwise. Two sets of four widening warps take
// alternate tiles, each with its own A and accumulator columns.
//
// Warp roles: 0 loads, 1 owns TMEM and issues the MMAs, 2..5 run the epilogue,
// 6..13 widen (4-bit pages).

#include "common.cuh"
#include "head_sum.cuh"
#include "int4.cuh"
#include "kernels.h"

namespace dsrows {

namespace {

constexpr int kTileKeys = 128;
constexpr int kHalfBytes = kTileKeys * 64 * 2;     // one 64-column SW128 block of a bf16 tile
constexpr int kBf16Tile = 2 * kHalfBytes;
constexpr int kQHalf = kIdxHeads * 64 * 2;         // one 64-column block of the query
constexpr int kInt4Row = kIdxDim / 2 + kIdxDim / int4::kGroup;  // 72 bytes
constexpr int kInt4Tile = kTileKeys * kInt4Row;
constexpr int kKeyWords = kIdxDim / 2;             // TMEM columns of a widened key (bf16 pairs)
constexpr int kEpiWarps = 4;

template <bool kInt4>
struct Shape {
    static constexpr int kStages = kInt4 ? 12 : 4;
    static constexpr int kStageBytes = kInt4 ? kInt4Tile : kBf16Tile;
    static constexpr int kSets = 2;                // of four widening warps
    static constexpr int kThreads = 64 + 32 * kEpiWarps + (kInt4 ? 32 * 4 * kSets : 0);
    static constexpr uint32_t kAccCols = kIdxHeads;
    static constexpr uint32_t kKeyCol = 2 * kAccCols;  // widened keys: kSets * kKeyWords columns
    static constexpr uint32_t kTmemCols = kInt4 ? 256 : 128;
    static constexpr size_t keys = 0;
    static constexpr size_t q = keys + (size_t)kStages * kStageBytes;
    static constexpr size_t bars = q + 2 * (size_t)kQHalf;
};
static_assert(Shape<true>::q % 1024 == 0 && Shape<false>::q % 1024 == 0, "the swizzled query is 1-KiB aligned");

template <bool kInt4>
struct __align__(8) Bars {
    uint64_t full[Shape<kInt4>::kStages];
    uint64_t empty[Shape<kInt4>::kStages];
    uint64_t key_full[2];   // a widened tile is in TMEM
    uint64_t key_empty[2];  // its MMAs are done
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint32_t bad[Shape<kInt4>::kStages];  // sub-pages of the tile without a page
    uint32_t tmem_base;
    uint32_t abort_flag;
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

template <bool kInt4>
__global__ void __launch_bounds__(Shape<kInt4>::kThreads, 1)
    paged_indexer_kernel(const __grid_constant__ PagedIndexerParams p) {
    using S = Shape<kInt4>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* keys_s = smem + S::keys;
    uint8_t* q_s = smem + S::q;
    Bars<kInt4>* bar = reinterpret_cast<Bars<kInt4>*>(smem + S::bars);
    const int warp = threadIdx.x >> 5;
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
        for (int a = 0; a < 2; ++a) {
            mbar_init(&bar->key_full[a], 4);
            mbar_init(&bar->key_empty[a], 1);
            mbar_init(&bar->acc_full[a], 1);
            mbar_init(&bar->acc_empty[a], kEpiWarps);
        }
        bar->abort_flag = 0;
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
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_base;

    if (warp == 0) {
        // ---- loads: a lane holds the page id of (tile, sub-page) of the next tiles ----
        const uint32_t batch = 32 / subs;
        const int32_t* table = p.cache.table + (size_t)e * p.cache.table_stride;
        auto page_ids = [&](uint32_t k0) -> int32_t {
            const uint32_t k = k0 + lane / subs;
            if (k >= mine) return -1;
            const uint32_t key = (first + k * step) * kTileKeys + (lane % subs) * sub_rows;
            return key < kv_len ? table[key >> shift] : -1;
        };
        const uint64_t policy = l2_policy_evict_first();
        int32_t next = page_ids(0), ids = 0;
        bool ok = true;
        uint32_t it = 0;
        for (; it < mine; ++it) {
            if (it % batch == 0) {
                ids = next;
                next = page_ids(it + batch);
            }
            const uint32_t s = it % S::kStages;
            ok = mbar_wait(&bar->empty[s], ((it / S::kStages) & 1) ^ 1, nullptr);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            const uint32_t key0 = (first + it * step) * kTileKeys;
            const uint32_t in_page = shift < 7 ? 0u : key0 & ((1u << shift) - 1);  // the slice's first row
            // Lane `sub` has sub-page `sub`'s id.
            const int32_t id = __shfl_sync(0xFFFFFFFFu, ids, (it % batch) * subs + lane % subs);
            const bool wanted = (uint32_t)lane < subs && key0 + lane * sub_rows < kv_len;
            const bool have = wanted && id >= 0 && (uint32_t)id < p.cache.num_pages;
            const uint32_t have_bits = __ballot_sync(0xFFFFFFFFu, have);
            const uint32_t bad_bits = __ballot_sync(0xFFFFFFFFu, wanted && !have);
            const uint32_t sub_bytes = sub_rows * (kInt4 ? kInt4Row : kIdxDim * 2);
            uint8_t* dst = keys_s + (size_t)s * S::kStageBytes;
            if (lane == 0) {
                bar->bad[s] = bad_bits;
                mbar_arrive_expect_tx(&bar->full[s], __popc(have_bits) * sub_bytes);
            }
            __syncwarp();
            if (kInt4) {
                if (shift < 7) {
                    if (have)
                        bulk_copy_g2s(dst + lane * sub_bytes, p.cache.pages + (size_t)(uint32_t)id * sub_bytes,
                                      sub_bytes, &bar->full[s]);
                } else if (have_bits && lane < 5) {
                    // The slice's rows of each plane, and their scales.
                    const uint8_t* page = p.cache.pages + ((size_t)(uint32_t)id << shift) * kInt4Row;
                    const uint32_t width = lane < 4 ? 16 : 8;
                    bulk_copy_g2s(dst + lane * kTileKeys * 16,
                                  page + ((size_t)lane << shift) * 16 + (size_t)in_page * width, kTileKeys * width,
                                  &bar->full[s]);
                }
            } else if (have) {
                const int y = (int)(((uint32_t)id << shift) + in_page);
                uint8_t* d = dst + lane * sub_rows * 128;
                tma_load_2d(d, &p.kmap, &bar->full[s], 0, y, policy);
                tma_load_2d(d + kHalfBytes, &p.kmap, &bar->full[s], 64, y, policy);
            }
        }
        if (!ok && lane == 0) atomicExch(&bar->abort_flag, 1u);
        // Every load this warp issued has landed before the CTA exits.
        for (uint32_t k = it > (uint32_t)S::kStages ? it - S::kStages : 0; k < it; ++k)
            (void)mbar_wait(&bar->full[k % S::kStages], (k / S::kStages) & 1, nullptr);
    } else if (warp == 1) {
        // ---- MMA issuer -------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(kTileKeys, kIdxHeads);
            const uint32_t b_base = smem_u32(q_s);
            uint32_t it = 0;
            for (; it < mine; ++it) {
                if (*(volatile uint32_t*)&bar->abort_flag) break;
                const uint32_t a = it & 1, ph = (it >> 1) & 1;
                const uint32_t s = it % S::kStages;
                if (kInt4) {
                    if (!mbar_wait(&bar->key_full[a], ph, nullptr)) break;
                } else {
                    if (!mbar_wait(&bar->full[s], (it / S::kStages) & 1, nullptr)) break;
                }
                if (!mbar_wait(&bar->acc_empty[a], ph ^ 1, nullptr)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem + a * S::kAccCols;
                const uint32_t a_base = smem_u32(keys_s + (size_t)s * S::kStageBytes);
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
            // The MMAs issued are done before TMEM is freed.
            for (uint32_t k = it > 2 ? it - 2 : 0; k < it; ++k)
                (void)mbar_wait(&bar->acc_full[k & 1], (k >> 1) & 1, nullptr);
        }
        __syncwarp();
    } else if (warp < 2 + kEpiWarps) {
        // ---- epilogue: one key per thread ---------------------------------------------
        const int quarter = warp & 3;
        const uint64_t keep = l2_policy_evict_last();  // the top-k reads the scores next
        float wr[kIdxHeads];
        const float4* w = reinterpret_cast<const float4*>(p.w + (size_t)p.q_row[e] * kIdxHeads);
        const bool w16 = (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
#pragma unroll
        for (int h = 0; h < kIdxHeads; h += 4) {
            if (w16) {
                *reinterpret_cast<float4*>(&wr[h]) = w[h / 4];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) wr[h + i] = reinterpret_cast<const float*>(w)[h + i];
            }
        }
        float* out = p.scores + (size_t)e * p.score_stride;
        for (uint32_t it = 0; it < mine; ++it) {
            const uint32_t a = it & 1, ph = (it >> 1) & 1;
            const uint32_t j = (first + it * step) * kTileKeys + quarter * 32 + lane;
            // A bf16 key without a page is left out here (a widened one is NaN).
            bool have = true;
            if (!kInt4 && j < kv_len) {
                const int32_t id = p.cache.table[(size_t)e * p.cache.table_stride + (j >> shift)];
                have = id >= 0 && (uint32_t)id < p.cache.num_pages;
            }
            if (!mbar_wait(&bar->acc_full[a], ph, nullptr)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + a * S::kAccCols;
            uint32_t v[64];
            tmem_ld_x32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
            tmem_ld_x32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->acc_empty[a]);
            const float sc = head_sum(v, wr, nullptr);
            if (j < kv_len) st_global_hint(out + j, finite_f(sc) && have ? sc : -INFINITY, keep);
        }
    } else {
        // ---- widening: one key per thread, alternate tiles per set ----------------------
        const int set = (warp - 2 - kEpiWarps) >> 2;
        const int quarter = warp & 3;
        const uint32_t key = quarter * 32 + lane;
        const uint32_t sub = key / sub_rows, row = key % sub_rows;
        const uint32_t base = sub * sub_rows * kInt4Row;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + S::kKeyCol + set * kKeyWords;
        for (uint32_t it = set; it < mine; it += S::kSets) {
            const uint32_t s = it % S::kStages;
            if (!mbar_wait(&bar->full[s], (it / S::kStages) & 1, nullptr)) break;
            const uint8_t* src = keys_s + (size_t)s * S::kStageBytes + base;
            uint4 d[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) d[c] = *reinterpret_cast<const uint4*>(src + (c * sub_rows + row) * 16);
            const uint2 sc = *reinterpret_cast<const uint2*>(src + sub_rows * (kIdxDim / 2) + row * 8);
            const bool bad = (bar->bad[s] >> sub) & 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->empty[s]);
            if (!mbar_wait(&bar->key_empty[set], ((it >> 1) & 1) ^ 1, nullptr)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // Two groups a plane. A key without a page becomes NaN (its score -inf).
                const float2 s2 = int4::scales2((c & 1 ? (c & 2 ? sc.y : sc.x) >> 16 : (c & 2 ? sc.y : sc.x)));
                const int4::Factors f0 = int4::factors(bad ? __int_as_float(0x7FC00000) : s2.x);
                const int4::Factors f1 = int4::factors(bad ? __int_as_float(0x7FC00000) : s2.y);
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
            if (lane == 0) mbar_arrive(&bar->key_full[set]);
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
