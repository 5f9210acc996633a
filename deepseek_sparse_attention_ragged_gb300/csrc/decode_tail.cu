// Top-k selection and sink-softmax sparse attention of each row in one kernel
// (mlx-native deepseek_rows.metal: the top-k kernels
// deepseek_indexer_topk_*_rows_i32 followed by
// deepseek_sparse_attention_score_rows_bf16 / _reduce_rows_bf16; gather
// semantics of deepseek_sparse_attention_gather_rows_bf16).
//
// Per row e and head h over the selected slots t (index i_t):
//   l_t = scale * q_h . KV[i_t],  m = max(sink_h, max l_t),
//   den = exp(sink_h - m) + sum exp(l_t - m),  out_h = sum exp(l_t - m) KV[i_t] / den.
//
// One 8-CTA thread-block cluster per row, 512 threads per CTA. CTA r owns the
// 128-slot chunk c = r / 2 and the head half r % 2 (32 heads).
//   1. select (decode only): every CTA streams its slice of the row's scores
//      and stores the candidates at or above the level-0 threshold bin, in
//      index order, into the shared memory of every CTA of the cluster (an
//      all-gather); after one cluster barrier each CTA refines the exact
//      threshold over the gathered candidates and places the winners in index
//      order: slot t holds the winner with the t-th smallest index. Every CTA
//      computes the same selection, so no winner or slot crosses the cluster.
//      The caller's best-first index list comes from a ninth cluster, which
//      sorts each row's published winners best first (or, without attention,
//      from each CTA ranking its 64 slots). With indices given by the caller,
//      each CTA sorts them ascending (sentinels last) into the same slot order;
//   2. attend, on tcgen05 tensor cores with fp32 accumulators in TMEM: gather
//      the chunk's 128 KV rows into the 128-byte-swizzled K-major layout, then
//        logits  D[128 slots x 32 heads] = KV_chunk . Q_half^T   (K = 512,
//                as four accumulators over the K-steps k = a mod 4, added
//                as (D0 + D1) + (D2 + D3)),
//      the chunk softmax (max and sum over the 128 slots, per head), and
//        P G     D[128 features x 64] = KV_chunk^T . [P_hi; P_lo]^T  (K = 128 slots)
//      for the four 128-feature blocks, where the same KV buffer is the
//      MN-major operand and P enters as a bf16 hi + lo pair stacked along N
//      (acc = D[:, h] + D[:, 32 + h]);
//   3. combine: the chunk partials go to the workspace (the feature block a
//      CTA combines itself stays in its shared memory); after a cluster
//      barrier CTA r combines feature columns [128 c, 128 c + 128) of its 32
//      heads over the chunks in chunk order:
//        m = max(sink, m_c), den = exp(sink - m) + sum_c l_c exp(m_c - m),
//        out = sum_c acc_c exp(m_c - m) / den.
// Every reduction order depends on the row's width and its indices alone, and
// the stand-alone attention runs this kernel on the caller's indices in the
// same ascending order, so the decode's output is bitwise the attention of
// its own best-first index list.
//
// Over a paged cache (sparse_attn_paged_kernel) the rows come from the pages of a pool, in
// bf16 or widened from 8 or 4 bits as they are gathered, and the partials cross the cluster in
// distributed shared memory; every reduction is the same, so the output is bitwise that of
// the rows that the cache stands for.
//
// Fail-closed rules: a caller's index < -1 or >= kv_len flags the whole row; a
// non-finite logit (non-finite q or KV element, or overflow) flags its head;
// a non-finite sink or denominator flags the head; a flagged head is written
// as zeros, and any non-finite output element is written as zero.
//
// Bounded waits: a wait for the tensor cores that gives up (DS_STATUS_WAIT_TIMEOUT)
// stops the CTA's attention work (no further MMA, no TMEM read) and flags the
// row, so every head of it is written as zeros; the CTA still takes part in
// every cluster barrier, and before it frees TMEM it waits (bounded) once more
// for the MMAs it issued.

#include <cooperative_groups.h>

#include "attend.cuh"
#include "common.cuh"
#include "fp8.cuh"
#include "int4.cuh"
#include "kernels.h"
#include "select.cuh"

namespace dsrows {

namespace cg = cooperative_groups;
using attend::combine_shared;
using attend::combine_slice;
using attend::cp_async16;
using attend::cp_async4;
using attend::cp_async_commit;
using attend::cp_async_wait_all;
using namespace rowsel;

namespace {

constexpr int kChunkSlots = 128;                         // slots per chunk (UMMA M of the logits)
constexpr int kHalfHeads = kHeads / 2;                   // heads per CTA (UMMA N)
constexpr uint32_t kTmemCols = 512;                      // logits (4 x 32) + P G (4 x 64)
constexpr uint32_t kPvCol = 128;                         // first TMEM column of P G
// MMAs are issued by one thread in each of this many warps, into independent
// accumulators: one thread issues a tcgen05.mma in about 80 cycles, far longer
// than these N=32/64 MMAs take, so the issue rate sets the phase's time.
constexpr int kIssuers = 4;
constexpr int kGBlock = kChunkSlots * 128;               // one 64-column block of the KV rows: 16 KiB
constexpr int kQBlock = kHalfHeads * 128;                // one 64-column block of the query half: 4 KiB
constexpr int kPBlock = 2 * kHalfHeads * 128;            // 64 slots of [P_hi; P_lo] (64 rows): 8 KiB
static_assert(kCluster * kChunkSlots == 2 * kTopK, "4 chunks x 2 head halves per row");
static_assert(kThreads == 512, "16 warps");

struct TailLayout {
    static constexpr size_t g = 0;                                     // KV rows [128][512], K-major SW128
    static constexpr size_t q = g + 8 * (size_t)kGBlock;               // query half [32][512], K-major SW128
    static constexpr size_t pmat = q + 8 * (size_t)kQBlock;            // [P_hi; P_lo] [64][128 slots], K-major SW128
    static constexpr size_t idx = pmat + 2 * (size_t)kPBlock;          // i32 [128] this chunk's slots
    static constexpr size_t sel = idx + (size_t)kChunkSlots * 4;       // u64 [512] the row's winners
    static constexpr size_t red = sel + (size_t)kTopK * 8;             // [4 quarters][32 heads] max, sum, bad
    static constexpr size_t misc = red + 3 * 4 * (size_t)kHalfHeads * 4;
    static constexpr size_t sinks = misc + 64;                         // f32 [32] this head half's sinks
    static constexpr size_t ranks = sinks + (size_t)kHalfHeads * 4;    // u32 [64] best-first ranks
    static constexpr size_t total = ranks + 64 * 4;
    // Aliases used before the KV rows are gathered and P is written: the
    // gathered candidates ([8][kCandCap] u64) and the selection state.
    static constexpr size_t regions = g;
    static constexpr size_t gather = pmat;
};
static_assert(TailLayout::regions + (size_t)kCluster * kCandCap * 8 <= TailLayout::q, "candidates overlap the query");
static_assert(TailLayout::gather + sizeof(GatherSmem) <= TailLayout::idx, "selection state overlaps the slots");
static_assert(TailLayout::misc % 8 == 0, "alignment");
// Paged: the other chunks' partials of this CTA's feature block arrive in shared memory,
// two in the query's place (free once the logits are done) and one behind the rest.
struct PagedLayout : TailLayout {
    static constexpr size_t recv = (TailLayout::total + 15) & ~size_t(15);           // f32 [32][128]
    static constexpr size_t ml = recv + (size_t)kHalfHeads * 128 * 4;                // f32 [4 chunks][m[32], l[32]]
    static constexpr size_t bad_heads = ml + 4 * 2 * (size_t)kHalfHeads * 4;         // u32 [4 chunks]
    static constexpr size_t bad_rows = bad_heads + 4 * 4;                            // u32 [8 CTAs], then this one's
    static constexpr size_t total = bad_rows + (kCluster + 1) * 4;
};
constexpr size_t kPagedSmem = PagedLayout::total + 1024;
static_assert(kPagedSmem <= 227 * 1024, "shared memory");
static_assert(2 * (size_t)kHalfHeads * 128 * 4 <= 8 * (size_t)kQBlock, "two partials in the query's place");

constexpr size_t kTailSmem = TailLayout::total + 1024;  // + slack to align the swizzled buffers to 1 KiB
static_assert(kTailSmem <= 227 * 1024, "shared memory");

// Reduce 8 values over the warp by a butterfly that halves what a lane holds: the first
// three steps exchange 4, 2 and 1 values, so 9 shuffles do the work of 40, in the order
// of the plain butterfly (lane distances 16, 8, 4, 2, 1: the same bits). Returns the
// reduction of value reduced_of(lane).
__device__ __forceinline__ int reduced_of(int lane) { return (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1); }
template <class Op>
__device__ __forceinline__ float warp_reduce8(const float (&x)[8], int lane, Op op) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = x[k];
#pragma unroll
    for (int n = 4; n > 0; n >>= 1) {
        const bool upper = lane & (4 * n);
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float other = __shfl_xor_sync(0xFFFFFFFFu, upper ? v[k] : v[k + n], 4 * n);
            v[k] = op(upper ? v[k + n] : v[k], other);
        }
    }
    v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 2));
    return op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
}

// Byte offset of 16-byte chunk ch (0..63) of row r in a K-major SW128 buffer of
// 64-column blocks `block` bytes apart (rows of 128 B per block).
__device__ __forceinline__ uint32_t sw128_chunk(int r, int ch, int block) {
    return (uint32_t)((ch >> 3) * block + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// Where the KV rows lie: one contiguous bf16 cache per entry, or the pages of a
// pool in bf16 or 4 bits (the caller's indices only).
enum class Cache { kContiguous, kPagedBf16, kPagedInt4, kPagedFp8 };
constexpr int kInt4RowBytes = kDim / 2 + kDim / int4::kGroup;
constexpr int kFp8RowBytes = kDim + kDim / fp8::kBlock;  // of a page: its rows' values, then their exponents

constexpr uint32_t kNoIndex = 0xFFFFFFFFu;

// Sort 512 values in ascending order, one per thread, as bitonic512_desc does; `between`
// runs after the stages inside the warps (it hides a load's latency behind them).
template <class F>
__device__ __forceinline__ uint32_t bitonic512_asc(uint32_t x, uint32_t* buf, F&& between) {
    const uint32_t t = threadIdx.x;
    int b = 0;
#pragma unroll
    for (uint32_t k = 2; k <= 512; k <<= 1) {
        if (k == 64) between();
#pragma unroll
        for (uint32_t j = k >> 1; j > 0; j >>= 1) {
            uint32_t y;
            if (j >= 32) {
                buf[b * 512 + t] = x;
                __syncthreads();
                y = buf[b * 512 + (t ^ j)];
                b ^= 1;
            } else {
                y = __shfl_xor_sync(0xFFFFFFFFu, x, j);
            }
            const bool keep_min = ((t & j) == 0) == ((t & k) == 0);
            x = keep_min ? min(x, y) : max(x, y);
        }
    }
    return x;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

}  // namespace

// The paged instantiations differ from the contiguous one up to the gather and in the
// exchange of the partials: these go from CTA to CTA through distributed shared memory, and
// the flags with them, so nothing in the workspace has to be cleared before the call (it
// holds the status word only). One row of 37: 10.6 us; eight rows of 512: 12.1 us in 4 bits,
// 11.7 us in bf16 (ragged). With global partials behind the clear's launch 11.6 and 13.3 us;
// sending the blocks as bulk copies, counted on a barrier, was no faster (10.9 and 12.8 us).
// Bound by the chain of phases, in cycles of about 21,000: set-up and inputs 2,000, sort
// 2,500, gather and widening 3,800, logits 1,900, softmax 3,500, P G 2,300, exchange 3,800,
// combine 2,000. The bytes (1.2 MB of rows) take 0.2 us.
template <Cache kCache, class Params>
__device__ __forceinline__ void tail_body(const Params& p) {
    constexpr bool kPaged = kCache != Cache::kContiguous;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using T = TailLayout;
    uint8_t* g_s = smem + T::g;
    uint8_t* q_s = smem + T::q;
    uint8_t* p_s = smem + T::pmat;
    int* idx_s = reinterpret_cast<int*>(smem + T::idx);
    uint64_t* sel = reinterpret_cast<uint64_t*>(smem + T::sel);
    float* red_max = reinterpret_cast<float*>(smem + T::red);
    float* red_sum = red_max + 4 * kHalfHeads;
    uint32_t* red_bad = reinterpret_cast<uint32_t*>(red_sum + 4 * kHalfHeads);
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(smem + T::misc);
    uint64_t* mma_bar = reinterpret_cast<uint64_t*>(smem + T::misc + 8);
    float* sinks_s = reinterpret_cast<float*>(smem + T::sinks);
    uint64_t* regions = reinterpret_cast<uint64_t*>(smem + T::regions);
    float* own_s = reinterpret_cast<float*>(smem + T::g);  // after P·G: this CTA's combined feature block
    GatherSmem& gs = *reinterpret_cast<GatherSmem*>(smem + T::gather);

    // The stream's next kernel may launch while this one runs: it waits for this
    // grid to complete (griddepcontrol.wait) before it reads or writes anything
    // this kernel uses.
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t rank = cluster.block_rank();
    const int e = blockIdx.x / kCluster;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    // With attention: [8] "winners published" flags after the row flags, and the
    // winners' numbers after the published winners.
    auto pub_flag = [&](uint32_t r) { return p.flags + kRowsMax * kHeads + kRowsMax + r; };
    auto pub_n = [&](uint32_t r) { return reinterpret_cast<uint32_t*>(p.pub + (size_t)kRowsMax * kTopK) + r; };

    if (!kPaged && e >= (int)p.rows) {
        // ---- one more cluster ranks the rows' winners (decode with attention):
        // CTA r waits for row r to publish its winners in index order, sorts
        // them best first and writes the row's index list. No row waits for it.
        const uint32_t re = rank;
        if (re >= p.rows) return;
        pdl_wait();  // the publish flags were zeroed by earlier work
        uint32_t ok = 1;
        if (t == 0) {
            const uint64_t start = global_timer_ns();
            while (ld_acquire_gpu(pub_flag(re)) == 0)
                if (global_timer_ns() - start > kWaitBudgetNs) {
                    atomicOr(p.status, kStatusWaitTimeout);
                    ok = 0;
                    break;
                }
        }
        ok = __syncthreads_and(t != 0 || ok);
        __threadfence();
        const uint64_t x0 = ok ? __ldcg(p.pub + (size_t)re * kTopK + t) : 0ull;
        const uint32_t nsel = ok ? __ldcg(pub_n(re)) : 0u;
        const uint64_t x = bitonic512_desc(x0, reinterpret_cast<uint64_t*>(gs.h));
        if ((uint32_t)t < p.width[re])
            p.indices[p.index_offset[re] + t] = (uint32_t)t < nsel ? (int32_t)(~(uint32_t)x) + p.offset[re] : -1;
        return;
    }

    const uint32_t c = rank >> 1;          // chunk: slots [128 c, 128 c + 128)
    const int half = (int)(rank & 1);      // heads [32 half, 32 half + 32)
    const int head0 = half * kHalfHeads;
    const uint32_t L = p.kv_len[e];
    const uint32_t W = p.width[e];
    const uint32_t q_row = p.q_row[e];
    const uint32_t nchunks = (W + kChunkSlots - 1) / kChunkSlots;
    const bool has_chunk = c < nchunks;

    // ---- setup: counters, barrier, TMEM, and the query (an input of the call) --
    if (t == 0) {
        mbar_init(mma_bar, kIssuers);
        fence_barrier_init();
    }
    if (t < kChunkSlots) idx_s[t] = -1;  // slots past the last winner stay empty
    sel[t] = 0;
    if (warp == 0 && p.attend) {
        tmem_alloc(tmem_s, kTmemCols);
        tmem_relinquish();
    }
    // The query half (cp.async into the swizzled layout; waited for before the
    // logits) and the sinks (possibly in host memory; the combine uses them last).
    auto fetch_inputs = [&]() {
        const __nv_bfloat16* qh = p.q + ((size_t)q_row * kHeads + head0) * kDim;
        for (int k = t; k < kHalfHeads * (kDim / 8); k += kThreads) {
            const int h = k >> 6, ch = k & 63;
            cp_async16(q_s + sw128_chunk(h, ch, kQBlock), qh + (size_t)h * kDim + ch * 8);
        }
        if (t < kHalfHeads) cp_async4(sinks_s + t, p.sinks + (size_t)q_row * p.sinks_row_stride + head0 + t);
        cp_async_commit();
    };
    if (!kPaged && p.attend && !p.q_after_wait) fetch_inputs();
    uint32_t* bad_rows = reinterpret_cast<uint32_t*>(smem + PagedLayout::bad_rows);  // paged only
    if (kPaged && t == 0) bad_rows[kCluster] = 0;
    tc_fence_before();
    if (kPaged) __syncthreads();
    else cluster.sync();  // every CTA's counters are set before anyone stores into them
    tc_fence_after();
    const uint32_t tmem = p.attend ? *tmem_s : 0u;
    pdl_wait();  // scores and histogram (decode) or indices (caller) come from earlier work
    if (kPaged || (p.attend && p.q_after_wait)) fetch_inputs();
    // The first block starts first; a wait that gives up reports seconds later.
    if (kPaged && blockIdx.x == 0 && t == 0) *p.status = 0;

    const uint32_t first = c * kChunkSlots;
    uint32_t nsel = 0;
    bool bad_row = false;  // an index or a page id out of range (paged)
    if constexpr (kPaged) {
        // ---- the caller's indices in ascending order (-1 last), as below. A slot of this
        // chunk then holds its row's place in the pool instead of its index.
        const int32_t* table = p.cache.table + (size_t)e * p.cache.table_stride;
        const uint32_t shift = p.cache.page_shift;
        auto place_of = [&](uint32_t g) -> int32_t {
            const int32_t id = __ldcg(table + (g >> shift));
            if (id < 0 || (uint32_t)id >= p.cache.num_pages) return -1;
            return (int32_t)(((uint32_t)id << shift) + (g & ((1u << shift) - 1)));
        };
        uint32_t g = kNoIndex;
        if ((uint32_t)t < W) {
            const int i = __ldcg(p.given + p.index_offset[e] + t);
            if (i < -1 || i >= (int)L) bad_row = true;
            else if (i >= 0) g = (uint32_t)i;
        }
        // Every CTA sorts the whole list, and on the way fetches an eighth of the rows (and their
        // page ids) into L2.
        const uint32_t mine = g;
        g = bitonic512_asc(g, reinterpret_cast<uint32_t*>(gs.h), [&] {
            if (((uint32_t)t >> 6) == rank && mine != kNoIndex) {
                const int32_t at = place_of(mine);
                if (at >= 0 && kCache == Cache::kPagedFp8) {
                    const uint32_t page_rows = 1u << shift, in_page = (uint32_t)at & (page_rows - 1);
                    const uint8_t* page = p.cache.pages + (size_t)((uint32_t)at - in_page) * kFp8RowBytes;
                    for (uint32_t o = 0; o < (uint32_t)kDim; o += 128) prefetch_l2(page + (size_t)in_page * kDim + o);
                    prefetch_l2(page + (size_t)page_rows * kDim + in_page * (kDim / fp8::kBlock));
                } else if (at >= 0) {
                    for (uint32_t o = 0; o < p.cache.row_bytes; o += 128)
                        prefetch_l2(p.cache.pages + (size_t)at * p.cache.row_bytes + o);
                }
            }
        });
        if ((uint32_t)t - first < (uint32_t)kChunkSlots && g != kNoIndex) {
            const int32_t at = place_of(g);
            bad_row = bad_row || at < 0;
            idx_s[t - first] = max(at, 0);
        }
    } else if (p.given == nullptr) {
        // ---- select: gather the candidates, then every CTA selects the same winners
        const float* s = p.scores + (size_t)e * p.score_stride;
        const Gathered gat = select_collect_all(s, L, W, p.hist + (size_t)e * kHistBins, rank, gs, regions);
        cluster.sync();  // every CTA's candidates are in every CTA; no CTA touches
                         // another's shared memory after this barrier
        nsel = select_slots(gat, s, L, W, gs, regions, sel, idx_s, first, p.status);
    } else {
        // ---- the caller's indices, in ascending order (sentinels last): the
        // attention is a function of the index multiset. An index < -1 or
        // >= kv_len flags the row (it is written as zeros) and takes no slot.
        uint64_t v = 0;
        if ((uint32_t)t < W) {
            const int g = __ldcg(p.given + p.index_offset[e] + t);
            if (g < -1 || g >= (int)L) atomicOr(&p.flags[kRowsMax * kHeads + e], 1u);
            else if (g >= 0) v = (uint64_t)(~(uint32_t)g);
        }
        v = bitonic512_desc(v, reinterpret_cast<uint64_t*>(gs.h));
        if ((uint32_t)t - first < (uint32_t)kChunkSlots && v != 0) idx_s[t - first] = (int32_t)(~(uint32_t)v);
    }
    __syncthreads();  // this chunk's slots are in place (and the candidates consumed)
    // Publish the winners (index order) for the ranking cluster. The flag that
    // releases them is set after the gather is issued, by a thread that issues
    // no MMA, so the fence does not delay this CTA's attention.
    constexpr int kPublisher = kThreads - 32;
    const bool publish = p.ranker && rank == 0;
    if (publish) {
        p.pub[(size_t)e * kTopK + t] = sel[t];
        if (t == 0) *pub_n(e) = nsel;
    }
    // The gather of the chunk's KV rows starts now.
    const size_t part0_off = ((size_t)2 * p.chunk_begin[e] + (size_t)half * nchunks) * kPartFloats;
    if constexpr (kCache == Cache::kPagedBf16) {
        if (has_chunk)
            for (int k = t; k < kChunkSlots * (kDim / 8); k += kThreads) {
                const int r = k >> 6, ch = k & 63;
                const int i = idx_s[r];
                uint8_t* dst = g_s + sw128_chunk(r, ch, kGBlock);
                if (i >= 0) cp_async16(dst, p.cache.pages + (size_t)i * (2 * kDim) + ch * 16);
                else *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
            }
    } else if constexpr (kCache == Cache::kPagedInt4) {
        // A unit is 32 values (16 bytes) of a row and their two scales. A warp has eight rows,
        // and per step four neighbouring units of each: whole sectors are read, and eight
        // lanes store into eight rows, which the swizzle puts into different banks. All loads
        // are issued before the first unit is widened.
        constexpr int kUnits = kDim / 32 / 4;
        static_assert(8 * (kThreads / 32) == kChunkSlots, "eight rows a warp");
        if (has_chunk) {
            const int r = 8 * warp + (lane & 7);
            const int i = idx_s[r];
            const uint8_t* row = p.cache.pages + (size_t)max(i, 0) * kInt4RowBytes;
            uint4 d[kUnits];
            uint32_t sc[kUnits];
#pragma unroll
            for (int n = 0; n < kUnits; ++n) {
                const int u = 4 * n + (lane >> 3);
                // An empty slot is zeros: n + 8 = 8 in every value, s = 0.
                d[n] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
                sc[n] = 0;
                if (i >= 0) {
                    d[n] = __ldcg(reinterpret_cast<const uint4*>(row + 16 * u));
                    sc[n] = __ldcg(reinterpret_cast<const uint16_t*>(row + kDim / 2 + 2 * u));
                }
            }
#pragma unroll
            for (int n = 0; n < kUnits; ++n) {
                const int u = 4 * n + (lane >> 3);
                int4::Factors f[2];
                int4::factors2<0>(sc[n], f[0], f[1]);
                const uint32_t w[4] = {d[n].x, d[n].y, d[n].z, d[n].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[4];
                    int4::widen(w[c], f[c >> 1], o);
                    *reinterpret_cast<uint4*>(g_s + sw128_chunk(r, 4 * u + c, kGBlock)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    } else if constexpr (kCache == Cache::kPagedFp8) {
        // The same with units of 16 values (16 bytes), eight steps in two halves: half of a row's
        // loads are in flight while the other half is widened.
        constexpr int kUnits = kDim / 16 / 4, kHalf = kUnits / 2;
        if (has_chunk) {
            const int r = 8 * warp + (lane & 7);
            const int i = idx_s[r];
            const uint32_t shift = p.cache.page_shift, at = (uint32_t)max(i, 0), in_page = at & ((1u << shift) - 1);
            const uint8_t* page = p.cache.pages + (size_t)(at - in_page) * kFp8RowBytes;
            const uint8_t* row = page + (size_t)in_page * kDim;
            // An empty slot is zeros (its exponent any in range).
            uint32_t ex = 0x7F7F7F7Fu;
            if (i >= 0) ex = __ldcg(reinterpret_cast<const uint32_t*>(page + ((size_t)kDim << shift)) + in_page);
            uint4 d[2][kHalf];
            auto load = [&](int half) {
#pragma unroll
                for (int n = 0; n < kHalf; ++n) {
                    d[half][n] = make_uint4(0, 0, 0, 0);
                    const int u = 4 * (half * kHalf + n) + (lane >> 3);
                    if (i >= 0) d[half][n] = __ldcg(reinterpret_cast<const uint4*>(row + 16 * u));
                }
            };
            load(0);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half == 0) load(1);
#pragma unroll
                for (int n = 0; n < kHalf; ++n) {
                    const int u = 4 * (half * kHalf + n) + (lane >> 3);
                    const uint32_t f = fp8::factor(ex >> (8 * ((half * kHalf + n) / 2)) & 0xFFu);  // 8 units a block
                    uint32_t o[8];
                    fp8::widen(d[half][n].x, f, o);
                    fp8::widen(d[half][n].y, f, o + 2);
                    fp8::widen(d[half][n].z, f, o + 4);
                    fp8::widen(d[half][n].w, f, o + 6);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<uint4*>(g_s + sw128_chunk(r, 2 * u + c, kGBlock)) =
                            make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                }
            }
        }
    } else if (has_chunk && p.attend) {
        const __nv_bfloat16* kv = p.kv[e];
        for (int k = t; k < kChunkSlots * (kDim / 8); k += kThreads) {
            const int r = k >> 6, ch = k & 63;
            const int i = idx_s[r];
            uint8_t* dst = g_s + sw128_chunk(r, ch, kGBlock);
            if (i >= 0 && (uint32_t)i < L) cp_async16(dst, kv + (size_t)i * kDim + ch * 8);
            else *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
        }
    }
    // Best-first ranks (decode): CTA `rank` ranks the winners of slots
    // [64 rank, 64 rank + 64) against all of them (group t / 64 of 64 each) and
    // writes their indices at their ranks; slots past the last winner (up to
    // the width) are -1. With attention this runs inside the cluster barrier
    // that precedes the combine.
    auto rank_indices = [&]() {
        uint32_t* rk = reinterpret_cast<uint32_t*>(smem + T::ranks);
        if (t < 64) rk[t] = 0;
        __syncthreads();
        const uint32_t k = rank * 64 + (uint32_t)(t & 63);
        const uint64_t ck = sel[k];
        const uint64_t* grp = sel + (t >> 6) * 64;
        uint32_t nb = 0;
#pragma unroll 16
        for (int j = 0; j < 64; ++j) nb += grp[j] > ck ? 1u : 0u;
        atomicAdd(&rk[t & 63], nb);
        __syncthreads();
        if (t < 64) {
            int32_t* out = p.indices + p.index_offset[e];
            if (k < nsel) out[rk[t]] = (int32_t)(~(uint32_t)ck) + p.offset[e];
            else if (k < W) out[k] = -1;
        }
    };
    const bool want_ranks = p.given == nullptr && p.indices != nullptr && !p.ranker;
    if (!p.attend) {
        if (want_ranks) rank_indices();
        return;
    }

    // ---- attend: 128 slots x 32 heads on the tensor cores ------------------------
    cp_async_wait_all();      // the query and the KV rows
    fence_proxy_async_smem();  // ... are visible to the tensor cores
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (publish && t == kPublisher) {
        // Every thread's winner store precedes the barrier above.
        __threadfence();
        st_release_gpu(pub_flag(e), 1u);
    }

    // The issuing thread of warps 0..3. Paged: elected in a warp known to be uniform, which
    // keeps the descriptors in uniform registers (25 cycles an MMA instead of 80).
    const int uwarp = kPaged ? __shfl_sync(0xFFFFFFFFu, warp, 0) : warp;
    auto issuer = [&]() -> bool {
        if (kPaged) return uwarp < kIssuers && elect_one();
        return lane == 0 && warp < kIssuers;
    };

    // Paged: where chunk `from`'s partial of feature block `block` lies in the CTA that combines it.
    auto recv = [&](uint32_t from, int block) -> float* {
        const uint32_t i = from < (uint32_t)block ? from : from - 1;
        return reinterpret_cast<float*>(i < 2 ? smem + T::q + i * ((size_t)kHalfHeads * 128 * 4)
                                              : smem + PagedLayout::recv);
    };

    // `alive`: every tensor-core wait of this CTA has succeeded (uniform over the
    // CTA); `pending`: the mma_bar phase of MMAs whose completion was not seen.
    bool alive = true;
    int pending = -1;
    if (has_chunk) {
        const uint32_t g_addr = smem_u32(g_s), q_addr = smem_u32(q_s);
        if (issuer()) {
            // Accumulator a = warp takes the K-steps kk = 4 j + a.
            constexpr uint32_t idesc = idesc_bf16_f32(128, kHalfHeads);
            const uint32_t koff = (uint32_t)uwarp * 32;  // 16 bf16 = 32 B inside the 128-B row
#pragma unroll
            for (int j = 0; j < kDim / 64; ++j)
                umma_bf16(tmem + 32 * uwarp, smem_desc_sw128_kmajor(g_addr + j * kGBlock + koff),
                          smem_desc_sw128_kmajor(q_addr + j * kQBlock + koff), idesc, j > 0 ? 1u : 0u);
            umma_commit(mma_bar);
        }
    }
    if (has_chunk) {
        alive = __syncthreads_and(mbar_wait(mma_bar, 0, kPaged ? nullptr : p.status)) != 0;
        if (!alive) pending = 0;
    }
    if (kPaged) cluster_arrive_relaxed();  // this CTA's query has been read: others may write there
    if (has_chunk && alive) {
        tc_fence_after();
        // ---- chunk softmax: warp -> (32 slots, 8 heads), lane -> one slot ----------
        const int qt = warp & 3, hg = warp >> 2;
        const int slot = 32 * qt + lane;
        uint32_t v[4][8];
#pragma unroll
        for (int a = 0; a < 4; ++a) tmem_ld_x8(tmem + ((uint32_t)(32 * qt) << 16) + 32 * a + 8 * hg, v[a]);
        tmem_ld_wait();
        const bool live = idx_s[slot] >= 0;
        float l[8];
        uint32_t bad_bits = 0;  // head i of this warp's 8 has a non-finite live logit
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            l[i] = ((__uint_as_float(v[0][i]) + __uint_as_float(v[1][i])) +
                    (__uint_as_float(v[2][i]) + __uint_as_float(v[3][i]))) * p.scale;
            const bool ok = live && finite_f(l[i]);
            bad_bits |= (live && !ok) ? 1u << i : 0u;
            if (!ok) l[i] = -INFINITY;
        }
        bad_bits = __reduce_or_sync(0xFFFFFFFFu, bad_bits);
        const float m = warp_reduce8(l, lane, [](float a, float b) { return fmaxf(a, b); });
        const int red_at = qt * kHalfHeads + 8 * hg + reduced_of(lane);
        if ((lane & 3) == 0) {
            red_max[red_at] = m;
            red_bad[red_at] = (bad_bits >> reduced_of(lane)) & 1u;
        }
        __syncthreads();
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int h = 8 * hg + i;
            const float mh = fmaxf(fmaxf(red_max[h], red_max[kHalfHeads + h]),
                                   fmaxf(red_max[2 * kHalfHeads + h], red_max[3 * kHalfHeads + h]));
            const float w = l[i] == -INFINITY ? 0.0f : expf(l[i] - mh);
            const __nv_bfloat16 hi = __float2bfloat16_rn(w);
            const __nv_bfloat16 lo = __float2bfloat16_rn(w - __bfloat162float(hi));
            // 16 bits of each weight reach the product, twice the output's 8. Row h holds
            // P_hi, row 32 + h P_lo (same swizzle phase: 32 is a multiple of 8).
            const uint32_t off = (uint32_t)((slot >> 6) * kPBlock + h * 128 +
                                            ((((slot & 63) >> 3) ^ (h & 7)) << 4) + ((slot & 7) << 1));
            *reinterpret_cast<__nv_bfloat16*>(p_s + off) = hi;
            *reinterpret_cast<__nv_bfloat16*>(p_s + off + kHalfHeads * 128) = lo;
            sum[i] = w;
        }
        fence_proxy_async_smem();  // P is visible to the tensor cores
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        const uint32_t g_addr = smem_u32(g_s);
        if (issuer()) {
            // Feature block b = warp: features [128 b, 128 b + 128).
            constexpr uint32_t idesc = idesc_bf16_f32(128, 2 * kHalfHeads) | kIdescAMnMajor;
            const uint32_t p_addr = smem_u32(p_s);
            const int b = uwarp;
#pragma unroll
            for (int ks = 0; ks < kChunkSlots / 16; ++ks) {
                // A: features [128 b, 128 b + 128) x slots [16 ks, 16 ks + 16), MN-major.
                const uint64_t ad = smem_desc_sw128_mnmajor(g_addr + 2 * b * kGBlock + ks * 2048, kGBlock, 1024);
                const uint64_t bd = smem_desc_sw128_kmajor(p_addr + (ks >> 2) * kPBlock + (ks & 3) * 32);
                umma_bf16(tmem + kPvCol + 64 * b, ad, bd, idesc, ks != 0 ? 1u : 0u);
            }
            umma_commit(mma_bar);
        }
        // While the tensor cores run P G: the chunk's sum per head (a fixed warp
        // tree, then the four quarters) and the head flags.
        const float total = warp_reduce8(sum, lane, [](float a, float b) { return a + b; });
        if ((lane & 3) == 0) red_sum[red_at] = total;
        __syncthreads();
        float* part = p.part + part0_off + (size_t)c * kPartFloats;
        if (kPaged) cluster_wait_acquire();  // nor any other CTA's
        if (t < kHalfHeads) {
            const float mh = fmaxf(fmaxf(red_max[t], red_max[kHalfHeads + t]),
                                   fmaxf(red_max[2 * kHalfHeads + t], red_max[3 * kHalfHeads + t]));
            const float lh = (red_sum[t] + red_sum[kHalfHeads + t]) +
                             (red_sum[2 * kHalfHeads + t] + red_sum[3 * kHalfHeads + t]);
            const uint32_t bad = red_bad[t] | red_bad[kHalfHeads + t] | red_bad[2 * kHalfHeads + t] |
                                 red_bad[3 * kHalfHeads + t];
            if constexpr (kPaged) {
                const uint32_t bits = __ballot_sync(0xFFFFFFFFu, bad != 0);
                const uint32_t at = smem_u32(smem + PagedLayout::ml) + (2 * kHalfHeads * c + t) * 4;
#pragma unroll
                for (uint32_t b = 0; b < kCluster / 2; ++b) {
                    const uint32_t to = 2 * b + half;
                    st_cluster_u32(cluster_addr(at, to), __float_as_uint(mh));
                    st_cluster_u32(cluster_addr(at + kHalfHeads * 4, to), __float_as_uint(lh));
                    if (t == 0) st_cluster_u32(cluster_addr(smem_u32(smem + PagedLayout::bad_heads) + 4 * c, to), bits);
                }
            } else {
                part[t] = mh;
                part[kHalfHeads + t] = lh;
                if (bad) atomicOr(&p.flags[e * kHeads + head0 + t], 1u);
            }
        }
        alive = __syncthreads_and(mbar_wait(mma_bar, 1, kPaged ? nullptr : p.status)) != 0;
        if (!alive) pending = 1;
        if (alive) {
            tc_fence_after();
            // ---- partial: warp -> (32 features, 32 heads) of block warp / 4 -------------
            const int b = warp >> 2;
            uint32_t ahi[32], alo[32];
            const uint32_t tcol = tmem + ((uint32_t)(32 * qt) << 16) + kPvCol + 64 * b;
            tmem_ld_x32(tcol, ahi);
            tmem_ld_x32(tcol + kHalfHeads, alo);
            tmem_ld_wait();
            if (b == (int)c) {
                // Feature block c is combined by this CTA: it stays in shared
                // memory (the KV buffer is free once P·G is done), [32 heads][128].
                float* o = own_s + 32 * qt + lane;
#pragma unroll
                for (int h = 0; h < kHalfHeads; ++h) o[h * 128] = __uint_as_float(ahi[h]) + __uint_as_float(alo[h]);
            } else if constexpr (kPaged) {
                // Block b goes to the CTA that combines it.
                const uint32_t o = cluster_addr(smem_u32(recv(c, b)) + (32 * qt + lane) * 4, 2 * b + half);
#pragma unroll
                for (int h = 0; h < kHalfHeads; ++h)
                    st_cluster_u32(o + h * 512, __float_as_uint(__uint_as_float(ahi[h]) + __uint_as_float(alo[h])));
            } else {
                float* pacc = part + 2 * kHalfHeads + 128 * b + 32 * qt + lane;
#pragma unroll
                for (int h = 0; h < kHalfHeads; ++h)
                    pacc[(size_t)h * kDim] = __uint_as_float(ahi[h]) + __uint_as_float(alo[h]);
            }
        }
    }
    // A CTA whose tensor-core wait gave up has no valid partial: the whole row
    // is written as zeros.
    if constexpr (kPaged) {
        if (!has_chunk || pending == 0) cluster_wait_acquire();  // the wait that the others did above
        if (bad_row || (!alive && t == 0)) atomicOr(&bad_rows[kCluster], 1u);
        if (!alive && t == 0) atomicOr(p.status, kStatusWaitTimeout);
        __syncthreads();
        if (t < kCluster) st_cluster_u32(cluster_addr(smem_u32(bad_rows + rank), t), bad_rows[kCluster]);
    } else if (!alive && t == 0) {
        atomicOr(&p.flags[kRowsMax * kHeads + e], 1u);
    }
    tc_fence_before();
    // Every chunk's partial and flags are visible to the cluster after this
    // barrier; the best-first ranks are written while it completes.
    cluster_arrive_release();
    if (want_ranks) rank_indices();
    cluster_wait_acquire();
    tc_fence_after();

    // ---- combine: feature columns [128 c, 128 c + 128) of the 32 heads ----------
    __nv_bfloat16* out = p.out + ((size_t)q_row * kHeads + head0) * kDim;
    uint32_t* invalid = p.invalid && c == 0 ? p.invalid + (size_t)q_row * kHeads + head0 : nullptr;
    if constexpr (kPaged) {
        const uint32_t* bad = reinterpret_cast<const uint32_t*>(smem + PagedLayout::bad_heads);
        uint32_t bad_heads = 0, bad_any = 0;
        for (uint32_t i = 0; i < nchunks; ++i) bad_heads |= bad[i];
        for (int i = 0; i < kCluster; ++i) bad_any |= bad_rows[i];
        combine_shared<kHalfHeads, kThreads, 128>(
            [&](int i) { return i == (int)c ? own_s : recv((uint32_t)i, (int)c); },
            reinterpret_cast<const float*>(smem + PagedLayout::ml), (int)nchunks, (int)(128 * c),
            bad_any ? 0xFFFFFFFFu : bad_heads, sinks_s, out, invalid);
    } else {
        combine_slice<kHalfHeads, kThreads, 128>(p.part + part0_off, kPartFloats, (int)nchunks, (int)(128 * c), own_s,
                                                 has_chunk ? (int)c : -1, sinks_s, p.flags + kRowsMax * kHeads + e,
                                                 p.flags + e * kHeads + head0, out, invalid);
    }

    // MMAs whose completion was not seen may still write TMEM: wait once more
    // (bounded) before it is freed.
    if (pending >= 0) (void)mbar_wait(mma_bar, (uint32_t)pending, nullptr);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    decode_tail_kernel(const __grid_constant__ TailParams p) {
    tail_body<Cache::kContiguous>(p);
}

// The attention of the caller's indices over a paged cache.
template <Cache kCache>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    sparse_attn_paged_kernel(const __grid_constant__ PagedTailParams p) {
    tail_body<kCache>(p);
}

size_t decode_tail_smem_bytes() { return kTailSmem; }

cudaError_t launch_decode_tail(const TailParams& p, cudaStream_t stream, bool pdl) {
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t err = set_smem_limit_once(decode_tail_kernel, kTailSmem, smem_set);
    if (err != cudaSuccess) return err;
    if (p.rows == 0) return cudaSuccess;
    const uint32_t clusters = p.rows + (p.ranker ? 1u : 0u);
    return launch_kernel(decode_tail_kernel, dim3(clusters * kCluster), dim3(kThreads), kTailSmem, stream, pdl, p);
}

template <Cache kCache>
static cudaError_t launch_paged(const PagedTailParams& p, cudaStream_t stream, bool pdl) {
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t err = set_smem_limit_once(sparse_attn_paged_kernel<kCache>, kPagedSmem, smem_set);
    if (err != cudaSuccess) return err;
    return launch_kernel(sparse_attn_paged_kernel<kCache>, dim3(p.rows * kCluster), dim3(kThreads), kPagedSmem, stream,
                         pdl, p);
}

cudaError_t launch_sparse_attn_paged(const PagedTailParams& p, int format, cudaStream_t stream, bool pdl) {
    if (p.rows == 0) return cudaSuccess;
    if (format == DS_CACHE_INT4) return launch_paged<Cache::kPagedInt4>(p, stream, pdl);
    if (format == DS_CACHE_FP8) return launch_paged<Cache::kPagedFp8>(p, stream, pdl);
    return launch_paged<Cache::kPagedBf16>(p, stream, pdl);
}

}  // namespace dsrows
