// Tokens and pages of the paged caches: the accepted path of a draft tree moved
// to the front of its tokens, requests that share or give back pages, and the
// pool of page counts behind them.  No call reads anything back to the host.
//
// All of it is copying and counting: a large move is bound by HBM (row bytes read
// and written once), the rest by latency: chains of dependent loads (lengths, lists,
// page table, counts, entries) of 0.6 to 1 us each.  Measured: 64 children of
// 8,229 tokens with a partial page in each of 99 caches 36 us (7.0 TB/s, the reads
// mostly from the L2: one source page a cache); 128 accepted paths of 16 tokens in 99
// caches 16.3 us (4.4 TB/s); one path in 5 caches 2.2 us; 256 rows giving back and
// taking about 100,000 of 131,072 pages 16.6 us; 8 rows of a pool of 1,024 6.2 us.
#include <algorithm>

#include "dsa_internal.cuh"
#include "indexer_common.cuh"
#include "mla_common.cuh"
#include "select_common.cuh"
#include "sm100.cuh"

namespace dsa {

int device_sm_count();

namespace pages {

constexpr int kMaxCaches = 128;                            // caches of one launch (passed by value)
constexpr int kMaxRows = 4096;                             // requests of one reserve or fork call
constexpr int kMaxAccept = 64;
constexpr int kCopyThreads = 256;
constexpr int kPoolThreads = 1024;
constexpr int kPerThread = kMaxRows / kPoolThreads;         // requests of a thread of the pool calls

struct CacheList {
    uint8_t* data[kMaxCaches];
    uint8_t kind[kMaxCaches];
};

// A page of a cache: 64 token rows of `row16` 16-byte pieces, row_bytes apart
// from the page's start, and for the index-K kinds one 4-byte scale word per
// token behind them.
struct Layout {
    int64_t page_bytes;
    int row16;
    int scale_at;                                          // 0: no scale words
};
__device__ __forceinline__ Layout layout_of(int kind) {
    if (kind == DSA_CACHE_KV) return Layout{DSA_KV_PAGE_BYTES, DSA_KV_TOKEN_BYTES / 16, 0};
    if (kind == DSA_CACHE_IDXK) return Layout{DSA_IDXK_PAGE_BYTES, 8, kPage * 128};
    return Layout{DSA_IDXK_MXFP4_PAGE_BYTES, 4, kPage * 64};
}

// ---------------------------------------------------------------- commit
// One block per (request, run of caches): the moves are worked out once, by a chain
// of dependent loads (lengths, list, page table), and then applied cache by cache.
// A warp moves one row at a time, 41 (KV) or 8 / 4 (index-K) pieces of 16 bytes; a
// round reads up to 144 rows of as many whole caches as they make into shared memory,
// all in flight at once, before the barrier and writes them after it, so a row may be
// another row's target.  128 requests x 99 caches: 45 us with a block per cache, most
// of it the chain; 20.5 with the rows in registers, which allow 64 a round; 16.6 so.
constexpr int kCommitWarps = kCopyThreads / 32;
constexpr int kCommitRows = 144;                           // of a round: 94 KB, two blocks a SM
constexpr int kCommitSmem = kCommitRows * DSA_KV_TOKEN_BYTES;
static_assert(DSA_KV_TOKEN_BYTES >= DSA_INDEX_HEAD_DIM + 4, "an index key and its scale word take a row's place");
// Blocks of a launch, per SM: three times what is resident.  More caches a block take
// more rounds one after another, fewer repeat the chain: 24.3 / 18.8 / 16.6 / 17.8 /
// 18.2 us with 2 / 4 / 6 / 8 / 12.
constexpr int kCommitBlocks = 6;

__global__ void __launch_bounds__(kCopyThreads)
commit_kernel(const int32_t* __restrict__ accept, int width, BatchDev b, CacheList cl, int n_caches, int per_block,
              int32_t* __restrict__ new_len, int32_t* __restrict__ st) {
    __shared__ int32_t s_src[kMaxAccept], s_dst[kMaxAccept];
    __shared__ int32_t s_n;
    pdl_wait();
    pdl_trigger();
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool speaks = blockIdx.y == 0;                   // one block per request records and writes the length
    if (warp == 0) {
        const int qs = b.q_start[r], qe = b.q_start[r + 1], L = b.seq_len[r];
        int a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) a[h] = h * 32 + lane < width ? accept[(int64_t)r * width + h * 32 + lane] : -1;
        const int qn = qe - qs, P = L - qn;
        int kept = 0;
        bool open = true;                                  // the list has not ended yet
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const unsigned end = __ballot_sync(0xffffffffu, a[h] < 0 || a[h] >= qn);
            const int n = !open ? 0 : end ? __ffs(end) - 1 : 32;
            if (open && end && speaks) {
                const int bad = __shfl_sync(0xffffffffu, a[h], __ffs(end) - 1);
                if (lane == 0 && bad >= 0) record_error(st, DSA_DEVERR_INDEX_RANGE, bad);
            }
            kept += n;
            open = open && !end;
        }
        if (P < 0) {                                       // more new tokens than the request holds
            if (lane == 0 && speaks) record_error(st, DSA_DEVERR_INDEX_RANGE, P);
            kept = 0;
        }
        if (speaks && lane == 0 && new_len) new_len[r] = P < 0 ? L : P + kept;
        int n_moves = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = h * 32 + lane;
            int src = -1, dst = -1;
            if (k < kept && a[h] != k) {                   // a token already in place stays
                const int js = P + a[h], jd = P + k;
                if (js / kPage >= b.max_pages || jd / kPage >= b.max_pages) {
                    if (speaks) record_error(st, DSA_DEVERR_INDEX_RANGE, js);
                } else {
                    const int64_t ps = b.page_table[(int64_t)r * b.max_pages + js / kPage];
                    const int64_t pd = b.page_table[(int64_t)r * b.max_pages + jd / kPage];
                    if (ps < 0 || ps >= b.num_pages || pd < 0 || pd >= b.num_pages) {
                        if (speaks) record_error(st, DSA_DEVERR_PAGE_RANGE, ps < 0 || ps >= b.num_pages ? ps : pd);
                    } else {
                        src = (int32_t)(ps * kPage + js % kPage);
                        dst = (int32_t)(pd * kPage + jd % kPage);
                    }
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, src >= 0);
            const int at = n_moves + __popc(m & ((1u << lane) - 1));
            if (src >= 0) {
                s_src[at] = src;
                s_dst[at] = dst;
            }
            n_moves += __popc(m);
        }
        if (lane == 0) s_n = n_moves;
    }
    __syncthreads();
    const int n = s_n;
    if (n == 0) return;
    extern __shared__ __align__(16) uint8_t smem[];
    const int c_end = min(n_caches, (int)(blockIdx.y + 1) * per_block);
    const int round = kCommitRows / n;                     // caches of a round, at least two
    for (int c0 = blockIdx.y * per_block; c0 < c_end; c0 += round) {
        const int rows = min(round, c_end - c0) * n;
        for (int x = warp; x < rows; x += kCommitWarps) {
            const int c = c0 + x / n, s = s_src[x % n];
            const Layout lo = layout_of(cl.kind[c]);
            const uint8_t* page = cl.data[c] + (int64_t)(s / kPage) * lo.page_bytes;
            const uint4* from = reinterpret_cast<const uint4*>(page) + (s % kPage) * lo.row16;
            const uint32_t to = sm100::smem_addr(smem) + x * DSA_KV_TOKEN_BYTES;
            if (lane < lo.row16) mlc::cp_async_16(to + lane * 16, from + lane);
            if (lane + 32 < lo.row16) mlc::cp_async_16(to + (lane + 32) * 16, from + lane + 32);
            if (lo.scale_at && lane == 0) mlc::cp_async_4(to + lo.row16 * 16, page + lo.scale_at + (s % kPage) * 4);
        }
        mlc::cp_async_wait_all();                          // a lane stores what it has read
        __syncthreads();                                   // every source row of these caches has been read
        for (int x = warp; x < rows; x += kCommitWarps) {
            const int c = c0 + x / n, d = s_dst[x % n];
            const Layout lo = layout_of(cl.kind[c]);
            uint8_t* page = cl.data[c] + (int64_t)(d / kPage) * lo.page_bytes;
            uint4* to = reinterpret_cast<uint4*>(page) + (d % kPage) * lo.row16;
            const uint4* from = reinterpret_cast<const uint4*>(smem + x * DSA_KV_TOKEN_BYTES);
            if (lane < lo.row16) to[lane] = from[lane];
            if (lane + 32 < lo.row16) to[lane + 32] = from[lane + 32];
            if (lo.scale_at && lane == 0)
                *reinterpret_cast<uint32_t*>(page + lo.scale_at + (d % kPage) * 4) = *reinterpret_cast<const uint32_t*>(from + lo.row16);
        }
    }
}

// ---------------------------------------------------------------- release
// One block per (request, chunk of its table row).  An entry is exchanged for
// -1, so a row named twice gives a page back once; the counts' sums do not
// depend on the order of the atomics.
constexpr int kReleaseThreads = 256;

__global__ void __launch_bounds__(kReleaseThreads)
release_kernel(int32_t* __restrict__ ref, int64_t num_pages, int32_t* __restrict__ table, int rows, int max_pages,
               const int32_t* __restrict__ row, const int32_t* __restrict__ first, const int32_t* __restrict__ end,
               int32_t* __restrict__ st) {
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x;
    const int r = row[i];
    if (r < 0 || r >= rows) {
        if (threadIdx.x == 0 && blockIdx.y == 0) record_error(st, DSA_DEVERR_INDEX_RANGE, r);
        return;
    }
    const int lo = max(first[i], 0), hi = min(end[i], max_pages);
    int32_t* t = table + (int64_t)r * max_pages;
    for (int64_t k = (int64_t)lo + blockIdx.y * kReleaseThreads + threadIdx.x; k < hi; k += gridDim.y * kReleaseThreads) {
        const int32_t pg = atomicExch(t + k, -1);
        if (pg < 0) continue;
        if (pg >= num_pages) {
            record_error(st, DSA_DEVERR_PAGE_RANGE, pg);
        } else if (atomicSub(ref + pg, 1) <= 0) {
            atomicAdd(ref + pg, 1);
            record_error(st, DSA_DEVERR_PAGE_COUNT, pg);
        }
    }
}

// ---------------------------------------------------------------- taking pages
// One cluster of up to eight blocks walks the counts.  Each round covers 16 counts
// per thread and block, a block's next round in flight while the blocks tell one
// another how many free pages they hold; the ranks follow from a scan inside the
// block.  A block lists its free pages, so that its threads take them side by side:
// the threads that found them would each take up to 16 one after the other, a round
// trip each.  (About 100,000 pages from 131,072 counts with the release before it:
// 131 us with one block, 27 with eight, 21 with the list, 17 with a warp's entries next
// to one another, whose owner is then mostly known.)
constexpr int kPoolBlocks = 8;                             // the largest cluster every launch may have
constexpr int kStep = 16 * kPoolThreads;                   // counts of a block's round

constexpr int kSlots = 4 * kMaxRows;                       // of the table of rows, at most half of them in use

// Dynamic shared memory of the calls that take pages.
struct PoolShared {
    int32_t a[kMaxRows];
    int32_t cnt[kMaxRows + 4];                             // entries before each request
    union {
        uint32_t slot[kSlots];                             // rows mentioned (struct Mentions), before the walk
        uint16_t free_at[kStep];                           // the block's free pages, from the round's first one
    };
    int scratch[32];
    int total[2][kPoolBlocks];                             // free pages of each block's round
    int next;                                              // fill_rest: the first entry that got no page of the round's
};

struct Counts {
    int4 v[4];
};
__device__ __forceinline__ void load_counts(Counts& c, const int32_t* ref, int64_t num_pages, int64_t at) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (at + 4 * u + 4 <= num_pages) {
            c.v[u] = *reinterpret_cast<const int4*>(ref + at + 4 * u);
        } else {                                           // the tail: pages that are not there count as held
            c.v[u].x = at + 4 * u < num_pages ? ref[at + 4 * u] : 1;
            c.v[u].y = at + 4 * u + 1 < num_pages ? ref[at + 4 * u + 1] : 1;
            c.v[u].z = at + 4 * u + 2 < num_pages ? ref[at + 4 * u + 2] : 1;
            c.v[u].w = 1;
        }
    }
}
// Where this thread's counts of the block's first round begin.
__device__ __forceinline__ int64_t first_count() { return (int64_t)blockIdx.x * kStep + (int64_t)threadIdx.x * 16; }

// Where a block's e-th free page is listed.  Threads that found 16 pages write 32 bytes
// apart; turned by the groups of 64, they hit 32 banks.
__device__ __forceinline__ int listed(int e) { return e ^ (e >> 6 & 7) << 1; }

// The first `want` free pages in ascending order go to entry(0, i), entry(1, i), .. (i: the
// caller's hint, 0 at first); an entry that holds a page keeps it if `keep`.  Returns how many pages there were (at most
// want), the same in every block.  c: the counts from first_count() on, loaded by the
// caller.
template <typename Entry>
__device__ __forceinline__ int walk_free(Counts c, int32_t* ref, int64_t num_pages, int want, bool keep, PoolShared& sh,
                                         Entry entry) {
    static_assert(kStep <= 1 << 16, "pages of a round as 16-bit numbers");
    const int tid = threadIdx.x, blocks = gridDim.x;
    const int64_t round = (int64_t)blocks * kStep;
    int found = 0, turn = 0;
    int64_t at = first_count();
    for (int64_t base = 0; base < num_pages && found < want; base += round, at += round, turn ^= 1) {
        Counts next;
        if (base + round < num_pages) load_counts(next, ref, num_pages, at + round);
        int n = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) n += (c.v[u].x == 0) + (c.v[u].y == 0) + (c.v[u].z == 0) + (c.v[u].w == 0);
        int mine;                                          // free pages of this block's round
        int place = sel::excl_scan<kPoolThreads, 0>(n, tid, sh.scratch, &mine);
        if (blocks > 1 && tid < blocks)
            sm100::st_cluster_u32(sm100::mapa_shared(sm100::smem_addr(&sh.total[turn][blockIdx.x]), tid), (uint32_t)mine);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int x[4] = {c.v[u].x, c.v[u].y, c.v[u].z, c.v[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (x[e] == 0) sh.free_at[listed(place++)] = (uint16_t)(tid * 16 + 4 * u + e);
        }
        int rank0 = found;                                 // of the block's first free page
        if (blocks > 1) {
            sm100::cluster_sync();                         // a block is never two rounds ahead: two sets of slots do
            for (int b = 0; b < blocks; ++b) {
                if (b < (int)blockIdx.x) rank0 += sh.total[turn][b];
                found += sh.total[turn][b];
            }
        } else {
            __syncthreads();
            found += mine;
        }
        const int64_t page0 = base + (int64_t)blockIdx.x * kStep;
        const int takes = max(0, min(mine, want - rank0));
        // a warp takes consecutive pages for consecutive entries, four round trips at a time
        const int chunk = (takes + kPoolThreads - 1) / kPoolThreads * 32, end = min(takes, ((tid >> 5) + 1) * chunk);
        int owner = 0;
        for (int e0 = (tid >> 5) * chunk + (tid & 31); e0 < end; e0 += 4 * 32) {
            int32_t* t[4];
            bool ours[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                t[u] = e0 + u * 32 < end ? entry(rank0 + e0 + u * 32, owner) : nullptr;
                ours[u] = t[u] != nullptr && (!keep || *t[u] < 0);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (ours[u]) {
                    const int64_t page = page0 + sh.free_at[listed(e0 + u * 32)];
                    *t[u] = (int32_t)page;
                    ref[page] = 1;
                }
        }
        __syncthreads();                                   // the list may be written again
        c = next;
    }
    return min(found, want);
}

// Entries [e, total) that lack a page take, in order, the free pages that are left: those
// that entries with a page of their own passed over.  By one block, behind a walk of all
// that ended without a page for each entry.  Returns the first entry that was not looked at
// with a page in hand.
template <typename Entry>
__device__ __noinline__ int fill_rest(int32_t* ref, int64_t num_pages, int e, int total, PoolShared& sh, Entry entry) {
    const int tid = threadIdx.x;
    for (int64_t base = 0; base < num_pages && e < total; base += kStep) {
        uint32_t free = 0;                                 // of this thread's 16 counts
        for (int u = 0; u < 16; ++u) {
            const int64_t page = base + tid * 16 + u;
            if (page < num_pages && __ldcg(ref + page) == 0) free |= 1u << u;
        }
        int mine;
        int place = sel::excl_scan<kPoolThreads, 0>(__popc(free), tid, sh.scratch, &mine);
        for (int u = 0; u < 16; ++u)
            if (free >> u & 1u) sh.free_at[place++] = (uint16_t)(tid * 16 + u);
        __syncthreads();
        for (int used = 0; used < mine && e < total;) {
            int owner = 0;
            int32_t* t = tid < total - e ? entry(e + tid, owner) : nullptr;   // there may be nearly 2^31 entries
            const bool lacks = t != nullptr && __ldcg(t) < 0;
            int n;
            const int rank = sel::excl_scan<kPoolThreads, 0>(lacks, tid, sh.scratch, &n);
            if (lacks && rank < mine - used) {
                const int64_t page = base + sh.free_at[used + rank];
                *t = (int32_t)page;
                ref[page] = 1;
            }
            if (lacks && rank == mine - used) sh.next = e + tid;
            __syncthreads();
            e = n > mine - used ? sh.next : e + min(total - e, kPoolThreads);
            used += min(n, mine - used);
            __syncthreads();                               // sh.next may be written again
        }
        __syncthreads();                                   // the list may be written again
    }
    return e;
}

// The rows that a call names, each with its least mention: an open hash table.
// row_of(m) is the row of mention m.
template <typename RowOf>
struct Mentions {
    uint32_t* slot;                                        // [kSlots]: mention + 1, 0 where free
    RowOf row_of;
    __device__ __forceinline__ uint32_t first_slot(int row) const { return (uint32_t)row * 0x9e3779b1u >> 18; }
    __device__ __forceinline__ void add(int m) {
        static_assert(kSlots == 1 << 14, "hash bits");
        const int row = row_of(m);
        for (uint32_t at = first_slot(row);; at = (at + 1) % kSlots) {
            const uint32_t was = atomicCAS(slot + at, 0u, m + 1u);
            if (was == 0) return;
            if (row_of(was - 1) == row) {
                atomicMin(slot + at, m + 1u);
                return;
            }
        }
    }
    __device__ __forceinline__ int least(int row) const {  // of a row that has been added
        uint32_t at = first_slot(row);
        while (row_of(slot[at] - 1) != row) at = (at + 1) % kSlots;
        return (int)slot[at] - 1;
    }
};
template <typename RowOf>
__device__ __forceinline__ Mentions<RowOf> no_mentions(uint32_t* slot, RowOf row_of) {   // a barrier must follow
    for (int i = threadIdx.x; i < kSlots / 4; i += kPoolThreads) reinterpret_cast<uint4*>(slot)[i] = make_uint4(0, 0, 0, 0);
    return {slot, row_of};
}

// Exclusive prefix sums of cnt[0 .. n) in place, cnt[n] = their total; n <= kMaxRows.
__device__ __forceinline__ int prefix_in_place(int32_t* cnt, int n, int* scratch) {
    constexpr int kPer = kPerThread;
    const int tid = threadIdx.x;
    int x[kPer], sum = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int i = tid * kPer + u;
        x[u] = i < n ? cnt[i] : 0;
        sum += x[u];
    }
    int tot;
    int at = sel::excl_scan<kPoolThreads, 0>(sum, tid, scratch, &tot);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int i = tid * kPer + u;
        if (i <= n) cnt[i] = at;
        at += x[u];
    }
    if (tid == 0) cnt[n] = tot;
    __syncthreads();
    return tot;
}

// The request whose entries hold rank e, which is `from` or one after it: the last i
// with cnt[i] <= e, cnt[n] > e.  Mostly `from` or the next; else a binary search.
__device__ __forceinline__ int owner_of(const int32_t* cnt, int n, int e, int from = 0) {
    int lo = from, hi = n - 1;
    if (e < cnt[lo + 1]) return lo;
    if (e < cnt[min(lo + 2, n)]) return lo + 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cnt[mid] <= e) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int len) { return len / kPage + (len % kPage != 0); }

// The e-th entry of the call takes the e-th free page, unless it holds one already; where
// that leaves entries without a page, they take the pages passed over.
__global__ void __launch_bounds__(kPoolThreads)
reserve_kernel(int32_t* __restrict__ ref, int64_t num_pages, int32_t* __restrict__ table, int rows, int max_pages,
               const int32_t* __restrict__ row, const int32_t* __restrict__ have, const int32_t* __restrict__ want, int n,
               int32_t* __restrict__ st) {
    extern __shared__ __align__(16) uint8_t smem[];
    PoolShared& sh = *reinterpret_cast<PoolShared*>(smem);
    int32_t *const s_at = sh.a, *const s_cnt = sh.cnt;     // the requests' rows, then their first entries in the table
    if (gridDim.x > 1) sm100::cluster_sync();              // the others' shared memory is there from here on
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const bool speaks = blockIdx.x == 0;                   // every block works the same requests out, one records
    Counts c;
    load_counts(c, ref, num_pages, first_count());
    auto named = no_mentions(sh.slot, [&](int m) { return s_at[m]; });
    int at[kPerThread], cnt[kPerThread];
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int i = tid + u * kPoolThreads;
        if (i >= n) continue;
        s_at[i] = at[u] = row[i];
        const int h = have[i], w = want[i], lo = pages_of(max(h, 0));
        int hi = pages_of(max(w, 0));
        cnt[u] = hi > max_pages ? -1 - w : lo > max_pages ? -1 - h : 0;   // -1 - a length beyond the table
        if (hi > max_pages) hi = max_pages;
        s_cnt[i] = max(0, hi - lo);
        at[u] = lo;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kPoolThreads) named.add(i);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int i = tid + u * kPoolThreads;
        if (i >= n) continue;
        const int r = s_at[i];
        const bool ok = r >= 0 && r < rows && named.least(r) == i;   // a row's first mention counts
        if (!ok) s_cnt[i] = 0;
        if (speaks && !ok) record_error(st, DSA_DEVERR_INDEX_RANGE, r);
        if (speaks && ok && cnt[u] < 0) record_error(st, DSA_DEVERR_INDEX_RANGE, -1 - cnt[u]);
        at[u] = ok && s_cnt[i] > 0 ? r * max_pages + at[u] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPerThread; ++u)
        if (tid + u * kPoolThreads < n) s_at[tid + u * kPoolThreads] = at[u];
    const int total = prefix_in_place(s_cnt, n, sh.scratch);
    auto entry = [=](int e, int& i) {                      // i: the owner of an earlier entry, then this one's
        i = owner_of(s_cnt, n, e, i);
        return table + s_at[i] + (e - s_cnt[i]);
    };
    int found = walk_free(c, ref, num_pages, total, true, sh, entry);
    if (found < total) {                                   // the same in every block
        if (gridDim.x > 1) sm100::cluster_sync();          // the others' entries and counts are written
        if (speaks) found = fill_rest(ref, num_pages, found, total, sh, entry);
    }
    int i = 0;
    if (speaks)                                            // what the pool does not hold; e passes 2^31 - 1
        for (int64_t e = (int64_t)found + tid; e < total; e += kPoolThreads)
            if (*entry((int)e, i) < 0) record_error(st, DSA_DEVERR_PAGE_POOL, row[i]);
}

// ---------------------------------------------------------------- fork
// A mention of a fork call counts if its rows are in range, it is the first to name
// its dst row, and that row is no source.  Asked of a whole block, which gets the
// answer in every thread.
__device__ __forceinline__ bool fork_counts(const int32_t* src, const int32_t* dst, int n, int f, int rows) {
    const int s = src[f], d = dst[f];
    bool ok = s >= 0 && s < rows && d >= 0 && d < rows;
    for (int j = threadIdx.x; j < n; j += blockDim.x) ok = ok && src[j] != d && (j >= f || dst[j] != d);
    return __syncthreads_and(ok);
}

__device__ __forceinline__ int fork_len(int len, int max_pages) {
    return (int)min((int64_t)max(len, 0), (int64_t)max_pages * kPage);
}

// First step: a free page for every child whose last page is partial.
__global__ void __launch_bounds__(kPoolThreads)
fork_take_kernel(int32_t* __restrict__ ref, int64_t num_pages, int32_t* __restrict__ table, int rows, int max_pages,
                 const int32_t* __restrict__ src, const int32_t* __restrict__ dst, const int32_t* __restrict__ length,
                 int n, int32_t* __restrict__ st) {
    extern __shared__ __align__(16) uint8_t smem[];
    PoolShared& sh = *reinterpret_cast<PoolShared*>(smem);
    int32_t *const s_dst = sh.a, *const s_cnt = sh.cnt;    // s_cnt: the source rows, then the pages taken before each child
    if (gridDim.x > 1) sm100::cluster_sync();              // the others' shared memory is there from here on
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const bool speaks = blockIdx.x == 0;                   // every block works the same children out, one records
    Counts c;
    load_counts(c, ref, num_pages, first_count());
    auto named = no_mentions(sh.slot, [&](int m) { return m < n ? s_cnt[m] : s_dst[m - n]; });   // as a source, then as a child
    for (int i = tid; i < n; i += kPoolThreads) {
        s_dst[i] = dst[i];
        s_cnt[i] = src[i];
    }
    __syncthreads();
    for (int i = tid; i < 2 * n; i += kPoolThreads) named.add(i);
    __syncthreads();
    int take[kPerThread];
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int i = tid + u * kPoolThreads;
        take[u] = 0;
        if (i >= n) continue;
        const int s = s_cnt[i], d = s_dst[i];
        if (s < 0 || s >= rows || d < 0 || d >= rows || named.least(d) != n + i) {   // no source, and no earlier child
            if (speaks) record_error(st, DSA_DEVERR_INDEX_RANGE, d);
            continue;
        }
        const int len = fork_len(length[i], max_pages);
        if (len != length[i] && speaks) record_error(st, DSA_DEVERR_INDEX_RANGE, length[i]);
        if (len % kPage == 0) continue;
        const int32_t pg = table[(int64_t)s * max_pages + len / kPage];
        take[u] = pg >= 0 && pg < num_pages;
        if (pg >= num_pages && speaks) record_error(st, DSA_DEVERR_PAGE_RANGE, pg);
        if (!take[u] && speaks) table[(int64_t)d * max_pages + len / kPage] = -1;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPerThread; ++u)
        if (tid + u * kPoolThreads < n) s_cnt[tid + u * kPoolThreads] = take[u];
    __syncthreads();
    const int total = prefix_in_place(s_cnt, n, sh.scratch);
    auto last = [&](int i) { return table + (int64_t)s_dst[i] * max_pages + fork_len(length[i], max_pages) / kPage; };
    const int found = walk_free(c, ref, num_pages, total, false, sh, [&](int e, int& i) { return last(i = owner_of(s_cnt, n, e, i)); });
    if (speaks)                                            // children that the pool holds no page for
        for (int e = found + tid; e < total; e += kPoolThreads) {
            const int i = owner_of(s_cnt, n, e);
            *last(i) = -1;
            record_error(st, DSA_DEVERR_PAGE_POOL, s_dst[i]);
        }
}

// Second step, one block per (child, job): jobs 0 .. n_caches - 1 copy the last
// page's rows in one cache, the others share a chunk of the full pages and clear
// the entries behind the last.
__global__ void __launch_bounds__(kCopyThreads)
fork_copy_kernel(int32_t* __restrict__ ref, int64_t num_pages, int32_t* __restrict__ table, int rows, int max_pages,
                 const int32_t* __restrict__ src, const int32_t* __restrict__ dst, const int32_t* __restrict__ length,
                 int n, CacheList cl, int n_caches, int share_jobs, int32_t* __restrict__ st) {
    pdl_wait();
    pdl_trigger();
    const int f = blockIdx.x, job = blockIdx.y, tid = threadIdx.x;
    if (!fork_counts(src, dst, n, f, rows)) return;
    const int len = fork_len(length[f], max_pages), full = len / kPage, part = len % kPage;
    const int32_t* ts = table + (int64_t)src[f] * max_pages;
    int32_t* td = table + (int64_t)dst[f] * max_pages;
    if (job >= n_caches) {
        for (int64_t k = (int64_t)(job - n_caches) * kCopyThreads + tid; k < max_pages; k += share_jobs * kCopyThreads) {
            if (k == full && part) continue;               // the copied page, set by the first step
            int32_t pg = -1;
            if (k < full) {
                pg = ts[k];
                if (pg >= num_pages) {
                    record_error(st, DSA_DEVERR_PAGE_RANGE, pg);
                    pg = -1;
                }
                if (pg >= 0) atomicAdd(ref + pg, 1);
                else pg = -1;
            }
            td[k] = pg;
        }
        return;
    }
    if (part == 0) return;
    const int64_t ps = ts[full], pd = td[full];
    if (ps < 0 || ps >= num_pages || pd < 0 || pd >= num_pages) return;   // recorded by the first step, or no page left
    const Layout lo = layout_of(cl.kind[job]);
    const uint4* from = reinterpret_cast<const uint4*>(cl.data[job] + ps * lo.page_bytes);
    uint4* to = reinterpret_cast<uint4*>(cl.data[job] + pd * lo.page_bytes);
    constexpr int kRowPieces = (kPage * (DSA_KV_TOKEN_BYTES / 16) + kCopyThreads - 1) / kCopyThreads;
    const int total = part * lo.row16;                     // rows are contiguous from the page's start
    uint4 v[kRowPieces];
#pragma unroll
    for (int u = 0; u < kRowPieces; ++u) {
        const int e = tid + u * kCopyThreads;
        if (e < total) v[u] = from[e];
    }
#pragma unroll
    for (int u = 0; u < kRowPieces; ++u) {
        const int e = tid + u * kCopyThreads;
        if (e < total) to[e] = v[u];
    }
    if (lo.scale_at && tid < part)
        reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(to) + lo.scale_at)[tid] =
            reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(from) + lo.scale_at)[tid];
}

// ---------------------------------------------------------------- host side
static dsa_status check_caches(const dsa_cache* caches, int32_t n) {
    if (n < 0 || (n > 0 && !caches)) return DSA_ERR_INVALID_ARGUMENT;
    for (int32_t c = 0; c < n; ++c) {
        if (!caches[c].data || caches[c].kind < DSA_CACHE_KV || caches[c].kind > DSA_CACHE_IDXK_MXFP4)
            return DSA_ERR_INVALID_ARGUMENT;
        if (!aligned16(caches[c].data)) return DSA_ERR_ALIGNMENT;
    }
    return DSA_OK;
}
static CacheList list_of(const dsa_cache* caches, int32_t at, int32_t n) {
    CacheList cl = {};
    for (int32_t c = 0; c < n; ++c) {
        cl.data[c] = caches[at + c].data;
        cl.kind[c] = (uint8_t)caches[at + c].kind;
    }
    return cl;
}
static dsa_status check_pool(const int32_t* page_ref, int64_t num_pages, const int32_t* page_table, int32_t rows,
                             int32_t max_pages, int32_t n) {
    if (n < 0 || num_pages < 1 || rows < 1 || max_pages < 1) return DSA_ERR_INVALID_ARGUMENT;
    if (num_pages * kPage > 0x7fffffffLL || (int64_t)rows * max_pages > 0x7fffffffLL || max_pages > 0x7fffffff / kPage)
        return DSA_ERR_UNSUPPORTED;                        // 32-bit slots, table entries and lengths
    if (n == 0) return DSA_OK;
    if (!page_ref || !page_table) return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(page_ref)) return DSA_ERR_ALIGNMENT;
    return DSA_OK;
}

// Blocks that walk the counts (one cluster): as many as have a count to look at.
static unsigned pool_blocks(int64_t num_pages) {
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((num_pages + kStep - 1) / kStep, kPoolBlocks));
}
// Blocks for a request's table entries: a thread takes one each up to 64 blocks (16K entries), then goes round again.
static unsigned entry_blocks(int32_t max_pages) { return (unsigned)std::min((max_pages + kReleaseThreads - 1) / kReleaseThreads, 64); }

}  // namespace pages
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_tree_commit(const int32_t* accept, int32_t width, const dsa_batch* b, const dsa_cache* caches,
                                      int32_t n_caches, int32_t* new_seq_len, int32_t* dev_status, void* stream) {
    dsa_status vs = validate_batch(b);
    if (vs != DSA_OK) return vs;
    if (width < 0) return DSA_ERR_INVALID_ARGUMENT;
    vs = pages::check_caches(caches, n_caches);
    if (vs != DSA_OK) return vs;
    if (width > pages::kMaxAccept || b->num_pages * kPage > 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;
    if (width > 0 && !accept) return DSA_ERR_INVALID_ARGUMENT;
    // several blocks read a request's seq_len, one writes its new length
    const uintptr_t from = reinterpret_cast<uintptr_t>(b->seq_len), to = reinterpret_cast<uintptr_t>(new_seq_len);
    const uintptr_t lens = sizeof(int32_t) * (uintptr_t)b->batch;
    if (new_seq_len && to < from + lens && from < to + lens) return DSA_ERR_INVALID_ARGUMENT;
    if (n_caches == 0 && !new_seq_len) return DSA_OK;
    if (ensure_smem_limit(reinterpret_cast<const void*>(&pages::commit_kernel), pages::kCommitSmem) != DSA_OK) return DSA_ERR_CUDA;
    int32_t at = 0;
    do {                                                   // 128 caches a launch; the first writes the lengths
        const int32_t n = n_caches - at < pages::kMaxCaches ? n_caches - at : pages::kMaxCaches;
        const int32_t want = std::min(std::max(1, pages::kCommitBlocks * device_sm_count() / b->batch), std::max(1, n));
        const int32_t per = std::max(1, (n + want - 1) / want);
        DSA_CHECK(launch_pdl(pages::commit_kernel, dim3((unsigned)b->batch, (unsigned)std::max(1, (n + per - 1) / per)),
                             dim3(pages::kCopyThreads), pages::kCommitSmem, as_stream(stream), 1, accept, (int)width, to_dev(b),
                             pages::list_of(caches, at, n), (int)n, (int)per, at == 0 ? new_seq_len : nullptr,
                             at == 0 ? dev_status : nullptr));
        at += n;
    } while (at < n_caches);
    return DSA_OK;
}

extern "C" dsa_status dsa_pages_reserve(int32_t* page_ref, int64_t num_pages, int32_t* page_table, int32_t rows,
                                        int32_t max_pages, const int32_t* row, const int32_t* have_len,
                                        const int32_t* want_len, int32_t n, int32_t* dev_status, void* stream) {
    const dsa_status vs = pages::check_pool(page_ref, num_pages, page_table, rows, max_pages, n);
    if (vs != DSA_OK || n == 0) return vs;
    if (!row || !have_len || !want_len) return DSA_ERR_INVALID_ARGUMENT;
    if (n > pages::kMaxRows) return DSA_ERR_UNSUPPORTED;
    const unsigned blocks = pages::pool_blocks(num_pages);
    if (ensure_smem_limit(reinterpret_cast<const void*>(&pages::reserve_kernel), sizeof(pages::PoolShared)) != DSA_OK) return DSA_ERR_CUDA;
    DSA_CHECK(launch_pdl(pages::reserve_kernel, dim3(blocks), dim3(pages::kPoolThreads), sizeof(pages::PoolShared), as_stream(stream), blocks,
                         page_ref, num_pages, page_table, (int)rows, (int)max_pages, row, have_len, want_len, (int)n,
                         dev_status));
    return DSA_OK;
}

extern "C" dsa_status dsa_pages_release(int32_t* page_ref, int64_t num_pages, int32_t* page_table, int32_t rows,
                                        int32_t max_pages, const int32_t* row, const int32_t* first_page,
                                        const int32_t* end_page, int32_t n, int32_t* dev_status, void* stream) {
    const dsa_status vs = pages::check_pool(page_ref, num_pages, page_table, rows, max_pages, n);
    if (vs != DSA_OK || n == 0) return vs;
    if (!row || !first_page || !end_page) return DSA_ERR_INVALID_ARGUMENT;
    DSA_CHECK(launch_pdl(pages::release_kernel, dim3((unsigned)n, pages::entry_blocks(max_pages)),
                         dim3(pages::kReleaseThreads), 0, as_stream(stream), 1, page_ref, num_pages, page_table, (int)rows,
                         (int)max_pages, row, first_page, end_page, dev_status));
    return DSA_OK;
}

extern "C" dsa_status dsa_pages_fork(int32_t* page_ref, int64_t num_pages, int32_t* page_table, int32_t rows,
                                     int32_t max_pages, const int32_t* src_row, const int32_t* dst_row,
                                     const int32_t* length, int32_t n, const dsa_cache* caches, int32_t n_caches,
                                     int32_t* dev_status, void* stream) {
    dsa_status vs = pages::check_pool(page_ref, num_pages, page_table, rows, max_pages, n);
    if (vs != DSA_OK) return vs;
    vs = pages::check_caches(caches, n_caches);
    if (vs != DSA_OK || n == 0) return vs;
    if (!src_row || !dst_row || !length) return DSA_ERR_INVALID_ARGUMENT;
    if (n > pages::kMaxRows) return DSA_ERR_UNSUPPORTED;
    const unsigned blocks = pages::pool_blocks(num_pages);
    if (ensure_smem_limit(reinterpret_cast<const void*>(&pages::fork_take_kernel), sizeof(pages::PoolShared)) != DSA_OK) return DSA_ERR_CUDA;
    DSA_CHECK(launch_pdl(pages::fork_take_kernel, dim3(blocks), dim3(pages::kPoolThreads), sizeof(pages::PoolShared), as_stream(stream), blocks,
                         page_ref, num_pages, page_table, (int)rows, (int)max_pages, src_row, dst_row, length, (int)n,
                         dev_status));
    const int chunks = (max_pages + pages::kCopyThreads - 1) / pages::kCopyThreads;
    int32_t at = 0;
    do {                                                   // the first launch shares the full pages too
        const int32_t c = n_caches - at < pages::kMaxCaches ? n_caches - at : pages::kMaxCaches;
        const int share = at == 0 ? (chunks < 16 ? chunks : 16) : 0;
        DSA_CHECK(launch_pdl(pages::fork_copy_kernel, dim3((unsigned)n, (unsigned)(c + share)), dim3(pages::kCopyThreads), 0,
                             as_stream(stream), 1, page_ref, num_pages, page_table, (int)rows, (int)max_pages, src_row,
                             dst_row, length, (int)n, pages::list_of(caches, at, c), (int)c, share, dev_status));
        at += c;
    } while (at < n_caches);
    return DSA_OK;
}
