// Tokens and pages of the paged caches: the accepted path of a draft tree moved
// to the front of its tokens, requests that share or give back pages, and the
// pool of page counts behind them.  No call reads anything back to the host.
//
// All of it is copying and counting: a move is bound by HBM (row bytes read and
// written once), the pool calls by latency (one pass over the counts up to the
// last page taken).
#include "dsa_internal.cuh"
#include "indexer_common.cuh"
#include "select_common.cuh"

namespace dsa {
namespace pages {

constexpr int kMaxCaches = 128;                            // caches of one launch (passed by value)
constexpr int kMaxRows = 4096;                             // requests of one reserve or fork call
constexpr int kMaxAccept = 64;
constexpr int kCopyThreads = 256;
constexpr int kPoolThreads = 1024;

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
// One block per (request, cache).  Every row that moves is read into registers
// (at most 64 rows x 41 pieces, 11 per thread, all loads in flight) before the
// barrier and written after it, so a row may be another row's target.
constexpr int kRowPieces = (kMaxAccept * (DSA_KV_TOKEN_BYTES / 16) + kCopyThreads - 1) / kCopyThreads;

__global__ void __launch_bounds__(kCopyThreads)
commit_kernel(const int32_t* __restrict__ accept, int width, BatchDev b, CacheList cl, int n_caches,
              int32_t* __restrict__ new_len, int32_t* __restrict__ st) {
    __shared__ int32_t s_src[kMaxAccept], s_dst[kMaxAccept];
    __shared__ int32_t s_n;
    pdl_wait();
    pdl_trigger();
    const int r = blockIdx.x, c = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    if (tid < 32) {
        const int qn = b.q_start[r + 1] - b.q_start[r];
        const int P = b.seq_len[r] - qn;
        int a[2], kept = 0;
        bool open = true;                                  // the list has not ended yet
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = h * 32 + lane;
            a[h] = k < width ? accept[(int64_t)r * width + k] : -1;
            const unsigned end = __ballot_sync(0xffffffffu, a[h] < 0 || a[h] >= qn);
            const int n = !open ? 0 : end ? __ffs(end) - 1 : 32;
            if (open && end && c == 0) {
                const int bad = __shfl_sync(0xffffffffu, a[h], __ffs(end) - 1);
                if (lane == 0 && bad >= 0) record_error(st, DSA_DEVERR_INDEX_RANGE, bad);
            }
            kept += n;
            open = open && !end;
        }
        if (P < 0 && kept > 0) {                           // more new tokens than the request holds
            if (lane == 0 && c == 0) record_error(st, DSA_DEVERR_INDEX_RANGE, P);
            kept = 0;
        }
        if (c == 0 && lane == 0 && new_len) new_len[r] = P + kept;
        int n_moves = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = h * 32 + lane;
            int src = -1, dst = -1;
            if (k < kept && a[h] != k) {                   // a token already in place stays
                const int js = P + a[h], jd = P + k;
                if (js / kPage >= b.max_pages || jd / kPage >= b.max_pages) {
                    if (c == 0) record_error(st, DSA_DEVERR_INDEX_RANGE, js);
                } else {
                    const int64_t ps = b.page_table[(int64_t)r * b.max_pages + js / kPage];
                    const int64_t pd = b.page_table[(int64_t)r * b.max_pages + jd / kPage];
                    if (ps < 0 || ps >= b.num_pages || pd < 0 || pd >= b.num_pages) {
                        if (c == 0) record_error(st, DSA_DEVERR_PAGE_RANGE, ps < 0 || ps >= b.num_pages ? ps : pd);
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
    if (n == 0 || c >= n_caches) return;
    const Layout lo = layout_of(cl.kind[c]);
    uint8_t* base = cl.data[c];
    const int total = n * lo.row16;
    uint4 v[kRowPieces];
    uint32_t word = 0;
#pragma unroll
    for (int u = 0; u < kRowPieces; ++u) {
        const int e = tid + u * kCopyThreads;
        if (e < total) {
            const int m = e / lo.row16, piece = e - m * lo.row16;
            const int32_t s = s_src[m];
            v[u] = *reinterpret_cast<const uint4*>(base + (int64_t)(s / kPage) * lo.page_bytes +
                                                   ((s % kPage) * lo.row16 + piece) * 16);
        }
    }
    if (lo.scale_at && tid < n)
        word = *reinterpret_cast<const uint32_t*>(base + (int64_t)(s_src[tid] / kPage) * lo.page_bytes + lo.scale_at +
                                                  (s_src[tid] % kPage) * 4);
    __syncthreads();                                       // every source row has been read
#pragma unroll
    for (int u = 0; u < kRowPieces; ++u) {
        const int e = tid + u * kCopyThreads;
        if (e < total) {
            const int m = e / lo.row16, piece = e - m * lo.row16;
            const int32_t d = s_dst[m];
            *reinterpret_cast<uint4*>(base + (int64_t)(d / kPage) * lo.page_bytes + ((d % kPage) * lo.row16 + piece) * 16) =
                v[u];
        }
    }
    if (lo.scale_at && tid < n)
        *reinterpret_cast<uint32_t*>(base + (int64_t)(s_dst[tid] / kPage) * lo.page_bytes + lo.scale_at +
                                     (s_dst[tid] % kPage) * 4) = word;
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
// Walks the free pages in ascending order and calls take(rank, page) for the
// first `want` of them; returns how many there were (at most want).  One block:
// each step covers 16 counts per thread, the next step's loads in flight while
// this one's ranks are scanned.
constexpr int kStep = 16 * kPoolThreads;

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

template <typename Take>
__device__ __forceinline__ int walk_free(const int32_t* ref, int64_t num_pages, int want, int* scratch, Take take) {
    const int tid = threadIdx.x;
    int found = 0;
    Counts next;
    load_counts(next, ref, num_pages, (int64_t)tid * 16);
    for (int64_t base = 0; base < num_pages && found < want; base += kStep) {
        const Counts c = next;
        if (base + kStep < num_pages) load_counts(next, ref, num_pages, base + kStep + (int64_t)tid * 16);
        int n = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) n += (c.v[u].x == 0) + (c.v[u].y == 0) + (c.v[u].z == 0) + (c.v[u].w == 0);
        int tot;
        int rank = found + sel::excl_scan<kPoolThreads, 0>(n, tid, scratch, &tot);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int x[4] = {c.v[u].x, c.v[u].y, c.v[u].z, c.v[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (x[e] == 0) {
                    if (rank < want) take(rank, base + (int64_t)tid * 16 + 4 * u + e);
                    ++rank;
                }
        }
        found += tot;
    }
    return min(found, want);
}

// Exclusive prefix sums of cnt[0 .. n) in place, cnt[n] = their total; n <= kMaxRows.
__device__ __forceinline__ int prefix_in_place(int32_t* cnt, int n, int* scratch) {
    constexpr int kPer = kMaxRows / kPoolThreads;
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

// The request whose entries hold rank e: the last i with cnt[i] <= e.
__device__ __forceinline__ int owner_of(const int32_t* cnt, int n, int e) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cnt[mid] <= e) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int len) { return len / kPage + (len % kPage != 0); }

__global__ void __launch_bounds__(kPoolThreads)
reserve_kernel(int32_t* __restrict__ ref, int64_t num_pages, int32_t* __restrict__ table, int rows, int max_pages,
               const int32_t* __restrict__ row, const int32_t* __restrict__ have, const int32_t* __restrict__ want, int n,
               int32_t* __restrict__ st) {
    __shared__ int32_t s_row[kMaxRows], s_cnt[kMaxRows + 1];
    __shared__ int scratch[64];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    for (int i = tid; i < n; i += kPoolThreads) s_row[i] = row[i];
    __syncthreads();
    for (int i = tid; i < n; i += kPoolThreads) {
        const int r = s_row[i];
        bool ok = r >= 0 && r < rows;
        for (int j = 0; j < i && ok; ++j) ok = s_row[j] != r;
        if (!ok) record_error(st, DSA_DEVERR_INDEX_RANGE, r);
        int hi = pages_of(max(want[i], 0));
        if (ok && hi > max_pages) {
            record_error(st, DSA_DEVERR_INDEX_RANGE, want[i]);
            hi = max_pages;
        }
        s_cnt[i] = ok ? max(0, hi - pages_of(max(have[i], 0))) : 0;
    }
    __syncthreads();
    const int total = prefix_in_place(s_cnt, n, scratch);
    auto entry = [&](int e) {
        const int i = owner_of(s_cnt, n, e);
        return table + (int64_t)s_row[i] * max_pages + pages_of(max(have[i], 0)) + (e - s_cnt[i]);
    };
    const int found = walk_free(ref, num_pages, total, scratch, [&](int rank, int64_t page) {
        int32_t* t = entry(rank);
        if (*t < 0) {
            *t = (int32_t)page;
            ref[page] = 1;
        }
    });
    for (int e = found + tid; e < total; e += kPoolThreads)
        if (*entry(e) < 0) record_error(st, DSA_DEVERR_PAGE_POOL, s_row[owner_of(s_cnt, n, e)]);
}

// ---------------------------------------------------------------- fork
// Whether mention f of a fork call counts: rows in range, the first to name its
// dst row, and that row no source.  One thread looks at every other mention.
__device__ __forceinline__ bool fork_counts(const int32_t* __restrict__ src, const int32_t* dst, int n, int f, int rows) {
    const int s = src[f], d = dst[f];
    bool ok = s >= 0 && s < rows && d >= 0 && d < rows;
    for (int j = 0; j < n && ok; ++j) ok = src[j] != d && (j >= f || dst[j] != d);
    return ok;
}
// The same with a whole block's threads (every thread gets the answer).
__device__ __forceinline__ bool fork_counts_block(const int32_t* src, const int32_t* dst, int n, int f, int rows) {
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
    __shared__ int32_t s_dst[kMaxRows], s_cnt[kMaxRows + 1];
    __shared__ int scratch[64];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    for (int i = tid; i < n; i += kPoolThreads) s_dst[i] = dst[i];
    __syncthreads();
    for (int i = tid; i < n; i += kPoolThreads) {
        int take = 0;
        if (!fork_counts(src, s_dst, n, i, rows)) {
            record_error(st, DSA_DEVERR_INDEX_RANGE, s_dst[i]);
        } else {
            const int len = fork_len(length[i], max_pages);
            if (len != length[i]) record_error(st, DSA_DEVERR_INDEX_RANGE, length[i]);
            if (len % kPage) {
                const int32_t pg = table[(int64_t)src[i] * max_pages + len / kPage];
                take = pg >= 0 && pg < num_pages;
                table[(int64_t)s_dst[i] * max_pages + len / kPage] = -1;   // until a page is found for it
                if (pg >= num_pages) record_error(st, DSA_DEVERR_PAGE_RANGE, pg);
            }
        }
        s_cnt[i] = take;
    }
    __syncthreads();
    const int total = prefix_in_place(s_cnt, n, scratch);
    const int found = walk_free(ref, num_pages, total, scratch, [&](int rank, int64_t page) {
        const int i = owner_of(s_cnt, n, rank);
        table[(int64_t)s_dst[i] * max_pages + fork_len(length[i], max_pages) / kPage] = (int32_t)page;
        ref[page] = 1;
    });
    for (int e = found + tid; e < total; e += kPoolThreads)
        record_error(st, DSA_DEVERR_PAGE_POOL, s_dst[owner_of(s_cnt, n, e)]);
}

// Second step, one block per (child, job): jobs 0 .. n_caches - 1 copy the last
// page's rows in one cache, the others share a chunk of the full pages and
// clear the entries behind the last.
__global__ void __launch_bounds__(kCopyThreads)
fork_copy_kernel(int32_t* __restrict__ ref, int64_t num_pages, int32_t* __restrict__ table, int rows, int max_pages,
                 const int32_t* __restrict__ src, const int32_t* __restrict__ dst, const int32_t* __restrict__ length,
                 int n, CacheList cl, int n_caches, int share_jobs, int32_t* __restrict__ st) {
    pdl_wait();
    pdl_trigger();
    const int f = blockIdx.x, job = blockIdx.y, tid = threadIdx.x;
    if (!fork_counts_block(src, dst, n, f, rows)) return;
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
    if (num_pages * kPage > 0x7fffffffLL || max_pages > 0x7fffffff / kPage) return DSA_ERR_UNSUPPORTED;
    if (n == 0) return DSA_OK;
    if (!page_ref || !page_table) return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(page_ref)) return DSA_ERR_ALIGNMENT;
    return DSA_OK;
}

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
    if (n_caches == 0 && !new_seq_len) return DSA_OK;
    int32_t at = 0;
    do {                                                   // 128 caches a launch; the first writes the lengths
        const int32_t n = n_caches - at < pages::kMaxCaches ? n_caches - at : pages::kMaxCaches;
        DSA_CHECK(launch_pdl(pages::commit_kernel, dim3((unsigned)b->batch, (unsigned)(n > 0 ? n : 1)),
                             dim3(pages::kCopyThreads), 0, as_stream(stream), 1, accept, (int)width, to_dev(b),
                             pages::list_of(caches, at, n), (int)n, at == 0 ? new_seq_len : nullptr,
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
    if (n > pages::kMaxRows || (int64_t)n * max_pages > 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;
    DSA_CHECK(launch_pdl(pages::reserve_kernel, dim3(1), dim3(pages::kPoolThreads), 0, as_stream(stream), 1, page_ref,
                         num_pages, page_table, (int)rows, (int)max_pages, row, have_len, want_len, (int)n, dev_status));
    return DSA_OK;
}

extern "C" dsa_status dsa_pages_release(int32_t* page_ref, int64_t num_pages, int32_t* page_table, int32_t rows,
                                        int32_t max_pages, const int32_t* row, const int32_t* first_page,
                                        const int32_t* end_page, int32_t n, int32_t* dev_status, void* stream) {
    const dsa_status vs = pages::check_pool(page_ref, num_pages, page_table, rows, max_pages, n);
    if (vs != DSA_OK || n == 0) return vs;
    if (!row || !first_page || !end_page) return DSA_ERR_INVALID_ARGUMENT;
    // a block's threads take one entry each up to 64 blocks a request (16K entries), then go round again
    const int chunks = (max_pages + pages::kReleaseThreads - 1) / pages::kReleaseThreads;
    DSA_CHECK(launch_pdl(pages::release_kernel, dim3((unsigned)n, (unsigned)(chunks < 64 ? chunks : 64)),
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
    DSA_CHECK(launch_pdl(pages::fork_take_kernel, dim3(1), dim3(pages::kPoolThreads), 0, as_stream(stream), 1, page_ref,
                         num_pages, page_table, (int)rows, (int)max_pages, src_row, dst_row, length, (int)n, dev_status));
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
