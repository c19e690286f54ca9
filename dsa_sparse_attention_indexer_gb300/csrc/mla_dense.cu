// MLA over a whole context of the paged latent cache: a sliding window with the
// context's first tokens (sinks), and trees of drafted tokens.
//   S_hj = scale * <q_h, [c_j * s_j | r_j]>,  out_h = sum_j softmax_j(S_hj) c_j
// over the positions j that the query row sees, 64 heads of 576 dims, in one
// pass over the pages with a running maximum and sum per head.
//
// Work split: a row's visible pages are taken two at a time, as tiles of 128
// tokens.  The tiles of all rows form one line that is cut into equal shares,
// one per CTA, so ragged contexts and any number of rows fill the GPU alike;
// every CTA counts the tiles itself (a block scan over the rows).  A row that
// several shares hold leaves one partial (O, running max, sum) per share, and a
// second kernel merges them by their log-sum-exp.
//
// Per tile, in transposed form so that tokens are the MMA rows:
//   S^T = K Q^T      tcgen05.mma kind::f16, M = 128 tokens, N = 64 heads, K = 576
//   O^T += V^T P^T   M = 4 x 128 latent dims, N = 64 heads, K = 128 tokens,
//                    A = the same tile read MN-major; 256 TMEM columns stay
//                    resident for the row
// The tile in fp16 (147 KB) and the row's Q (74 KB) fill shared memory, so the
// tile is recycled group by group: the loaders write 128 latent dims of the
// next tile as soon as the P.V MMAs of those dims have completed, and S^T of
// the next tile starts behind the last P.V.  P^T takes the place of the tile's
// RoPE block, which S^T has read by then.
//
// Warps 0-15 do everything but issue the MMAs; a tile's phases follow one another,
// so the same warps take them in turn:
//   softmax     a thread owns one token (TMEM lane) and 16 heads.  P is formed
//               against a reference that lags the maximum by up to 2^12 before
//               O^T is rescaled, and shifted up by 2^3, so that fp16 holds
//               probabilities down to 2^-28 of the reference;
//   next tile   its rows, read into registers a tile ahead (whole pages are
//               prefetched into L2 before that), are dequantised into the
//               128-byte-swizzled tile (exact for scales in [2^-15, 2^7]), each
//               part as soon as it is free.  Rows that are not seen become zeros;
//   next row    its Q, scaled by the power of two that puts its largest |q| in
//               [2^14, 2^15), while the last P.V runs; then the epilogue, while
//               the first S^T of the next row runs.
// Warp 16 issues the MMAs.
// Every wait is time-bounded; a timeout is recorded and the CTA winds down.
#include <algorithm>

#include "dsa_internal.cuh"
#include "indexer_common.cuh"
#include "mla_common.cuh"
#include "select_common.cuh"
#include "sm100.cuh"

namespace dsa {

int device_sm_count();

namespace mld {

struct Meta;

// Which positions a launch's rows see: window form (tree == NULL) or tree form.
struct View {
    const uint64_t* tree;       // [T] masks of new tokens, or NULL
    int32_t window, sinks;
};

struct Args {
    const uint16_t* q;          // [T,64,576] bf16
    const uint8_t* kv;          // latent cache
    BatchDev b;
    View view;
    float scale_log2;
    void* out;
    int out_f32;
    float* lse;
    float* part_o;              // [2 G, 64, 512]: unnormalised outputs of cut rows, two pieces per share
    float2* part_ml;            // [2 G, 64]: reference (log2 units), sum
    Meta* meta;          // [G]
    int32_t* st;
};

// One row's visible positions: j < sink_end or first <= j < end, and new token
// u at position prefix + u when bit u of mask is set.  They lie in `pages`
// pages: the first sink_pages, then those from first_page on.
struct Row {
    int32_t r;                  // request
    int32_t sink_end, first, end;
    int32_t prefix;
    uint64_t mask;
    int32_t sink_pages, first_page, pages;
    __device__ __forceinline__ int page(int u) const volatile { return u < sink_pages ? u : first_page + u - sink_pages; }
    // The positions of logical page lp that the row sees, one bit each.
    __device__ __forceinline__ uint64_t seen(int lp) const volatile {
        const int j = lp * kPage;
        const uint64_t sinks = below(sink_end - j), from = below(end - j) & ~below(first - j);
        const int sh = prefix - j;
        const uint64_t news = sh >= 64 || sh <= -64 ? 0ull : sh >= 0 ? mask << sh : mask >> -sh;
        return sinks | from | news;
    }
    static __device__ __forceinline__ uint64_t below(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }
};

// Row `row` of the batch.  A row that sees nothing keeps one (empty) page, so
// that every row of a request is written; rows behind the last request have none.
__device__ __forceinline__ Row row_view(const BatchDev& b, const View& v, int64_t row, int32_t* st) {
    Row w = {};
    if (row >= b.q_start[b.batch]) return w;
    w.r = row_request(b.q_start, b.batch, row);
    const int qs = b.q_start[w.r], qn = b.q_start[w.r + 1] - qs;
    const int64_t room = (int64_t)b.max_pages * kPage;
    int L = b.seq_len[w.r];
    if (L > room) {
        record_error(st, DSA_DEVERR_INDEX_RANGE, L);
        L = (int)room;
    }
    w.prefix = b.seq_len[w.r] - qn;
    w.pages = 1;
    if (L <= 0 || w.prefix < 0) return w;
    if (v.tree) {
        const int known = min(qn, 64);
        w.mask = v.tree[row] & (known >= 64 ? ~0ull : (1ull << known) - 1);
        w.end = min(w.prefix, L);
        const int64_t last = w.mask ? (int64_t)w.prefix + 64 - __clzll((long long)w.mask) : w.end;
        if (last > L) w.mask = L > w.prefix ? w.mask & ((1ull << (L - w.prefix)) - 1) : 0;
        w.pages = max(1, (int)((min(last, (int64_t)L) + kPage - 1) / kPage));
        return w;
    }
    const int end = (int)min((int64_t)w.prefix + (row - qs) + 1, (int64_t)L);
    w.end = end;
    w.first = max(0, w.prefix + (int)(row - qs) + 1 - v.window);
    w.sink_end = min(v.sinks, end);
    w.sink_pages = w.sink_end / kPage + (w.sink_end % kPage != 0);
    w.first_page = max(w.sink_pages, w.first / kPage);
    w.pages = max(1, w.sink_pages + max(0, (end + kPage - 1) / kPage - w.first_page));
    return w;
}

using namespace sm100;
using namespace mlc;

constexpr int kTok = 128;                                  // tokens per tile: two pages
constexpr int kBlk = kTok * 128;                           // one 64-dim K-block of the tile
constexpr int kWorkWarps = 16;
constexpr int kWorkThreads = kWorkWarps * 32;
constexpr int kHeads = 16;                                 // heads of a warp in the softmax: four warps a TMEM lane quarter
constexpr int kMmaWarp = kWorkWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;              // five warpgroups; the last one's first warp issues the MMAs
constexpr int kWorkBar = 1;
constexpr int kSteps = kTok / kWorkWarps / 4;              // a warp's 8 tokens of a tile, four at a time
constexpr float kTau = 12.0f;                              // lazy-rescale threshold, log2 units
constexpr float kShift = 3.0f;                             // P is scaled by 2^3 ..
constexpr uint32_t kPMaxH = 0x7800;                        // .. so at most 2^(kTau + kShift) = 2^15, as fp16 bits
constexpr float kNoRef = 0x1p100f;                         // minus the reference of a head without one: P of any score is inf
constexpr uint32_t kIdescQK = idesc_f16_f32(128, 64, false, false);
constexpr uint32_t kIdescPV = idesc_f16_f32(128, 64, true, true);
constexpr uint32_t kColS = 0;                              // TMEM: S^T [128 x 64]
constexpr uint32_t kColO = 64;                             // TMEM: O^T 4 x [128 x 64]

constexpr int kOffKV = 0;                                  // 8 latent K-blocks and the RoPE block (later P^T), [128 tokens x 128 B]
constexpr int kOffP = kOffKV + 8 * kBlk;
constexpr int kOffQ = kOffKV + 9 * kBlk;                   // 9 K-blocks of [64 heads x 128 B]
constexpr int kOffRed = kOffQ + 9 * 8192;                  // [2][4 lane quarters][64 heads] fp32
constexpr int kOffStat = kOffRed + 2 * 4 * 64 * 4;         // neg_ref, l_acc, alpha [64], 16 times -inf
constexpr int kOffBars = kOffStat + (3 * 64 + 16) * 4;
constexpr int kOffMisc = kOffBars + 16 * 8;
constexpr int kOffRows = kOffMisc + 512;                   // every warp's current row, re-read instead of held in registers
constexpr int kSmemUsed = kOffRows + (kThreads / 32) * (int)sizeof(Row);
static_assert(sizeof(Row) % 8 == 0, "rows are 8-byte aligned");
constexpr int kSmemAlloc = kSmemUsed + 1024;
static_assert(kSmemAlloc <= 232448, "shared memory budget");
static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kBlk % 1024 == 0, "swizzle atoms need 1 KB alignment");
static_assert(kOffStat % 16 == 0, "reference maxima are read as float4");

enum { B_QFULL = 0, B_FULL0, B_FULL4 = B_FULL0 + 4, B_SFULL, B_PREADY, B_PV0, B_PV3 = B_PV0 + 3, B_DRAIN, B_COUNT };
static_assert(B_COUNT <= 16, "barrier block");

struct Misc {
    uint32_t tmem_base;
    int32_t abort;
    uint32_t qmax[kWorkWarps];  // per warp: largest bf16 magnitude of the row's q
    int32_t scratch[32];
    int64_t total;              // tiles of the whole batch
    int32_t row0, tile0;        // where this CTA's share begins
};
static_assert(sizeof(Misc) <= 512, "misc block");

// Where a CTA's share begins, for the merge: its first row (-1: no share) and
// whether that row began in an earlier share.
struct Meta {
    int32_t row;
    int32_t inside;
};

__device__ __forceinline__ bool work_any(bool pred) { return bar_any<kWorkBar, kWorkThreads>(pred); }
__device__ __forceinline__ void work_sync() { bar_sync<kWorkBar, kWorkThreads>(); }

__device__ __forceinline__ int tiles_of(const Row& w) { return (w.pages + 1) >> 1; }

// Counts the tiles of all rows (the workers' threads, consecutive rows each)
// and finds where share g of G begins.  Returns the share's tiles.
__device__ __forceinline__ void plan_share(const Args& a, Misc* misc, int tid) {
    const int64_t T = a.b.total_q;
    const int64_t per = (T + kWorkThreads - 1) / kWorkThreads;
    const int64_t r0 = min(T, tid * per), r1 = min(T, r0 + per);
    int64_t mine = 0;
    for (int64_t r = r0; r < r1; ++r) mine += tiles_of(row_view(a.b, a.view, r, nullptr));
    // block scan in 64 bits: warps, then their totals
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if ((tid & 31) >= o) x += y;
    }
    int64_t* tot = reinterpret_cast<int64_t*>(misc->scratch);     // 16 warps
    if ((tid & 31) == 31) tot[tid >> 5] = x;
    work_sync();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kWorkThreads / 32; ++w) {
        if (w < (tid >> 5)) before += tot[w];
        all += tot[w];
    }
    before += x - mine;
    if (tid == 0) misc->total = all;
    const int64_t G = min((int64_t)gridDim.x, all);
    if ((int64_t)blockIdx.x < G) {
        int64_t at = (int64_t)blockIdx.x * all / G;
        if (at >= before && at < before + mine) {
            at -= before;
            int64_t r = r0;
            for (;; ++r) {
                const int n = tiles_of(row_view(a.b, a.view, r, nullptr));
                if (at < n) break;
                at -= n;
            }
            misc->row0 = (int32_t)r;
            misc->tile0 = (int32_t)at;
        }
    }
}

// Registers per thread: 96 at launch (65,536 / 640 threads, in eights), of which
// the MMA warpgroup gives most to the others: 512 x 112 + 128 x 32 = 640 x 96.
constexpr int kLaunchRegs = 96, kWorkRegs = 112, kMmaRegs = 32;
static_assert(kWorkThreads * kWorkRegs + 128 * kMmaRegs <= kThreads * kLaunchRegs, "more registers than the launch holds");
template <int R> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// The descriptors of an MMA are a base plus a constant.  Formed from a value the
// compiler cannot see through, they are not kept across the tile loop, where
// 68 pairs of them would spill.
__device__ __forceinline__ void keep_here(uint64_t& d) { asm volatile("" : "+l"(d)); }

// S^T += K-blocks [B0, B0 + NB) of the tile x the same blocks of Q, four K = 16
// steps per 64-dim block; the first MMA of a tile overwrites.
template <int B0, int NB>
__device__ __forceinline__ void qk_blocks(uint32_t d_tmem, uint64_t d_kv, uint64_t d_q) {
    keep_here(d_kv);
    keep_here(d_q);
#pragma unroll
    for (int bk = B0; bk < B0 + NB; ++bk)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma_f16(d_tmem, d_kv + (uint64_t)((bk * kBlk + kk * 32) >> 4), d_q + (uint64_t)((bk * 8192 + kk * 32) >> 4),
                    kIdescQK, (bk == 0 && kk == 0) ? 0u : 1u);
}
// O^T rows of latent block MB += V^T P^T over the tile's eight 16-token steps,
// then a commit that releases the block's part of the tile.
template <int MB>
__device__ __forceinline__ void pv_block(uint32_t o_tmem, uint64_t d_v, uint64_t d_p, bool acc0, uint64_t* bar) {
    keep_here(d_v);
    keep_here(d_p);
#pragma unroll
    for (int kt = 0; kt < kTok / 16; ++kt)
        mma_f16(o_tmem + MB * 64, d_v + (uint64_t)((2 * MB * kBlk + kt * 2048) >> 4), d_p + (uint64_t)((kt * 2048) >> 4),
                kIdescPV, (acc0 || kt > 0) ? 1u : 0u);
    mma_commit(bar);
}

__global__ void __launch_bounds__(kThreads, 1)
dense_mla_kernel(Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars);
    Misc* misc = reinterpret_cast<Misc*>(smem + kOffMisc);
    float* red = reinterpret_cast<float*>(smem + kOffRed);
    float* neg_ref = reinterpret_cast<float*>(smem + kOffStat);   // minus the heads' references, log2 units
    float* l_acc = neg_ref + 64;
    float* alpha = l_acc + 64;
    float* neg_inf = alpha + 64;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const BatchDev& b = a.b;
    volatile int32_t* abort_flag = &misc->abort;
    volatile Row& w = reinterpret_cast<Row*>(smem + kOffRows)[warp];
    auto enter_row = [&](int row, int32_t* st) -> int {     // this warp's row; returns its tiles
        const Row r = row_view(a.b, a.view, row, st);
        __syncwarp();
        if ((tid & 31) == 0) {
            w.r = r.r;
            w.sink_end = r.sink_end;
            w.first = r.first;
            w.end = r.end;
            w.prefix = r.prefix;
            w.mask = r.mask;
            w.sink_pages = r.sink_pages;
            w.first_page = r.first_page;
            w.pages = r.pages;
        }
        __syncwarp();
        return tiles_of(r);
    };

    if (tid == 0) {
        mbar_init(&bars[B_QFULL], kWorkWarps);
        for (int i = 0; i < 5; ++i) mbar_init(&bars[B_FULL0 + i], kWorkWarps);
        mbar_init(&bars[B_SFULL], 1);
        mbar_init(&bars[B_PREADY], kWorkWarps);
        for (int i = 0; i < 4; ++i) mbar_init(&bars[B_PV0 + i], 1);
        mbar_init(&bars[B_DRAIN], 1);
        misc->abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&misc->tmem_base, 512);
        tmem_relinquish();
    }
    pdl_wait();
    if (tid < kWorkThreads) plan_share(a, misc, tid);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc->tmem_base;
    const int64_t g = blockIdx.x;
    const int64_t N = misc->total, G = min((int64_t)gridDim.x, N);
    const int row_begin = misc->row0;
    const int tile_begin = misc->tile0;
    const int n_mine = g < G ? (int)((g + 1) * N / G - g * N / G) : 0;   // the host bounds it
    if (tid == 0) a.meta[g] = n_mine > 0 ? Meta{row_begin, tile_begin > 0 ? 1 : 0} : Meta{-1, 0};

    auto timeout = [&](int where) {
        record_error(a.st, DSA_DEVERR_TIMEOUT, where);
        *abort_flag = 1;
    };

    if (warp >= kMmaWarp) {
        // ================================================================ MMA issue (one thread)
        fewer_registers<kMmaRegs>();
        if (warp == kMmaWarp && lane == 0) {
            const uint32_t kv0 = smem_addr(smem + kOffKV), q0 = smem_addr(smem + kOffQ), p0 = smem_addr(smem + kOffP);
            const uint64_t d_kv = desc_kmajor_sw128(kv0), d_q = desc_kmajor_sw128(q0);
            const uint64_t d_v = desc_mnmajor_sw128(kv0, kBlk), d_p = desc_mnmajor_sw128(p0, 8192);
            bool ok = true;
            int gt = 0, left = n_mine;
            int t0 = tile_begin;
            int k = 0;
            for (int row = row_begin; left > 0 && ok; ++row) {
                const int n_row = tiles_of(row_view(b, a.view, row, nullptr)) - t0;
                const int n = min(n_row, left);
                left -= n;
                t0 = 0;
                if (n == 0) continue;
                if (!(ok = wait_ab(&bars[B_QFULL], (uint32_t)(k & 1), abort_flag))) break;
                ++k;
                for (int t = 0; t < n && ok; ++t, ++gt) {
                    const uint32_t ph = (uint32_t)(gt & 1);
                    if (!(ok = wait_ab(&bars[B_FULL0], ph, abort_flag))) break;
                    tc_fence_after();
                    qk_blocks<0, 2>(tmem + kColS, d_kv, d_q);
                    if (!(ok = wait_ab(&bars[B_FULL0 + 1], ph, abort_flag))) break;
                    tc_fence_after();
                    qk_blocks<2, 2>(tmem + kColS, d_kv, d_q);
                    if (!(ok = wait_ab(&bars[B_FULL0 + 2], ph, abort_flag))) break;
                    tc_fence_after();
                    qk_blocks<4, 2>(tmem + kColS, d_kv, d_q);
                    if (!(ok = wait_ab(&bars[B_FULL0 + 3], ph, abort_flag))) break;
                    tc_fence_after();
                    qk_blocks<6, 2>(tmem + kColS, d_kv, d_q);
                    if (!(ok = wait_ab(&bars[B_FULL4], ph, abort_flag))) break;
                    tc_fence_after();
                    qk_blocks<8, 1>(tmem + kColS, d_kv, d_q);
                    mma_commit(&bars[B_SFULL]);
                    if (!(ok = wait_ab(&bars[B_PREADY], ph, abort_flag))) break;
                    tc_fence_after();
                    pv_block<0>(tmem + kColO, d_v, d_p, t > 0, &bars[B_PV0]);
                    pv_block<1>(tmem + kColO, d_v, d_p, t > 0, &bars[B_PV0 + 1]);
                    pv_block<2>(tmem + kColO, d_v, d_p, t > 0, &bars[B_PV0 + 2]);
                    pv_block<3>(tmem + kColO, d_v, d_p, t > 0, &bars[B_PV0 + 3]);
                }
            }
            if (!ok) timeout(61);
            if (n_mine > 0) {                              // no MMA may be in flight when the TMEM is released
                mma_commit(&bars[B_DRAIN]);
                mbar_wait(&bars[B_DRAIN], 0, 500000000ull);
            }
        }
        __syncwarp();
    } else if (n_mine > 0) {
        // ================================================================ workers
        more_registers<kWorkRegs>();
        // ---- softmax: warp w reads TMEM lane quarter w % 4 (token / latent row st) and
        // heads [16 hh, 16 hh + 16), hh = w / 4
        const int q4 = warp & 3, hh = warp >> 2;
        const int st = q4 * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
        // ---- rows of a tile: the quarters of a page's tokens fetch that page, 8 tokens a
        // warp in two steps.  Eight consecutive lanes hold four 16-byte pieces of two tokens
        // whose numbers differ in bits 0 and 2, so that their swizzled 16-byte stores fall
        // into 32 different banks.  The lane's token of step 1 is that of step 0 with bit 2
        // flipped: in a tile block's address that flips bit 9 and, through the swizzle, bit 6.
        const int half = q4 >> 1;
        const int par = lane >> 2 & 1;
        const int tok0 = ((warp >> 2) * 2 + (warp & 1)) * 8 + par * 5 + (lane >> 4) * 2;
        const int c8 = (lane & 3) | (lane >> 3 & 1) << 2;  // 16-byte piece of a 128-byte group
        constexpr uint32_t kFlip = 512 + 64;
        const uint32_t row_at = (uint32_t)(half * kPage + tok0) * 128;
        const uint32_t put_at = smem_addr(smem + kOffKV) + (c8 >> 2) * kBlk + row_at + (((2 * (c8 & 3)) ^ (tok0 & 7)) << 4);
        const uint32_t rope_at = smem_addr(smem + kOffP) + row_at + ((c8 ^ (tok0 & 7)) << 4);
        const uint32_t p_at = smem_addr(smem + kOffP) + st * 128 + (((2 * hh) ^ (st & 7)) << 4);   // P^T row st, heads 16 hh ..

        int row = row_begin, t = tile_begin, left = n_mine, gt = 0;
        int t_end = 0;                                     // end of the row's piece
        bool ok = true;
        uint4 raw[2][kSteps], rope[kSteps], scv[kSteps];   // rows in flight: two latent groups, RoPE dims, scales
        // A tile as this warp fetches it: the lane's rows of step 0 and 1 in its half's page.
        // A token that is not seen takes a row of the page that is (its probability is 0, and
        // the product needs a finite latent); a page without any gives zeros (row0 = NULL).
        struct Aim {
            const uint8_t *row0, *row1;
        };
        Aim now = {}, next = {};                           // the tile in flight, and the one after it
        bool valid_now = false, valid_next = false;        // softmax: is this lane's token of those tiles seen
        int32_t pg = -1, pg1 = -1;                         // pages of the tile to aim at next and the one after
        // page id of this warp's half of tile x, -1 beyond the piece
        auto page_of = [&](int x) -> int32_t {
            const int u = 2 * x + half;
            if (x >= t_end || u >= w.pages) return -1;
            const int lp = w.page(u);
            return lp < b.max_pages ? __ldg(b.page_table + (int64_t)w.r * b.max_pages + lp) : -1;
        };
        auto aim = [&](int x) {                            // sets `next` to tile x
            const int u = 2 * x + half;
            uint64_t m = 0;
            if (u < w.pages) {
                const int lp = w.page(u);
                m = w.first <= lp * kPage && (lp + 1) * kPage <= w.end ? ~0ull : w.seen(lp);
            }
            if (m && (pg < 0 || pg >= b.num_pages)) {
                if (lane == 0 && (warp & ~2) == 0) record_error(a.st, DSA_DEVERR_PAGE_RANGE, pg);
                m = 0;
            }
            valid_next = m >> (st & 63) & 1u;
            next.row0 = next.row1 = nullptr;
            if (m) {
                const int some = __ffsll((long long)m) - 1;
                const uint8_t* page = a.kv + (int64_t)pg * kKvPageBytes + c8 * 16;
                next.row0 = page + ((m >> tok0 & 1u) ? tok0 : some) * kKvTokenBytes;
                next.row1 = page + ((m >> (tok0 ^ 4) & 1u) ? tok0 ^ 4 : some) * kKvTokenBytes;
            }
            pg = pg1;
            pg1 = page_of(x + 2);
            if ((warp & ~2) == 0 && lane == 0 && pg >= 0 && pg < b.num_pages)     // the page of the tile after
                prefetch_l2(a.kv + (int64_t)pg * kKvPageBytes, kKvPageBytes);
        };
        auto fetch = [&](uint4 (&dst)[kSteps], int at) {   // the 16 bytes at `at` + 16 c8 of the lane's rows
            if (now.row0 != nullptr) {
                dst[0] = ldg_pinned(reinterpret_cast<const uint4*>(now.row0 + at));
                dst[1] = ldg_pinned(reinterpret_cast<const uint4*>(now.row1 + at));
            } else {
                dst[0] = dst[1] = make_uint4(0, 0, 0, 0);
            }
        };
        auto fetch_scales = [&]() { fetch(scv, 512 - c8 * 16); };
        static_assert(kSteps == 2, "two rows a lane");
        // The fetched tile into shared memory, latent groups 0..3 (free once tile gt's P.V of
        // the group is done; `first`: nothing to wait for), then the RoPE block (free, as
        // P^T, with the last group).  The registers emptied take the group two ahead.
        auto put_tile = [&](int x, bool first) {
            const uint32_t ph = (uint32_t)(gt & 1);
            const bool more = x + 1 < t_end, zeros = now.row0 == nullptr;
            valid_now = valid_next;
            if (more) aim(x + 1);                          // while the first P.V runs
            uint32_t off_range = 0;                        // a latent scale or a RoPE value fp16 cannot hold
#pragma unroll
            for (int gg = 0; gg < 4; ++gg) {
                if (!first && ok) ok = wait_ab(&bars[B_PV0 + gg], ph, abort_flag);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const uint32_t scb = gg == 0 ? scv[i].x : gg == 1 ? scv[i].y : gg == 2 ? scv[i].z : scv[i].w;
                    off_range |= scb - 0x38000000u > 0x43000000u - 0x38000000u ? 1u : 0u;   // outside [2^-15, 2^7]
                    const __half2 sc2 = __float2half2_rn(__uint_as_float(scb));              // a power of two: exact
                    const uint4 v = raw[gg & 1][i];
                    // 16 FP8 dims 128 gg + 16 c8 .. -> K-block 2 gg + c8 / 4, 16-byte chunks 2 (c8 % 4), +1
                    const uint32_t at = (put_at ^ (i ? kFlip : 0u)) + 2 * gg * kBlk;
                    st_shared_v4(at, e4m3x2_scaled_h2(v.x & 0xffffu, sc2), e4m3x2_scaled_h2(v.x >> 16, sc2),
                                 e4m3x2_scaled_h2(v.y & 0xffffu, sc2), e4m3x2_scaled_h2(v.y >> 16, sc2));
                    st_shared_v4(at ^ 16, e4m3x2_scaled_h2(v.z & 0xffffu, sc2), e4m3x2_scaled_h2(v.z >> 16, sc2),
                                 e4m3x2_scaled_h2(v.w & 0xffffu, sc2), e4m3x2_scaled_h2(v.w >> 16, sc2));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_FULL0 + gg]);
                if (gg < 2) {
                    fetch(raw[gg], (gg + 2) * 128);
                } else if (more) {
                    if (gg == 2) now = next;
                    fetch(raw[gg - 2], (gg - 2) * 128);
                }
            }
            if (more) fetch_scales();
            uint32_t rope_max = 0;                         // two bf16 magnitudes, compared as integers
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const uint4 v = rope[i];
                rope_max = __vmaxu2(rope_max, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                       __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                st_shared_v4(rope_at ^ (i ? kFlip : 0u), bf16x2_to_h2_sat(v.x), bf16x2_to_h2_sat(v.y), bf16x2_to_h2_sat(v.z),
                             bf16x2_to_h2_sat(v.w));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_FULL4]);
            off_range |= (rope_max & 0xffffu) >= 0x4780u || rope_max >= 0x47800000u ? 1u : 0u;   // |r| >= 2^16
            if (off_range && !zeros) record_error(a.st, DSA_DEVERR_FP16_RANGE, lane);
            if (more) fetch(rope, 528);
        };
        // Fetches the first tile of the current piece and lays out the row's Q (fp16,
        // K-major, 128-byte swizzle): every S^T issued so far has completed, so Q is
        // free.  Returns the softmax scale in log2 units times 2^-kq of the row's Q.
        auto open_piece = [&]() -> float {
            pg = page_of(t);
            pg1 = page_of(t + 1);
            aim(t);
            now = next;
            fetch_scales();
            fetch(raw[0], 0);
            fetch(raw[1], 128);
            fetch(rope, 528);
            static_assert(64 * 72 == 9 * kWorkThreads, "nine 16-byte pieces of q per thread");
            const uint4* qrow = reinterpret_cast<const uint4*>(a.q + (int64_t)row * (64 * 576));
            uint32_t mx = 0;                               // two bf16 magnitudes, compared as integers
#pragma unroll 1
            for (int u0 = 0; u0 < 9; u0 += 3) {
                uint4 qv[3];
#pragma unroll
                for (int u = 0; u < 3; ++u) qv[u] = __ldg(qrow + tid + (u0 + u) * kWorkThreads);
#pragma unroll
                for (int u = 0; u < 3; ++u)
                    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(qv[u].x & 0x7fff7fffu, qv[u].y & 0x7fff7fffu),
                                               __vmaxu2(qv[u].z & 0x7fff7fffu, qv[u].w & 0x7fff7fffu)));
            }
            mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
            if (lane == 0) misc->qmax[warp] = mx;
            work_sync();
            mx = __reduce_max_sync(0xffffffffu, misc->qmax[lane & (kWorkWarps - 1)]);
            const int eq = mx == 0 ? 14 : (int)(mx >> 7) - 127;
            const int kq = min(126, max(-126, 14 - eq));
            const float sc = __int_as_float((127 + kq) << 23);
#pragma unroll 1
            for (int u0 = 0; u0 < 9; u0 += 3) {
                uint4 qv[3];
#pragma unroll
                for (int u = 0; u < 3; ++u) qv[u] = __ldg(qrow + tid + (u0 + u) * kWorkThreads);
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                    const int c = tid + (u0 + u) * kWorkThreads;
                    const int h = c / 72, cq = c % 72;
                    const int blk = cq >> 3, ch = cq & 7;
                    *reinterpret_cast<uint4*>(smem + kOffQ + blk * 8192 + h * 128 + ((ch ^ (h & 7)) * 16)) =
                        make_uint4(bf16x2_scaled_to_h2(qv[u].x, sc), bf16x2_scaled_to_h2(qv[u].y, sc),
                                   bf16x2_scaled_to_h2(qv[u].z, sc), bf16x2_scaled_to_h2(qv[u].w, sc));
                }
            }
            if (tid == 0 && mx >= 0x7f80u) record_error(a.st, DSA_DEVERR_FP16_RANGE, row);   // inf / NaN in q
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_QFULL]);
            return a.scale_log2 * __int_as_float((127 - kq) << 23);
        };

        float lsum[kHeads];                                // this token lane's running sums of its heads
#pragma unroll
        for (int c = 0; c < kHeads; ++c) lsum[c] = 0.f;
        if (tid < 16) neg_inf[tid] = -INFINITY;
        if (tid < 64) neg_ref[tid] = kNoRef;               // seen by all behind open_piece's barrier
        float sl2 = 0.f;
        bool fresh = true;                                 // the next softmax is its piece's first
        int k = 0;                                         // pieces opened
        for (;;) {
            bool ended = false;
            if (k > 0) {
                // ---- softmax of tile t
                if (ok) ok = wait_ab(&bars[B_SFULL], (uint32_t)(gt & 1), abort_flag);
                // a token that is not seen takes -inf for its references: every P is 0
                const float4* nr4 = reinterpret_cast<const float4*>(valid_now ? neg_ref + hh * kHeads : neg_inf);
                uint32_t most;                              // largest P of the thread, as two fp16
                // S^T row of this token for the warp's heads
                auto load_s = [&](float (&v)[kHeads]) {
                    uint32_t x[kHeads];
                    tmem_ld_32x32b_x16(lane_addr + kColS + hh * kHeads, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int h = 0; h < kHeads; ++h) v[h] = __uint_as_float(x[h]);
                };
                // P of the current references, and its P^T row (heads 16 hh.. as fp16, MN-major swizzle)
                auto write_p = [&](float (&v)[kHeads]) {
#pragma unroll
                    for (int c4 = 0; c4 < kHeads / 4; ++c4) {
                        const float4 m = nr4[c4];
                        v[4 * c4] = ex2_approx(fmaf(v[4 * c4], sl2, m.x));
                        v[4 * c4 + 1] = ex2_approx(fmaf(v[4 * c4 + 1], sl2, m.y));
                        v[4 * c4 + 2] = ex2_approx(fmaf(v[4 * c4 + 2], sl2, m.z));
                        v[4 * c4 + 3] = ex2_approx(fmaf(v[4 * c4 + 3], sl2, m.w));
                    }
                    uint32_t h[kHeads / 2];
#pragma unroll
                    for (int c = 0; c < kHeads / 2; ++c) h[c] = pack_h2(v[2 * c], v[2 * c + 1]);
                    st_shared_v4(p_at, h[0], h[1], h[2], h[3]);
                    st_shared_v4(p_at ^ 16, h[4], h[5], h[6], h[7]);
                    most = __vmaxu2(__vmaxu2(__vmaxu2(h[0], h[1]), __vmaxu2(h[2], h[3])),
                                    __vmaxu2(__vmaxu2(h[4], h[5]), __vmaxu2(h[6], h[7])));
                    fence_proxy_async_smem();
                };
                float v[kHeads];
                tc_fence_after();
                load_s(v);
                write_p(v);
                // ---- a score above its head's reference by more than 2^kTau (P above 2^(kTau + kShift))
                //      makes every warp take new references (always on the piece's first tile)
                const bool over = (most & 0xffffu) > kPMaxH || most >> 16 > kPMaxH;
                if (work_any(over || !ok)) {
                    if (work_any(!ok)) {
                        if (tid == 0) timeout(63);
                        break;
                    }
                    load_s(v);
#pragma unroll
                    for (int c = 0; c < kHeads; ++c) v[c] = valid_now ? v[c] * sl2 : -INFINITY;
                    xreduce16<true>(v, lane);                   // per-head tile max (consumes v)
                    if (lane < kHeads) red[q4 * 64 + hh * kHeads + lane] = v[0];
                    work_sync();
                    if (tid < 64) {
                        const float tm = fmaxf(fmaxf(red[tid], red[64 + tid]), fmaxf(red[128 + tid], red[192 + tid])) - kShift;
                        const float mo = -neg_ref[tid];
                        const bool need = tm > mo + kTau;
                        alpha[tid] = need ? exp2f(mo - tm) : 1.f;          // 0 for a first reference
                        if (need) neg_ref[tid] = -tm;
                    }
                    work_sync();
                    bool mine = false;                          // does a head of this warp have a new reference
#pragma unroll
                    for (int c = 0; c < kHeads; ++c) mine |= alpha[hh * kHeads + c] != 1.f;
                    if (mine) {
                        if (!fresh) {                           // rescale the resident O^T columns of these heads
#pragma unroll 1
                            for (int mb = 0; mb < 4; ++mb) {
                                uint32_t o[kHeads];
                                const uint32_t addr = lane_addr + kColO + mb * 64 + hh * kHeads;
                                tmem_ld_32x32b_x16(addr, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < kHeads; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[hh * kHeads + c]);
                                tmem_st_32x32b_x16(addr, o);
                            }
                            tmem_st_wait();
                        }
#pragma unroll
                        for (int c = 0; c < kHeads; ++c) lsum[c] *= alpha[hh * kHeads + c];
                    }
                    load_s(v);
                    write_p(v);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_PREADY]);    // P^T written, S^T read, O^T rescaled
#pragma unroll
                for (int c = 0; c < kHeads; ++c) lsum[c] += v[c];
                fresh = false;
                --left;
                ended = ++t == t_end;
            }
            // ---- the piece's sums; the next row
            int done = row;
            bool whole = false;
            float sl2_next = sl2;
            if (ended) {
                xreduce16<false>(lsum, lane);
                if (lane < kHeads) red[256 + q4 * 64 + hh * kHeads + lane] = lsum[0];
                whole = (k > 1 || tile_begin == 0) && w.pages <= 2 * t_end;
                __syncwarp();
            }
            if (left > 0 && (ended || k == 0)) {
                if (ended) {
                    ++row;
                    t = 0;
                }
                t_end = enter_row(row, tid == 0 ? a.st : nullptr);
                t_end = min(t_end, t + left);
                sl2_next = open_piece();
                ++k;
            }
            // ---- the next tile
            if (left > 0) put_tile(t, k == 1 && fresh);
            if (k == 1 && fresh) {
                sl2 = sl2_next;
                continue;
            }
            if (ended) {
                // ---- the piece's output
                if (ok) ok = wait_ab(&bars[B_PV3], (uint32_t)(gt & 1), abort_flag);   // O^T is final
                if (work_any(!ok)) {
                    if (tid == 0) timeout(64);
                    break;
                }
                tc_fence_after();
                if (tid < 64) l_acc[tid] = red[256 + tid] + red[320 + tid] + red[384 + tid] + red[448 + tid];
                work_sync();
                const int64_t unit = 2 * (int64_t)blockIdx.x + (done == row_begin ? 0 : 1);   // a share's first piece, or its last
#pragma unroll 1
                for (int mb = 0; mb < 4; ++mb) {
                    uint32_t o[kHeads];
                    tmem_ld_32x32b_x16(lane_addr + kColO + mb * 64 + hh * kHeads, o);
                    tmem_ld_wait();
                    const int d = mb * 128 + st;                           // latent dim of this TMEM lane
#pragma unroll
                    for (int c = 0; c < kHeads; ++c) {                     // a warp stores 32 consecutive dims
                        const int h = hh * kHeads + c;
                        const float ov = __uint_as_float(o[c]);
                        if (whole) {
                            const float l = l_acc[h];
                            const float val = l > 0.f ? ov / l : 0.f;
                            const int64_t oi = ((int64_t)done * 64 + h) * 512 + d;
                            if (a.out_f32) static_cast<float*>(a.out)[oi] = val;
                            else static_cast<__nv_bfloat16*>(a.out)[oi] = __float2bfloat16_rn(val);
                        } else {
                            a.part_o[(unit * 64 + h) * 512 + d] = ov;
                        }
                    }
                }
                tc_fence_before();
                if (tid < 64) {
                    const float l = l_acc[tid];
                    if (!whole) a.part_ml[unit * 64 + tid] = make_float2(-neg_ref[tid], l);
                    else if (a.lse) a.lse[(int64_t)done * 64 + tid] = l > 0.f ? (log2f(l) - neg_ref[tid]) * 0.69314718055994531f : -INFINITY;
                    neg_ref[tid] = kNoRef;
                }
                if (left == 0) break;
                sl2 = sl2_next;
                fresh = true;
#pragma unroll
                for (int c = 0; c < kHeads; ++c) lsum[c] = 0.f;
                work_sync();                                // O^T and the references may be reused
            }
            ++gt;
        }
    }
    tc_fence_before();
    __syncthreads();
    pdl_trigger();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- merge
// Block (x, y): share boundary x + 1 and its heads y, y + gridDim.y, ..  The
// boundary's row was cut when share x + 1 begins inside it; the first such
// boundary of a row merges its pieces.  Per head over the pieces u:
//   M = max m_u,  w_u = 2^(m_u - M),  L = sum w_u l_u,
//   out = sum_u w_u O_u / L,  lse = (M + log2 L) ln 2.
constexpr int kMergeThreads = 128;                         // 512 dims, four per thread
constexpr int kMaxPieces = 1024;

__global__ void __launch_bounds__(kMergeThreads)
dense_merge_kernel(Args a, int G) {
    __shared__ float w_s[kMaxPieces];
    __shared__ float red_s[8];
    __shared__ int np_s;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bd = blockIdx.x + 1;
    const Meta me = a.meta[bd], prev = a.meta[bd - 1];
    if (!me.inside || (prev.inside && prev.row == me.row)) return;
    const int64_t row = me.row;
    // the row's pieces: the last piece of share bd - 1, then the first ones of bd, bd + 1, .. while they begin inside the row
    if (tid == 0) np_s = 1 + G - bd;
    __syncthreads();
    for (int i = tid; bd + i < G; i += kMergeThreads) {
        const Meta m = a.meta[bd + i];
        if (!m.inside || m.row != me.row) {
            atomicMin(&np_s, 1 + i);
            break;
        }
    }
    __syncthreads();
    const int np = np_s;
    const int64_t unit0 = 2 * (int64_t)(bd - 1) + (prev.row == me.row ? 0 : 1);
    for (int h = blockIdx.y; h < 64; h += gridDim.y) {
        auto unit = [&](int i) { return i == 0 ? unit0 : 2 * (int64_t)(bd - 1 + i); };
        float M = -INFINITY;
        for (int i = tid; i < np; i += kMergeThreads) {
            const float2 ml = __ldcg(a.part_ml + unit(i) * 64 + h);
            if (ml.y > 0.f) M = fmaxf(M, ml.x);
        }
        M = warp_max(M);
        if (lane == 0) red_s[warp] = M;
        __syncthreads();
        M = fmaxf(fmaxf(red_s[0], red_s[1]), fmaxf(red_s[2], red_s[3]));
        float L = 0.f;
        for (int i = tid; i < np; i += kMergeThreads) {
            const float2 ml = __ldcg(a.part_ml + unit(i) * 64 + h);
            const float w = ml.y > 0.f ? exp2f(ml.x - M) : 0.f;
            w_s[i] = w;
            L += w * ml.y;
        }
        L = warp_sum(L);
        if (lane == 0) red_s[4 + warp] = L;
        __syncthreads();
        L = red_s[4] + red_s[5] + red_s[6] + red_s[7];
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q0 = 0; q0 < np; q0 += 8) {                // eight pieces' loads in flight
            float4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = q0 + j < np ? __ldcg(reinterpret_cast<const float4*>(a.part_o + (unit(q0 + j) * 64 + h) * 512) + tid)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = q0 + j < np ? w_s[q0 + j] : 0.f;
                if (w == 0.f) continue;                    // a piece that saw nothing holds no numbers
                acc.x += w * v[j].x;
                acc.y += w * v[j].y;
                acc.z += w * v[j].z;
                acc.w += w * v[j].w;
            }
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int64_t o = (row * 64 + h) * 512 + tid * 4;
        if (a.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        } else {
            __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
            __nv_bfloat162 hi2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + o) =
                make_uint2(*reinterpret_cast<uint32_t*>(&lo2), *reinterpret_cast<uint32_t*>(&hi2));
        }
        if (a.lse && tid == 0) a.lse[row * 64 + h] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
        __syncthreads();                                    // w_s and red_s may be reused
    }
}

static size_t ws_bytes(int G) {
    const size_t n = (size_t)2 * G * 64 * (512 + 2) * 4 + (size_t)G * sizeof(Meta);
    return (n + 255) / 256 * 256;
}

// Tiles that one row can have, at most.
static int64_t most_tiles(const dsa_batch* b, const View& v) {
    int64_t pages = ((int64_t)b->max_seq_len + kPage - 1) / kPage;
    if (!v.tree) pages = std::min(pages, (int64_t)v.sinks / kPage + 1 + (int64_t)v.window / kPage + 2);
    return (pages + 1) / 2;
}

static dsa_status launch(const void* q, const uint8_t* kv, const dsa_batch* b, View view, float softmax_scale, void* out,
                         int32_t out_dtype, float* lse, void* ws, size_t bytes, int32_t* st, void* stream) {
    if (out_dtype != DSA_DTYPE_BF16 && out_dtype != DSA_DTYPE_F32) return DSA_ERR_INVALID_ARGUMENT;
    if (!(softmax_scale > 0.f) || softmax_scale > 3.0e38f) return DSA_ERR_INVALID_ARGUMENT;
    if (b->num_pages * DSA_PAGE_TOKENS > 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;        // int32 cache slots
    if (b->total_q == 0) return DSA_OK;
    if (!q || !kv || !out) return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(q) || !aligned16(kv) || !aligned16(out)) return DSA_ERR_ALIGNMENT;
    if (b->total_q * most_tiles(b, view) / device_sm_count() > 0x7ffffff0LL) return DSA_ERR_UNSUPPORTED;   // 32-bit tile counts of a share
    if (!ws) return DSA_ERR_INVALID_ARGUMENT;
    if (bytes < ws_bytes(device_sm_count())) return DSA_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(ws)) return DSA_ERR_ALIGNMENT;
    if (ensure_smem_limit(reinterpret_cast<const void*>(&dense_mla_kernel), kSmemAlloc) != DSA_OK) return DSA_ERR_CUDA;
    const int sms = device_sm_count();
    const int G = (int)std::min<int64_t>(sms, b->total_q * most_tiles(b, view));
    Args a = {};
    a.q = static_cast<const uint16_t*>(q);
    a.kv = kv;
    a.b = to_dev(b);
    a.view = view;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.out = out;
    a.out_f32 = out_dtype == DSA_DTYPE_F32;
    a.lse = lse;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)2 * sms * 64 * 512);
    a.meta = reinterpret_cast<Meta*>(a.part_ml + (size_t)2 * sms * 64);
    a.st = st;
    const cudaStream_t s = as_stream(stream);
    DSA_CHECK(launch_pdl(dense_mla_kernel, dim3((unsigned)G), dim3(kThreads), kSmemAlloc, s, 1, a));
    if (G > 1) {
        // boundaries x heads: a block per head where few rows can be cut (each may have many
        // pieces), four heads a block where many can (most blocks then have nothing to merge)
        const unsigned cuts = (unsigned)(G - 1);
        DSA_CHECK(launch_pdl(dense_merge_kernel, dim3(cuts, b->total_q < 32 ? 64 : 16), dim3(kMergeThreads), 0, s, 1, a, G));
    }
    return DSA_OK;
}

}  // namespace mld
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_dense_mla_workspace_size(const dsa_batch* b, size_t* bytes) {
    const dsa_status vs = validate_batch(b);
    if (vs != DSA_OK) return vs;
    if (!bytes) return DSA_ERR_INVALID_ARGUMENT;
    *bytes = mld::ws_bytes(device_sm_count());
    return DSA_OK;
}

extern "C" dsa_status dsa_window_mla(const void* q, const uint8_t* kv_cache, const dsa_batch* b, int32_t window,
                                     int32_t sinks, float softmax_scale, void* out, int32_t out_dtype, float* lse,
                                     void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
    const dsa_status vs = validate_batch(b);
    if (vs != DSA_OK) return vs;
    if (window < 1 || sinks < 0) return DSA_ERR_INVALID_ARGUMENT;
    return mld::launch(q, kv_cache, b, mld::View{nullptr, window, sinks}, softmax_scale, out, out_dtype, lse, ws, ws_bytes,
                       dev_status, stream);
}

extern "C" dsa_status dsa_tree_mla(const void* q, const uint64_t* tree_mask, const uint8_t* kv_cache, const dsa_batch* b,
                                   float softmax_scale, void* out, int32_t out_dtype, float* lse, void* ws,
                                   size_t ws_bytes, int32_t* dev_status, void* stream) {
    const dsa_status vs = validate_batch(b);
    if (vs != DSA_OK) return vs;
    if (b->max_q_len > 64) return DSA_ERR_UNSUPPORTED;
    if (b->total_q > 0 && !tree_mask) return DSA_ERR_INVALID_ARGUMENT;
    if (reinterpret_cast<uintptr_t>(tree_mask) & 7) return DSA_ERR_ALIGNMENT;
    return mld::launch(q, kv_cache, b, mld::View{tree_mask, 0, 0}, softmax_scale, out, out_dtype, lse, ws, ws_bytes,
                       dev_status, stream);
}
