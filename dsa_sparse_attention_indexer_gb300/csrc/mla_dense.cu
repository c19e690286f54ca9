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
// Warps 0-15 (workers) do what a tile's phases ask for one after the other:
//   softmax     a thread owns one token (TMEM lane) and 16 heads.  P is formed
//               against a reference per head that is renewed, and O^T rescaled,
//               only when a P passes 2^15, and once behind a piece's first tiles;
//   next tile   its rows, read into registers two groups ahead, are dequantised into the
//               128-byte-swizzled tile (exact for scales in [2^-15, 2^7]), each
//               part as soon as it is free.  Rows that are not seen become zeros or
//               another row, with probability 0;
//   next row    its Q, copied into its place as bf16 during the softmax, then scaled
//               by the power of two that puts its largest |q| in [2^14, 2^15), while
//               the last P.V runs; then the epilogue, while the first S^T of the
//               next row runs.
// Warp 16 issues the MMAs.  Warp 17 lays out the tiles of the CTA's share up to four
// ahead: pages, masks of what is seen, where a row's piece begins and ends; it also
// prefetches the pages into L2.
// Every wait is time-bounded; a timeout is recorded and the CTA winds down.
//
// What bounds it (64 tree rows in each of 8 requests of up to 32K tokens: 2.83 ms, 696
// TFLOP/s; 2048 rows with a window of 2048: 0.95 ms, 618 TFLOP/s; one row in each of 4
// requests with a window of 131072: 130 us, 2.7 TB/s): the workers.  A tile takes about
// 6,950 cycles, of which the tensor core is busy 2,180.  The workers issue 700
// instructions per warp and tile, mostly conversions and fp16 products of the
// dequantisation at half rate, and 4,300 passes through the load/store pipe (1,430 for
// shared stores, most of them the fp16 tile's, 1,900 for the rows' loads), one phase
// after the other.
// Neighbouring rows of a request read the same tiles, but two rows' O^T (2 x 256
// columns) leave no TMEM for S^T; two CTAs that dequantise half a tile each and copy
// it to one another move in step, and wait more than they save (2.94 -> 3.93 ms).
//
// One row of 512 tokens takes 16 us, all of it latency: the share 2, tile and page 1.5,
// Q 2, tile 1.5, S^T 0.5, softmax 1.5, P.V 1, the partial's 131 KB at 30 bytes a cycle 2.5,
// the merge 3.
#include <algorithm>
#include <type_traits>

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
    float scale;
    void* out;
    int out_f32;
    float* lse;
    float* part_o;              // [2 G, 16, 512, 4]: unnormalised outputs of cut rows, two pieces per share, four heads side by side
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
    __device__ __forceinline__ int page(int u) const { return u < sink_pages ? u : first_page + u - sink_pages; }
    // The positions of logical page lp that the row sees, one bit each.
    __device__ __forceinline__ uint64_t seen(int lp) const {
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
    // In a batch of equal query lengths the row's request is this one.  Its loads depend on
    // nothing and are one round trip; any other batch searches.
    w.r = min(b.batch - 1, (int)(((float)row + 0.5f) * (float)b.batch / (float)b.total_q));
    const int rows = b.q_start[b.batch];
    int qs = b.q_start[w.r], qe = b.q_start[w.r + 1], len = b.seq_len[w.r];
    const uint64_t bits = v.tree ? v.tree[row] : 0;
    if (row >= rows) {
        w.r = 0;
        return w;
    }
    if (row < qs || row >= qe) {
        w.r = row_request(b.q_start, b.batch, row);
        qs = b.q_start[w.r];
        qe = b.q_start[w.r + 1];
        len = b.seq_len[w.r];
    }
    const int qn = qe - qs;
    const int64_t room = (int64_t)b.max_pages * kPage;
    int L = len;
    if (L > room) {
        record_error(st, DSA_DEVERR_INDEX_RANGE, L);
        L = (int)room;
    }
    w.prefix = len - qn;
    w.pages = 1;
    if (L <= 0 || w.prefix < 0) return w;
    if (v.tree) {
        const int known = min(qn, 64);
        w.mask = bits & (known >= 64 ? ~0ull : (1ull << known) - 1);
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
    const int last_page = end / kPage + (end % kPage != 0);        // end + 63 may pass 2^31
    w.pages = max(1, w.sink_pages + max(0, last_page - w.first_page));
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
constexpr int kAimWarp = kMmaWarp + 1;
constexpr int kThreads = (kWorkWarps + 4) * 32;            // five warpgroups; the last one issues the MMAs and lays out the tiles
constexpr int kWorkBar = 1, kVoteBar = 2;                  // workers; workers and the MMA warp
constexpr int kAhead = 4;                                  // tiles laid out ahead
// P is held in fp16 against a reference per head, renewed when a P passes 2^kTau.  A first
// reference puts the largest P at 2^kFirst, which leaves a head room to grow.  Behind kSettle
// tiles of a piece, references move down to where the sum of the P so far is 2^kSettled, so
// that behind a dominating position the many small ones keep their bits: P is off by 2^-11 of
// itself or by 2^-25, which is 2^-28 of the sum in the first tiles and 2^-34 in all others:
// 4096 times 2^-28 and a million times 2^-34 are less than 2^-13 of the largest latent.
// (Settled after 8 tiles, prefill with 17 tiles a row takes 952 us instead of 917; with
// references that put every tile's largest P at 2^9, or its sum at 2^8, flat heads
// outgrow them tile after tile: 1077 and 993 us.)
constexpr float kTau = 15.0f, kFirst = 3.0f, kSettled = 9.0f;
constexpr int kSettle = 32;
constexpr uint32_t kPMaxH = 0x7800;                        // 2^kTau as fp16 bits
constexpr float kNoRef = INFINITY;                         // minus the reference of a head without one: P of any score is inf
constexpr uint32_t kIdescQK = idesc_f16_f32(128, 64, false, false);
constexpr uint32_t kIdescPV = idesc_f16_f32(128, 64, true, true);
constexpr uint32_t kColS = 0;                              // TMEM: S^T [128 x 64]
constexpr uint32_t kColO = 64;                             // TMEM: O^T 4 x [128 x 64]

constexpr int kOffKV = 0;                                  // 8 latent K-blocks and the RoPE block (later P^T), [128 tokens x 128 B]
constexpr int kOffP = kOffKV + 8 * kBlk;
constexpr int kOffQ = kOffKV + 9 * kBlk;                   // 9 K-blocks of [64 heads x 128 B]
constexpr int kOffRed = kOffQ + 9 * 8192;                  // [2][4 lane quarters][64 heads] fp32
constexpr int kOffStat = kOffRed + 2 * 4 * 64 * 4;         // neg_ref, l_acc, alpha [64], 32 times -inf
constexpr int kOffBars = kOffStat + (3 * 64 + 32) * 4;
constexpr int kOffMisc = kOffBars + 24 * 8;
constexpr int kSmemUsed = kOffMisc + 512;
constexpr int kSmemAlloc = kSmemUsed + 1024;
static_assert(kSmemAlloc <= 232448, "shared memory budget");
static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kBlk % 1024 == 0, "swizzle atoms need 1 KB alignment");
static_assert(kOffStat % 16 == 0, "reference maxima are read as float4");

enum { B_QFULL = 0, B_FULL0, B_FULL4 = B_FULL0 + 4, B_SFULL, B_PV0, B_PV3 = B_PV0 + 3, B_DRAIN, B_AIM0,
       B_FREE0 = B_AIM0 + kAhead, B_COUNT = B_FREE0 + kAhead };
static_assert(B_COUNT <= 24, "barrier block");

// A tile of the share, as the aim warp lays it out: its two pages, which of their
// positions the row sees, and where it stands in the row's piece.
struct Tile {
    uint64_t seen[2];
    int32_t page[2];            // -1: no position of the page is seen, or it is outside the cache
    uint32_t row;               // row << kRowShift | flags: FIRST, LAST tile of the piece; WHOLE: the piece is the whole row;
                                // SETTLE: its tile kSettle, LATE: that one or a later one
};
enum { T_FIRST = 1, T_LAST = 2, T_WHOLE = 4, T_SETTLE = 8, T_LATE = 16 };
constexpr int kRowShift = 5;

struct Misc {
    uint32_t tmem_base;
    int32_t abort;
    Tile tile[kAhead];          // by tile of the share, modulo kAhead
    uint32_t qmax[kWorkWarps];  // per warp: largest bf16 magnitude of the row's q
    int64_t scratch[kWorkWarps];
    int32_t mine, row0, tile0;  // tiles of this CTA's share, and where it begins
};
static_assert(sizeof(Misc) <= 512, "misc block");

// Where a CTA's share begins, for the merge: its first row (-1: no share) and
// whether that row began in an earlier share.
struct Meta {
    int32_t row;
    int32_t inside;
};

// Has any worker, or the MMA warp, `pred` set?  (All of them call it.)
__device__ __forceinline__ bool vote(bool pred) { return bar_any<kVoteBar, kWorkThreads + 32>(pred); }
__device__ __forceinline__ void work_sync() { bar_sync<kWorkBar, kWorkThreads>(); }

__device__ __forceinline__ int tiles_of(const Row& w) { return (w.pages + 1) >> 1; }

// Counts the tiles of all rows (the workers' threads, consecutive rows each) and
// finds this CTA's share of them.
__device__ __noinline__ void plan_share(const Args& a, Misc* misc, int tid) {
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
    int64_t* tot = misc->scratch;                                 // one per warp
    if ((tid & 31) == 31) tot[tid >> 5] = x;
    work_sync();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kWorkThreads / 32; ++w) {
        if (w < (tid >> 5)) before += tot[w];
        all += tot[w];
    }
    before += x - mine;
    // shares of n or n + 1 tiles, the longer ones first
    const int64_t n = all >> 32 ? all / gridDim.x : (uint32_t)all / gridDim.x;
    const int64_t longer = all - n * gridDim.x, g = blockIdx.x;
    if (tid == 0) misc->mine = (int32_t)n + (g < longer);  // the host bounds it
    int64_t at = g * n + min(g, longer);
    if (at >= before && at < before + mine) {
        at -= before;
        int64_t r = r0;
        for (; r + 1 < r1; ++r) {
            const int t = tiles_of(row_view(a.b, a.view, r, nullptr));
            if (at < t) break;
            at -= t;
        }
        misc->row0 = (int32_t)r;
        misc->tile0 = (int32_t)at;
    }
}

// Registers per thread: 96 at launch (65,536 / 640 threads, in eights), of which
// the last warpgroup gives some to the workers: 512 x 112 + 128 x 32 = 640 x 96.
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
dense_mla_kernel(const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars);
    Misc* misc = reinterpret_cast<Misc*>(smem + kOffMisc);
    float* red = reinterpret_cast<float*>(smem + kOffRed);
    float* neg_ref = reinterpret_cast<float*>(smem + kOffStat);   // minus the heads' references, scores of the scaled Q
    float* l_acc = neg_ref + 64;
    float* alpha = l_acc + 64;
    float* neg_inf = alpha + 64;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const BatchDev& b = a.b;
    volatile int32_t* abort_flag = &misc->abort;

    if (tid == 0) {
        mbar_init(&bars[B_QFULL], kWorkWarps);
        for (int i = 0; i < 5; ++i) mbar_init(&bars[B_FULL0 + i], kWorkWarps);
        mbar_init(&bars[B_SFULL], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&bars[B_PV0 + i], 1);
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(&bars[B_AIM0 + i], 1);
            mbar_init(&bars[B_FREE0 + i], kWorkWarps + 1);
        }
        mbar_init(&bars[B_DRAIN], 1);
        misc->abort = 0;
        // what a worker finds whose wait for a tile ran out: pages of the cache or none, at any time
        for (int i = 0; i < kAhead; ++i) misc->tile[i] = Tile{{0, 0}, {-1, -1}, 0};
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&misc->tmem_base, 512);
        tmem_relinquish();
    }
    uint32_t tmem = 0;
    int row_begin = 0, tile_begin = 0, n_mine = 0;         // this CTA's share
    auto share = [&]() {                                   // every thread, the workers behind plan_share
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        tmem = misc->tmem_base;
        row_begin = misc->row0;
        tile_begin = misc->tile0;
        n_mine = misc->mine;
        if (tid == 0) a.meta[blockIdx.x] = n_mine > 0 ? Meta{row_begin, tile_begin > 0 ? 1 : 0} : Meta{-1, 0};
    };
    auto start_worker = [&]() {
        more_registers<kWorkRegs>();
        pdl_wait();
        plan_share(a, misc, tid);
        share();
        return n_mine > 0;
    };
    auto timeout = [&](int where) {
        record_error(a.st, DSA_DEVERR_TIMEOUT, where);
        *abort_flag = 1;
    };
    auto wait = [&](int bar, uint32_t parity) { return wait_ab(&bars[bar], parity, abort_flag, b.wait_ns); };

    if (warp >= kMmaWarp) {
        fewer_registers<kMmaRegs>();
        pdl_wait();
        share();
        if (warp == kMmaWarp && n_mine > 0) {
            // ============================================================ MMA issue (lane 0; the warp joins the votes)
            const uint32_t kv0 = smem_addr(smem + kOffKV), q0 = smem_addr(smem + kOffQ), p0 = smem_addr(smem + kOffP);
            const uint64_t d_kv = desc_kmajor_sw128(kv0), d_q = desc_kmajor_sw128(q0);
            const uint64_t d_v = desc_mnmajor_sw128(kv0, kBlk), d_p = desc_mnmajor_sw128(p0, 8192);
            bool ok = true;                                // of lane 0
            int k = 0;                                     // rows' Qs so far
            for (int n = 0; n < n_mine; ++n) {
                const uint32_t ph = (uint32_t)(n & 1);
                bool first = false;
                if (lane == 0) {
                    ok = ok && wait(B_AIM0 + n % kAhead, (uint32_t)(n / kAhead & 1));
                    if (ok) first = reinterpret_cast<volatile Tile*>(misc->tile)[n % kAhead].row & T_FIRST;
                    mbar_arrive(&bars[B_FREE0 + n % kAhead]);
                    if (ok && first) ok = wait(B_QFULL, (uint32_t)(k++ & 1));
                    auto next = [&](int bar) {
                        ok = ok && wait(bar, ph);
                        tc_fence_after();
                        return ok;
                    };
                    if (next(B_FULL0)) qk_blocks<0, 2>(tmem + kColS, d_kv, d_q);
                    if (next(B_FULL0 + 1)) qk_blocks<2, 2>(tmem + kColS, d_kv, d_q);
                    if (next(B_FULL0 + 2)) qk_blocks<4, 2>(tmem + kColS, d_kv, d_q);
                    if (next(B_FULL0 + 3)) qk_blocks<6, 2>(tmem + kColS, d_kv, d_q);
                    if (next(B_FULL4)) {
                        qk_blocks<8, 1>(tmem + kColS, d_kv, d_q);
                        mma_commit(&bars[B_SFULL]);
                    }
                }
                __syncwarp();
                if (vote(!ok)) {                           // P^T is written; or new references, or a timeout
                    if (vote(!ok)) break;
                    vote(false);                           // P^T is written again, O^T rescaled
                }
                if (lane == 0) {
                    tc_fence_after();
                    pv_block<0>(tmem + kColO, d_v, d_p, !first, &bars[B_PV0]);
                    pv_block<1>(tmem + kColO, d_v, d_p, !first, &bars[B_PV0 + 1]);
                    pv_block<2>(tmem + kColO, d_v, d_p, !first, &bars[B_PV0 + 2]);
                    pv_block<3>(tmem + kColO, d_v, d_p, !first, &bars[B_PV0 + 3]);
                }
                __syncwarp();
            }
            if (lane == 0) {
                if (!ok) timeout(61);
                mma_commit(&bars[B_DRAIN]);                // no MMA may be in flight when the TMEM is released
                mbar_wait(&bars[B_DRAIN], 0, 500000000ull);
            }
        } else if (warp == kAimWarp && n_mine > 0) {
            // ============================================================ tiles of the share, one after the other
            bool ok = true;
            int row = row_begin, t = tile_begin;
            Row w = row_view(b, a.view, row, lane == 0 ? a.st : nullptr);
            bool cut = t > 0;                              // the row began in an earlier share
            int at = 0;                                    // of the piece's tiles
            for (int n = 0; n < n_mine; ++n) {
                // until the workers and the MMA warp have read the slot's last tile (a phase that
                // counts as over the first time round)
                ok = __all_sync(0xffffffffu, wait(B_FREE0 + n % kAhead, (uint32_t)(n / kAhead + 1 & 1)));
                if (!ok) break;
                Tile* tile = &misc->tile[n % kAhead];
                const int u = 2 * t + lane;
                const bool end_of_row = t + 1 == tiles_of(w);
                if (lane < 2) {                            // page u of the row
                    const int lp = w.page(u);
                    uint64_t m = u < w.pages ? w.seen(lp) : 0ull;
                    int32_t page = -1;
                    if (m) {
                        const int64_t pg = lp < b.max_pages ? b.page_table[(int64_t)w.r * b.max_pages + lp] : -1;
                        if (pg >= 0 && pg < b.num_pages) {
                            page = (int32_t)pg;
                            prefetch_l2(a.kv + pg * kKvPageBytes, kKvPageBytes);
                        } else {
                            record_error(a.st, DSA_DEVERR_PAGE_RANGE, pg);
                            m = 0;
                        }
                    }
                    tile->page[lane] = page;
                    tile->seen[lane] = m;
                }
                if (lane == 0) {
                    const bool last = end_of_row || n + 1 == n_mine;
                    tile->row = (uint32_t)row << kRowShift | (at == 0 ? T_FIRST : 0) | (last ? T_LAST : 0) |
                                (last && end_of_row && !cut ? T_WHOLE : 0) | (at == kSettle ? T_SETTLE : 0) | (at >= kSettle ? T_LATE : 0);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_AIM0 + n % kAhead]);
                at = end_of_row ? 0 : at + 1;
                ++t;
                if (end_of_row && n + 1 < n_mine) {
                    ++row;
                    t = 0;
                    cut = false;
                    w = row_view(b, a.view, row, lane == 0 ? a.st : nullptr);
                }
            }
            if (!ok && lane == 0) timeout(65);
        }
        __syncwarp();
    } else if (start_worker()) {
        // ================================================================ workers
        // ---- softmax: warp w reads TMEM lane quarter w % 4 (token / latent row st) and
        // heads [16 hh, 16 hh + 16), hh = w / 4
        const int q4 = warp & 3, hh = warp >> 2;
        const int st = q4 * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t p_at = smem_addr(smem + kOffP) + st * 128 + (((2 * hh) ^ (st & 7)) << 4);   // P^T row st, heads 16 hh ..
        // ---- rows of a tile: a warp takes four tokens of each page, a lane token tok of
        // both.  Eight consecutive lanes hold the 128 bytes of a token's group, which begin
        // anywhere and so lie in one or two lines; halves of two tokens would lie in three
        // or four (14 passes a load against 10: 91.9 -> 89.2 us for 64 windows of 4096).
        // 16 FP8 dims make two 16-byte chunks; where the group's second K-block has them in
        // turn, the eight lanes' stores fall into 32 different banks.
        const int tok = warp * 4 + (lane >> 3), c8 = lane & 7;   // c8: 16-byte piece of the group
        const uint32_t put = smem_addr(smem + kOffKV) + (c8 >> 2) * kBlk + tok * 128 + (((2 * (c8 & 3) + (c8 >> 2)) ^ (tok & 7)) << 4);
        const uint32_t putx = put ^ 16;
        const uint32_t put_rope = smem_addr(smem + kOffP) + tok * 128 + ((c8 ^ (tok & 7)) << 4);

        bool ok = true;
        int n = 0;                                         // the tile whose softmax comes next
        uint32_t row = 0, row_next = 0;                    // row and flags of tile n and the one after it
        bool valid = false, valid_next = false;            // softmax: is the lane's token of those tiles seen
        uint4 raw[2][2] = {}, rope[2] = {}, scv[2] = {};   // rows of the tile after tile n in flight: two latent groups, RoPE dims, scales
        // Where the rows are, one per page.  A token that is not seen takes a row of its page
        // that is (its probability is 0, and the product needs a finite latent); a page without
        // any gives zeros (NULL, slot -1).
        const uint8_t* src[2] = {};                        // of the tile in flight
        int32_t slot_next[2] = {};                         // of the one after it, as cache slots
        auto aim = [&](int x) {                            // lays slot_next, row_next, .. on tile x
            ok = wait(B_AIM0 + x % kAhead, (uint32_t)(x / kAhead & 1)) && ok;   // if not: an older tile, or none
            const Tile* tile = &misc->tile[x % kAhead];
            row_next = tile->row;
            valid_next = tile->seen[q4 >> 1] >> (st & 63) & 1u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint64_t m = tile->seen[h];
                slot_next[h] = tile->page[h] * kPage + tok;
                if (m != ~0ull) slot_next[h] = m == 0 ? -1 : (m >> tok & 1u) ? slot_next[h] : slot_next[h] - tok + __ffsll((long long)m) - 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_FREE0 + x % kAhead]);
        };
        auto follow = [&]() {                              // fetches are for the tile aimed at from here on
#pragma unroll
            for (int h = 0; h < 2; ++h)
                src[h] = slot_next[h] < 0 ? nullptr : a.kv + (int64_t)slot_next[h] * kKvTokenBytes + c8 * 16;
        };
        static_assert(kKvPageBytes == kPage * kKvTokenBytes, "slots are rows");
        auto fetch_row = [&](uint4 (&dst)[2], int h, int at, uint32_t fill) {   // the 16 bytes at `at` + 16 c8 of the lane's row h
            if (src[h] != nullptr) dst[h] = ldg_pinned(reinterpret_cast<const uint4*>(src[h] + at));
            else dst[h] = make_uint4(fill, fill, fill, fill);
        };
        auto fetch = [&](uint4 (&dst)[2], int at, uint32_t fill) {
            fetch_row(dst, 0, at, fill);
            fetch_row(dst, 1, at, fill);
        };
        // The fetched tile x into shared memory, latent groups 0..3 as soon as the P.V of the
        // group has completed for tile x - 1 (for x = 0 that is a phase that counts as over),
        // then the RoPE block (free, as P^T, with the last group).  A row's registers take its
        // group two ahead as soon as they are empty, before the fence that hands the group over
        // (after it: 4 windows of 131072 133 us instead of 129).
        auto put_tile = [&](int x) {
            const uint32_t ph = (uint32_t)((x - 1) & 1);
            const bool more = x + 1 < n_mine;
            row = row_next;
            valid = valid_next;
            if (more) aim(x + 1);                          // while the first P.V runs
            // the scales as fp16 (exact), two blocks a word: every one in [2^-15, 2^7] = [0x0200, 0x5800]
            const uint32_t sc[2][2] = {{pack_h2(__uint_as_float(scv[0].x), __uint_as_float(scv[0].y)),
                                        pack_h2(__uint_as_float(scv[0].z), __uint_as_float(scv[0].w))},
                                       {pack_h2(__uint_as_float(scv[1].x), __uint_as_float(scv[1].y)),
                                        pack_h2(__uint_as_float(scv[1].z), __uint_as_float(scv[1].w))}};
            uint32_t bad = __vcmpgtu2(__vmaxu2(__vmaxu2(sc[0][0], sc[0][1]), __vmaxu2(sc[1][0], sc[1][1])), 0x58005800u) |
                           __vcmpltu2(__vminu2(__vminu2(sc[0][0], sc[0][1]), __vminu2(sc[1][0], sc[1][1])), 0x02000200u);
            auto hand_over = [&](int bar) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[bar]);
            };
            auto group = [&](auto gi) {
                constexpr int gg = decltype(gi)::value;
                ok = wait(B_PV0 + gg, ph) && ok;
                auto put_row = [&](auto hi) {
                    // 16 FP8 dims 128 gg + 16 c8 .. -> K-block 2 gg + c8 / 4, 16-byte chunks 2 (c8 % 4) + c8 / 4, and its neighbour
                    constexpr int h = decltype(hi)::value, kOff = 2 * gg * kBlk + h * kPage * 128;
                    const uint32_t sc2 = __byte_perm(sc[h][gg >> 1], 0, (gg & 1) ? 0x3232 : 0x1010);
                    const uint4 v = raw[gg & 1][h];
                    uint32_t o[8];
                    e4m3x4_scaled_h2(v.x, sc2, o[0], o[1]);
                    e4m3x4_scaled_h2(v.y, sc2, o[2], o[3]);
                    e4m3x4_scaled_h2(v.z, sc2, o[4], o[5]);
                    e4m3x4_scaled_h2(v.w, sc2, o[6], o[7]);
                    st_shared_v4<kOff>(put, o[0], o[1], o[2], o[3]);
                    st_shared_v4<kOff>(putx, o[4], o[5], o[6], o[7]);
                };
                put_row(std::integral_constant<int, 0>{});
                if (gg == 2 && more) follow();
                if (gg < 2 || more) fetch_row(raw[gg & 1], 0, ((gg + 2) & 3) * 128, 0u);
                put_row(std::integral_constant<int, 1>{});
                if (gg < 2 || more) fetch_row(raw[gg & 1], 1, ((gg + 2) & 3) * 128, 0u);
                hand_over(B_FULL0 + gg);
            };
            group(std::integral_constant<int, 0>{});
            group(std::integral_constant<int, 1>{});
            group(std::integral_constant<int, 2>{});
            group(std::integral_constant<int, 3>{});
            uint32_t rope_max = 0;                         // bf16 magnitudes, compared as integers: |r| < 2^16
            auto rope_row = [&](auto hi) {
                constexpr int h = decltype(hi)::value;
                const uint4 r = rope[h];
                rope_max = __vmaxu2(rope_max, __vmaxu2(__vmaxu2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu),
                                                       __vmaxu2(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu)));
                st_shared_v4<h * kPage * 128>(put_rope, bf16x2_to_h2_sat(r.x), bf16x2_to_h2_sat(r.y), bf16x2_to_h2_sat(r.z),
                                              bf16x2_to_h2_sat(r.w));
            };
            rope_row(std::integral_constant<int, 0>{});
            rope_row(std::integral_constant<int, 1>{});
            hand_over(B_FULL4);
            if (more) {
                fetch(scv, 512 - c8 * 16, 0x3f800000u);
                fetch(rope, 528, 0u);
            }
            if (bad | __vcmpgtu2(rope_max, 0x477f477fu)) record_error(a.st, DSA_DEVERR_FP16_RANGE, lane);
        };
        // The row's Q (fp16, K-major, 128-byte swizzle) in two steps: its bf16 on the way into
        // the place of the last one, which every S^T has read by then, and, a softmax later,
        // the same pieces as fp16.  put_q returns the softmax scale in log2 units times 2^-kq
        // of the Q.  Eight threads a head, a thread one 16-byte piece of each K-block.
        static_assert(64 * 8 == kWorkThreads, "a thread has piece tid % 8 of head tid / 8");
        auto q_at = [&](int u) {                           // K-block u; the odd latent ones have their chunks in turn
            return smem + kOffQ + u * 8192 + (tid >> 3) * 128 + (((tid ^ tid >> 3 ^ (u < 8 ? u & 1 : 0)) & 7) * 16);
        };
        auto fetch_q = [&](int q_row) {
            const uint4* qrow = reinterpret_cast<const uint4*>(a.q + (int64_t)q_row * (64 * 576)) + (tid >> 3) * 72 + (tid & 7);
#pragma unroll
            for (int u = 0; u < 9; ++u) cp_async_16(smem_addr(q_at(u)), qrow + u * 8);
        };
        auto put_q = [&](int q_row) -> float {
            cp_async_wait_all();
            uint32_t mx = 0;                               // two bf16 magnitudes, compared as integers
#pragma unroll
            for (int u = 0; u < 9; ++u) {
                const uint4 qv = *reinterpret_cast<const uint4*>(q_at(u));
                mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(qv.x & 0x7fff7fffu, qv.y & 0x7fff7fffu),
                                           __vmaxu2(qv.z & 0x7fff7fffu, qv.w & 0x7fff7fffu)));
            }
            mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
            if (lane == 0) misc->qmax[warp] = mx;
            work_sync();
            mx = __reduce_max_sync(0xffffffffu, misc->qmax[lane & (kWorkWarps - 1)]);
            const int eq = mx == 0 ? 14 : (int)(mx >> 7) - 127;
            const int kq = min(126, max(-126, 14 - eq));
            const float sc = __int_as_float((127 + kq) << 23);
#pragma unroll
            for (int u = 0; u < 9; ++u) {
                uint4* at = reinterpret_cast<uint4*>(q_at(u));
                const uint4 qv = *at;
                *at = make_uint4(bf16x2_scaled_to_h2(qv.x, sc), bf16x2_scaled_to_h2(qv.y, sc), bf16x2_scaled_to_h2(qv.z, sc),
                                 bf16x2_scaled_to_h2(qv.w, sc));
            }
            if (tid == 0 && mx >= 0x7f80u) record_error(a.st, DSA_DEVERR_FP16_RANGE, q_row);   // inf / NaN in q
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_QFULL]);
            // neither 0 nor inf: differences of scores are multiplied by it that may be inf or 0
            return fminf(fmaxf(a.scale * __int_as_float((127 - kq) << 23) * 1.4426950408889634f, 0x1p-126f), 0x1.fffffep127f);
        };

        float lsum[kHeads];                                // this token lane's running sums of its heads
#pragma unroll
        for (int c = 0; c < kHeads; ++c) lsum[c] = 0.f;
        if (tid < 32) neg_inf[tid] = -INFINITY;
        if (tid < 64) neg_ref[tid] = kNoRef;               // seen by all behind put_q's barrier
        fetch_q(row_begin);
        aim(0);
        follow();
        fetch(scv, 512 - c8 * 16, 0x3f800000u);
        fetch(raw[0], 0, 0u);
        fetch(raw[1], 128, 0u);
        fetch(rope, 528, 0u);
        float sl2 = put_q(row_begin);
        put_tile(0);
        int piece = 0;
        for (;; ++n) {
            const uint32_t done = row;                      // row and flags of this tile
            // ---- softmax of tile n
            ok = wait(B_SFULL, (uint32_t)(n & 1)) && ok;
            // a token that is not seen takes -inf for its references: every P is 0
            const float4* nr4 = reinterpret_cast<const float4*>(valid ? neg_ref + hh * kHeads : neg_inf);
            uint32_t most;                                  // largest P of the thread, as two fp16
            // S^T row of this token for the warp's heads
            auto load_s = [&](float (&v)[kHeads]) {
                uint32_t x[kHeads];
                tmem_ld_32x32b_x16(lane_addr + kColS + hh * kHeads, x);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < kHeads; ++h) v[h] = __uint_as_float(x[h]);
            };
            // P of the current references, and its P^T row (heads 16 hh.. as fp16, MN-major swizzle).
            // P = 2^((S - reference) sl2), with references of the scores' kind: the difference of near
            // ones is exact however large they are.
            auto write_p = [&](float (&v)[kHeads]) {
                most = 0;
                auto eight = [&](auto ci) {
                    constexpr int c = decltype(ci)::value * 8;
                    const float4 m0 = nr4[c / 4], m1 = nr4[c / 4 + 1];
                    const float2 s2 = make_float2(sl2, sl2);
                    const float2 x0 = add_scale2(make_float2(v[c], v[c + 1]), make_float2(m0.x, m0.y), s2);
                    const float2 x1 = add_scale2(make_float2(v[c + 2], v[c + 3]), make_float2(m0.z, m0.w), s2);
                    const float2 x2 = add_scale2(make_float2(v[c + 4], v[c + 5]), make_float2(m1.x, m1.y), s2);
                    const float2 x3 = add_scale2(make_float2(v[c + 6], v[c + 7]), make_float2(m1.z, m1.w), s2);
                    v[c] = ex2_approx(x0.x);
                    v[c + 1] = ex2_approx(x0.y);
                    v[c + 2] = ex2_approx(x1.x);
                    v[c + 3] = ex2_approx(x1.y);
                    v[c + 4] = ex2_approx(x2.x);
                    v[c + 5] = ex2_approx(x2.y);
                    v[c + 6] = ex2_approx(x3.x);
                    v[c + 7] = ex2_approx(x3.y);
                    const uint32_t h0 = pack_h2(v[c], v[c + 1]), h1 = pack_h2(v[c + 2], v[c + 3]);
                    const uint32_t h2 = pack_h2(v[c + 4], v[c + 5]), h3 = pack_h2(v[c + 6], v[c + 7]);
                    st_shared_v4(p_at ^ (c * 2), h0, h1, h2, h3);
                    most = __vmaxu2(most, __vmaxu2(__vmaxu2(h0, h1), __vmaxu2(h2, h3)));
                };
                eight(std::integral_constant<int, 0>{});
                eight(std::integral_constant<int, 1>{});
                fence_proxy_async_smem();
            };
            float v[kHeads];
            tc_fence_after();
            if (n + 1 < n_mine && (row_next & T_FIRST)) fetch_q((int)(row_next >> kRowShift));
            load_s(v);
            write_p(v);
            // ---- a score above its head's reference by more than 2^kTau
            //      makes every warp take new references (always on the piece's first tile)
            const bool over = (most & 0xffffu) > kPMaxH || most >> 16 > kPMaxH;
            tc_fence_before();
            if (vote(over || (done & T_SETTLE) || !ok)) {
                tc_fence_after();
                if (vote(!ok)) {
                    if (tid == 0) timeout(63);
                    cp_async_wait_all();                    // a next row's Q may be on its way
                    break;
                }
                load_s(v);
#pragma unroll
                for (int c = 0; c < kHeads; ++c) v[c] = valid ? v[c] : -INFINITY;
                xreduce16<true>(v, lane);                   // per-head tile max (consumes v)
                if (lane < kHeads) red[q4 * 64 + hh * kHeads + lane] = v[0];
                if (done & T_SETTLE) {                      // the sums so far
#pragma unroll
                    for (int c = 0; c < kHeads; ++c) v[c] = lsum[c];
                    xreduce16<false>(v, lane);
                    if (lane < kHeads) red[256 + q4 * 64 + hh * kHeads + lane] = v[0];
                }
                work_sync();
                if (tid < 64) {
                    const float tm = fmaxf(fmaxf(red[tid], red[64 + tid]), fmaxf(red[128 + tid], red[192 + tid]));
                    const float mo = -neg_ref[tid], d = (tm - mo) * sl2;   // d: -inf where the tile saw nothing (NaN if none did)
                    float from = mo, down = 0.f;            // a renewed reference is `from`, `down` log2 units lower
                    if (d > kTau) {
                        from = tm;
                        down = (done & T_LATE) ? kSettled : kFirst;
                    } else if ((done & T_SETTLE) && mo > -INFINITY) {
                        const float l = red[256 + tid] + red[320 + tid] + red[384 + tid] + red[448 + tid];
                        down = kSettled - fmaxf(log2f(l), d);   // this tile's P stay below 2^kSettled too
                    }
                    alpha[tid] = 1.f;
                    if (down > 0.f) {                       // rounded up: never further down; finite for the smallest sl2
                        const float mr = __fsub_ru(from, fminf(down / sl2, 0x1p64f));
                        alpha[tid] = exp2f((mo - mr) * sl2);   // 0 for a first reference
                        neg_ref[tid] = -mr;
                    }
                }
                work_sync();
                bool mine = false;                          // does a head of this warp have a new reference
#pragma unroll
                for (int c = 0; c < kHeads; ++c) mine |= alpha[hh * kHeads + c] != 1.f;
                if (mine) {
                    if (!(done & T_FIRST)) {                           // rescale the resident O^T columns of these heads
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
                tc_fence_before();
                vote(false);
            }
#pragma unroll
            for (int c = 0; c < kHeads; ++c) lsum[c] += v[c];
            // ---- the next row's Q and the next tile
            float sl2_next = sl2;
            if (n + 1 < n_mine) {
                if (row_next & T_FIRST) sl2_next = put_q((int)(row_next >> kRowShift));
                put_tile(n + 1);
            }
            if (!(done & T_LAST)) continue;
            // ---- the piece's output: O^T is final when its last P.V has completed
            ok = wait(B_PV3, (uint32_t)(n & 1)) && ok;
            if (n + 1 == n_mine) pdl_trigger();             // the merge's blocks may take their places
            xreduce16<false>(lsum, lane);
            if (lane < kHeads) red[256 + q4 * 64 + hh * kHeads + lane] = lsum[0];
            work_sync();                                    // a timeout here is seen by the next vote, or is the end
            tc_fence_after();
            if (tid < 64) {
                const float l = red[256 + tid] + red[320 + tid] + red[384 + tid] + red[448 + tid];
                l_acc[tid] = l;
                alpha[tid] = l == 0.f ? 0.f : 1.f / l;      // its place is free until the next references
            }
            work_sync();
            const int64_t unit = 2 * (int64_t)blockIdx.x + (piece++ == 0 ? 0 : 1);   // a share's first piece, or its last
#pragma unroll 1
            for (int mb = 0; mb < 4; ++mb) {
                uint32_t o[kHeads];
                tmem_ld_32x32b_x16(lane_addr + kColO + mb * 64 + hh * kHeads, o);
                tmem_ld_wait();
                const int d = mb * 128 + (st ^ q4 >> 1 << 3);          // latent dim of this TMEM lane (chunks of odd K-blocks in turn)
                if (!(done & T_WHOLE)) {                               // a warp stores 32 dims of four heads at a time
                    float4* to = reinterpret_cast<float4*>(a.part_o) + (unit * 16 + hh * (kHeads / 4)) * 512 + d;
#pragma unroll
                    for (int c = 0; c < kHeads; c += 4)
                        to[c / 4 * 512] = make_float4(__uint_as_float(o[c]), __uint_as_float(o[c + 1]), __uint_as_float(o[c + 2]),
                                                      __uint_as_float(o[c + 3]));
                    continue;
                }
#pragma unroll
                for (int c = 0; c < kHeads; ++c) {
                    const float inv = alpha[hh * kHeads + c];
                    o[c] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(o[c]) * inv);   // a NaN among what is seen stays one
                }
                const int64_t at = ((int64_t)(done >> kRowShift) * 64 + hh * kHeads) * 512;
                if (a.out_f32) {
                    float* to = static_cast<float*>(a.out) + at + d;
#pragma unroll
                    for (int c = 0; c < kHeads; ++c) to[c * 512] = __uint_as_float(o[c]);
                    continue;
                }
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + at + d;
#pragma unroll
                for (int c = 0; c < kHeads; ++c) to[c * 512] = __float2bfloat16_rn(__uint_as_float(o[c]));
            }
            tc_fence_before();
            if (tid < 64) {
                const float l = l_acc[tid];
                const float ref = -neg_ref[tid] * sl2;                 // in log2 units
                if (!(done & T_WHOLE)) a.part_ml[unit * 64 + tid] = make_float2(ref, l);
                else if (a.lse) a.lse[(int64_t)(done >> kRowShift) * 64 + tid] = l == 0.f ? -INFINITY : (log2f(l) + ref) * 0.69314718055994531f;
                neg_ref[tid] = kNoRef;
            }
            if (n + 1 == n_mine) {
                if (!ok && lane == 0) timeout(64);
                break;
            }
            sl2 = sl2_next;
#pragma unroll
            for (int c = 0; c < kHeads; ++c) lsum[c] = 0.f;
            work_sync();                                    // O^T and the references may be reused
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- merge
// Blocks of a row that was cut, four heads and 128 dims at a time.  Where there are
// more shares than rows, block x looks after row x (8 rows x 17 pieces 21.8 us; by
// boundary, most of whose blocks have nothing to do, 28.0); else after the row that
// share x + 1 begins inside, if it is the first to do so.  Per head over the pieces u:
//   M = max m_u,  w_u = 2^(m_u - M),  L = sum w_u l_u,
//   out = sum_u w_u O_u / L,  lse = (M + log2 L) ln 2.
// Every warp works the weights out by itself, eight pieces x four heads a step, the
// outputs of eight pieces in flight meanwhile: two round trips behind the shares'
// beginnings.
constexpr int kMergeThreads = 128;

__global__ void __launch_bounds__(kMergeThreads, 4)
dense_merge_kernel(const __grid_constant__ Args a, int G, int by_row) {
    __shared__ int32_t s_first[4], s_more[4], s_whole[4];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int row = blockIdx.x;
    if (!by_row) {
        const Meta me = a.meta[blockIdx.x + 1], prev = a.meta[blockIdx.x];
        if (!me.inside || (prev.inside && prev.row == me.row)) return;
        row = me.row;
    }
    // the shares that begin inside the row follow one another; the row's first piece is in
    // the one before them: its first if it begins with the row, else its last
    int first = INT32_MAX, more = 0, begins = 0;
    for (int i = tid; i < G; i += kMergeThreads) {
        const Meta m = a.meta[i];
        if (m.row != row) continue;
        if (m.inside) {
            first = min(first, i);
            ++more;
        } else {
            begins = 1;
        }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    more = __reduce_add_sync(0xffffffffu, more);
    begins = __reduce_or_sync(0xffffffffu, begins);
    if (lane == 0) {
        s_first[warp] = first;
        s_more[warp] = more;
        s_whole[warp] = begins;
    }
    __syncthreads();
    const int np = 1 + s_more[0] + s_more[1] + s_more[2] + s_more[3];
    if (np == 1) return;
    first = min(min(s_first[0], s_first[1]), min(s_first[2], s_first[3]));
    const int64_t unit0 = 2 * (int64_t)(first - 1) + (s_whole[0] | s_whole[1] | s_whole[2] | s_whole[3] ? 0 : 1);
    auto unit = [&](int i) { return i == 0 ? unit0 : 2 * (int64_t)(first - 1 + i); };
    for (int part = blockIdx.y; part < 64; part += gridDim.y) {
        const int h0 = part >> 2 << 2, d = (part & 3) * kMergeThreads + tid;   // heads h0 .. h0 + 3, dim d
        float4 v[8], next[8];
        auto load_o = [&](float4 (&v)[8], int q0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (q0 + j < np) v[j] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (unit(q0 + j) * 16 + (h0 >> 2)) * 512 + d);
        };
        // lane: piece q0 + lane / 4, head h0 + lane % 4; {-inf, 0} of a piece that saw nothing
        auto load_ml = [&](int q0) {
            float2 ml = make_float2(-INFINITY, 0.f);
            if (q0 + (lane >> 2) < np) ml = __ldcg(a.part_ml + unit(q0 + (lane >> 2)) * 64 + h0 + (lane & 3));
            if (ml.y == 0.f) ml.x = -INFINITY;
            return ml;
        };
        load_o(v, 0);
        float2 ml = load_ml(0), ml_next;
        float M = ml.x;
#pragma unroll 4
        for (int q0 = 8; q0 < np; q0 += 8) M = fmaxf(M, load_ml(q0).x);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q0 = 0; q0 < np; q0 += 8) {
            load_o(next, q0 + 8);
            ml_next = load_ml(q0 + 8);
            const float w = ml.y == 0.f ? 0.f : exp2f(ml.x - M);
            L += w * ml.y;                                 // NaN if any piece's sum is
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (q0 + j >= np) break;
                const float w0 = __shfl_sync(0xffffffffu, w, 4 * j), w1 = __shfl_sync(0xffffffffu, w, 4 * j + 1);
                const float w2 = __shfl_sync(0xffffffffu, w, 4 * j + 2), w3 = __shfl_sync(0xffffffffu, w, 4 * j + 3);
                if (w0 != 0.f) acc.x = fmaf(w0, v[j].x, acc.x);   // a piece that saw nothing holds no numbers
                if (w1 != 0.f) acc.y = fmaf(w1, v[j].y, acc.y);
                if (w2 != 0.f) acc.z = fmaf(w2, v[j].z, acc.z);
                if (w3 != 0.f) acc.w = fmaf(w3, v[j].w, acc.w);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = next[j];
            ml = ml_next;
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        const float inv = L == 0.f ? 0.f : 1.f / L;        // lane % 4: head
        const int64_t at = ((int64_t)row * 64 + h0) * 512 + d;
        const float x[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float val = x[e] * __shfl_sync(0xffffffffu, inv, e);
            if (a.out_f32) static_cast<float*>(a.out)[at + e * 512] = val;
            else static_cast<__nv_bfloat16*>(a.out)[at + e * 512] = __float2bfloat16_rn(val);
        }
        if (a.lse && (part & 3) == 0 && tid < 4)
            a.lse[(int64_t)row * 64 + h0 + tid] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
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
    // 32-bit tile counts of a share, rows with their flags in a word
    if (b->total_q * most_tiles(b, view) / device_sm_count() > 0x7ffffff0LL || b->total_q >> (32 - kRowShift)) return DSA_ERR_UNSUPPORTED;
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
    a.scale = softmax_scale;
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
        // A block per part of a row where few rows can be cut, which may have many pieces (4
        // rows x 38 pieces 137 us, with four parts a block 150), four parts a block where many
        // can (200 rows 127 us, with one part a block 137).
        const bool by_row = b->total_q < G;
        DSA_CHECK(launch_pdl(dense_merge_kernel, dim3(by_row ? (unsigned)b->total_q : (unsigned)(G - 1), b->total_q < 32 ? 64 : 16),
                             dim3(kMergeThreads), 0, s, 1, a, G, (int)by_row));
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
