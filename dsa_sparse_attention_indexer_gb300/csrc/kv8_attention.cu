// Attention of grouped heads over the KV8 cache, for the few query rows of decode and
// verify steps:
//   S_j = scale <q, k_j> 2^ek,  out = sum_j softmax(S)_j 2^ev v_j
// in one pass over the pages with a running reference and sum per row.
//
// What bounds it is the cache's bytes (2 dim + 1/2 a token and head, at 16 operations a
// byte for a group of 8), so everything but the pages stays in registers:
//   - A page's part of one head is contiguous (16.4 KB at 128 dims) and comes by one bulk
//     copy into a ring of as many stages as shared memory holds.
//   - A warp takes a block of 16 tokens.  S^T = K Q^T and O^T += V^T P^T are
//     mma.m16n8k16 in fp16 with tokens, then dims, as the 16 rows and the query rows as
//     the 8 columns: a group of 8 heads fills them, and codes go from shared memory to the
//     operand's registers, converted on the way (E4M3 is exact in fp16).  K's dims and
//     the block's tokens are taken in the order in which a thread's bytes lie.  P^T
//     comes from S^T by transposing 8 x 8 matrices within the warp.
//   - tcgen05 would have the codes converted into shared memory and read back from
//     there, 128 rows for the 8 that there are.
//
// Work split: row blocks of 8, 16, 32 or 64 query rows (tokens x the group's heads) of a
// request and head form one line of pages, cut into equal shares, one per CTA.  The eight
// consumer warps of a CTA take a share's blocks of tokens in turn, each with its own
// reference, sum and O^T, and are joined behind the share's part of a row block; a row
// block that several shares hold leaves one partial each, joined by a second kernel.
//
// Measured: 64 rows of 8 x 8 heads of 128 dims on 32768 tokens 680 us (6.3 TB/s, 93 % of a copy), of
// 64 dims 621 (3.5 TB/s); one row on 8192 16.7 us, two launches and a chain of loads; 16 x 6 tokens
// of 16 heads of 256 dims on 16381 162 us (3.2 TB/s, half of a copy): the chain of 24 rows' products and
// their softmax, 2,900 cycles a page of 33 KB, with the tensor pipe 37 % busy.  The shapes of 128
// and 256 dims spill 72 to 164 bytes a thread, but for <128, 2, 1>.  All requests of a call have
// the columns of its longest: 63 rows on 32768 beside a chunk, whose columns are 64, take 2.2 ms.
//
// P is held in fp16 against a reference per column and warp: a score and the exponent of
// its block's values, such that that position's P is 2^kFirst; it is renewed, and O^T
// rescaled, when a P passes 2^kTop.  P carries the block's 2^ev; its sum does not.
#include <algorithm>

#include "kv8.cuh"
#include "mla_common.cuh"

namespace dsa {

int device_sm_count();

namespace kv8 {

using namespace sm100;
using namespace mlc;

struct Meta {                   // where a CTA's share begins, for the second kernel
    int32_t r, rb, h;           // request, row block, head; r < 0: no share
    int32_t inside;             // the row block's pages of this head began in an earlier share
};

struct Args {
    const uint16_t* q;          // bf16 rows of heads
    int64_t q_tok, q_head;
    const uint8_t* cache;
    BatchDev b;
    int kv_heads, group;
    int max_rows;               // requests with more query rows are not this kernel's
    float scale;                // softmax scale * log2(e)
    void* out;
    int out_f32;
    float* lse;
    float* part_o;              // [2 G][cols][D]: normalised outputs of cut row blocks
    float4* part_ml;            // [2 G][cols]: reference, sum, log2 units of a score
    Meta* meta;                 // [G]
    int32_t* st;
};

constexpr int kConsumers = 8;                              // warps
constexpr int kThreads = (kConsumers + 4) * 32;             // a third warpgroup, of which one warp issues the copies
// Registers: 168 a thread at launch (65,536 / 384, in eights), of which the third
// warpgroup gives some to the consumers: 256 x 224 + 128 x 56 = 384 x 168.
constexpr int kLaunchRegs = 168, kConsRegs = 224, kProdRegs = 56;
static_assert(kConsumers * 32 * kConsRegs + 128 * kProdRegs <= kThreads * kLaunchRegs, "more registers than the launch holds");
constexpr int kConsBar = 1;
constexpr float kFirst = 7.0f, kTop = 15.0f;               // log2 of a reference's P, and of the largest

// GR: halves of the consumer warps.  With one, the halves take alternate pages, each with all
// columns of the row block; with two, each half takes every page with half of the columns, so
// that a page is copied once for as many rows as the registers of all warps hold (O^T is
// D / 4 * NB of them): 16 requests of 24 rows at 256 dims 182 us with two row blocks, 160 so.
template <int D, int NB, int GR> struct Shape {
    static constexpr int kCols = 8 * NB * GR;              // query rows of a row block
    static constexpr int kReaders = kPage / kBlock * GR;   // warps that read a page
    static constexpr int kKSteps = D / 16;
    static constexpr bool kQRegs = NB * D <= 256;          // Q stays in registers
    static constexpr int kHead = (int)head_bytes(D);
    static constexpr int kRedStride = D + 4;
    static constexpr int kRedBytes = kConsumers * 8 * kRedStride * 4;
    static constexpr int kQBytes = NB * GR * kKSteps * 32 * 8;
    static constexpr int kFixed = kRedBytes + kQBytes + 5120;
    // An even number, so that a stage's pages are all one half's of the warps: a warp that waits for
    // a stage's next page has seen the last one there, whose phase it could take for the next one's.
    static constexpr int kStages = (232448 - 1024 - kFixed) / kHead < 16 ? (232448 - 1024 - kFixed) / kHead / 2 * 2 : 16;
    static constexpr int kSmem = kStages * kHead + kFixed + 128;
};

struct Misc {
    uint64_t full[16], empty[16];
    int32_t valid[16];          // the stage holds a page
    int32_t abort;
    int32_t r0, rb0, h0;        // where the share begins
    int64_t page0, mine, at;    // page of the row block, pages of the share, of the line before it
    int64_t scratch[kThreads / 32];
    float c[64];                // log2 units of a column's score
    float ref[kConsumers][32], exp[kConsumers][32], sum[kConsumers][32];       // of a warp's columns
    float join[64][3];          // per column: reference, factor of O, sum
};
static_assert(sizeof(Misc) <= 5120, "misc block");

// A request's rows as this call sees them.
struct Request {
    int64_t row0;               // its first batch row
    int32_t prefix;             // tokens before its new ones (negative: some rows see nothing)
    int32_t rows;               // query rows: new tokens x group
    int32_t blocks;             // row blocks
    int64_t room;               // positions that the page table has
};
template <int COLS>
__device__ __forceinline__ Request request(const Args& a, int r) {
    const BatchDev& b = a.b;
    Request w;
    const int64_t end = min((int64_t)b.q_start[r + 1], b.total_q);
    w.row0 = b.q_start[r];
    const int n = (int)max((int64_t)0, end - w.row0);
    w.prefix = b.seq_len[r] - (b.q_start[r + 1] - b.q_start[r]);
    w.rows = n * a.group > a.max_rows ? 0 : n * a.group;
    w.blocks = (w.rows + COLS - 1) / COLS;
    w.room = (int64_t)b.max_pages * kPage;
    return w;
}
// Positions that row block rb sees together, and its pages: at least one, so that rows
// that see nothing are written.
template <int COLS>
__device__ __forceinline__ int64_t top_of(const Request& w, int rb, int group) {
    const int last = (min(w.rows, (rb + 1) * COLS) - 1) / group;
    return max((int64_t)0, min((int64_t)w.prefix + last + 1, w.room));
}
__device__ __forceinline__ int64_t pages_of(int64_t top) { return max((int64_t)1, (top + kPage - 1) / kPage); }

// Pages of all row blocks and heads of a request.
template <int COLS>
__device__ __forceinline__ int64_t line_of(const Args& a, const Request& w) {
    int64_t n = 0;
    for (int rb = 0; rb < w.blocks; ++rb) n += pages_of(top_of<COLS>(w, rb, a.group));
    return n * a.kv_heads;
}

// Counts the line's pages and finds this CTA's share of them.
template <int COLS>
__device__ __noinline__ void plan_share(const Args& a, Misc* misc, int tid) {
    const int B = a.b.batch, per = (B + kThreads - 1) / kThreads;
    const int r0 = min(B, tid * per), r1 = min(B, r0 + per);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += line_of<COLS>(a, request<COLS>(a, r));
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if ((tid & 31) >= o) x += y;
    }
    if ((tid & 31) == 31) misc->scratch[tid >> 5] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < (tid >> 5)) before += misc->scratch[w];
        all += misc->scratch[w];
    }
    before += x - mine;
    const int64_t n = all / gridDim.x, longer = all - n * gridDim.x, g = blockIdx.x;
    int64_t at = g * n + min(g, longer);
    if (tid == 0) misc->mine = n + (g < longer);
    if (at >= before && at < before + mine) {
        at -= before;
        int r = r0;
        for (;; ++r) {
            const int64_t t = line_of<COLS>(a, request<COLS>(a, r));
            if (at < t) break;
            at -= t;
        }
        const Request w = request<COLS>(a, r);
        int rb = 0;
        for (;; ++rb) {
            const int64_t t = pages_of(top_of<COLS>(w, rb, a.group)) * a.kv_heads;
            if (at < t) break;
            at -= t;
        }
        const int64_t p = pages_of(top_of<COLS>(w, rb, a.group));
        misc->r0 = r, misc->rb0 = rb, misc->h0 = (int)(at / p);
        misc->page0 = at % p;
    }
    __syncthreads();
}

// Walks a share's pieces: the part of a row block and head that the share holds.
template <int COLS>
struct Walk {
    int r, rb, h;
    int64_t page, end, pages;   // the piece's pages [page, end) of the row block's
    int64_t top;                // positions that the row block sees
    int64_t left;               // pages of the share behind this piece
    Request w;
    __device__ __forceinline__ void start(const Args& a, const Misc* m) {
        r = m->r0, rb = m->rb0, h = m->h0;
        page = m->page0;
        left = m->mine;
        w = request<COLS>(a, r);
        cut(a);
    }
    __device__ __forceinline__ void cut(const Args& a) {
        top = top_of<COLS>(w, rb, a.group);
        pages = pages_of(top);
        end = min(pages, page + left);
        left -= end - page;
    }
    __device__ __forceinline__ bool next(const Args& a) {
        if (left == 0) return false;
        page = 0;
        if (++h == a.kv_heads) {
            h = 0;
            ++rb;
            while (rb >= w.blocks) {                       // pages are left, so a request follows
                rb = 0;
                w = request<COLS>(a, ++r);
            }
        }
        cut(a);
        return true;
    }
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The bytes of a word that are NaN codes, as 4 bits.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    const uint32_t m = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) & 0x01010101u;
    return (m | m >> 7 | m >> 14 | m >> 21) & 15u;
}

template <int D, int NB, int GR>
__global__ void __launch_bounds__(kThreads, 1)
kv8_attention_kernel(const __grid_constant__ Args a) {
    using S = Shape<D, NB, GR>;
    constexpr int COLS = S::kCols, KS = S::kKSteps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
    float* red = reinterpret_cast<float*>(ring + S::kStages * S::kHead);
    uint2* qf = reinterpret_cast<uint2*>(ring + S::kStages * S::kHead + S::kRedBytes);
    Misc* misc = reinterpret_cast<Misc*>(ring + S::kStages * S::kHead + S::kRedBytes + S::kQBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int32_t* abort_flag = &misc->abort;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&misc->full[i], 1);
            mbar_init(&misc->empty[i], S::kReaders);
        }
        misc->abort = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    plan_share<COLS>(a, misc, tid);
    if (tid == 0)
        a.meta[blockIdx.x] = misc->mine > 0 ? Meta{misc->r0, misc->rb0, misc->h0, misc->page0 > 0} : Meta{-1, 0, 0, 0};
    if (misc->mine == 0) return;
    auto timeout = [&](int where) {
        record_error(a.st, DSA_DEVERR_TIMEOUT, where);
        *abort_flag = 1;
    };
    Walk<COLS> k;
    k.start(a, misc);

    if (warp >= kConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProdRegs));
        if (warp > kConsumers) return;
        // ==================================================== producer: a page's part of the head a stage
        uint32_t n = 0;                                    // stages so far (a share's pages are bounded by the host)
        bool ok = true;
        do {
            const int32_t* table = a.b.page_table + (int64_t)k.r * a.b.max_pages;
            if (lane == 0 && k.page == 0 && k.h == 0 && k.rb == 0) {
                if (k.w.prefix < 0) record_error(a.st, DSA_DEVERR_INDEX_RANGE, k.w.prefix);
                else if (a.b.seq_len[k.r] > k.w.room) record_error(a.st, DSA_DEVERR_INDEX_RANGE, a.b.seq_len[k.r]);
            }
            for (int64_t p0 = k.page; p0 < k.end; p0 += 32) {
                int32_t id = -1;
                if (p0 + lane < k.end && (p0 + lane) * kPage < k.top) {
                    id = table[p0 + lane];
                    if (id < 0 || id >= a.b.num_pages) {
                        record_error(a.st, DSA_DEVERR_PAGE_RANGE, id);
                        id = -1;
                    }
                }
                const int m = (int)min((int64_t)32, k.end - p0);
                for (int i = 0; i < m; ++i, ++n) {
                    const int s = n % S::kStages;
                    const int64_t page = __shfl_sync(0xffffffffu, id, i);
                    if (lane == 0 && ok && n >= S::kStages &&
                        !wait_for(&misc->empty[s], (n / S::kStages - 1) & 1, abort_flag, a.b.wait_ns)) {
                        timeout(1);
                        ok = false;
                    }
                    // the stage's last copy has ended (its readers waited for it): a second arrival in one phase would be a fault
                    if (lane == 0 && ok && n >= S::kStages && !mbar_test_wait(&misc->full[s], (n / S::kStages - 1) & 1)) {
                        timeout(3);
                        ok = false;
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) {
                        misc->valid[s] = page >= 0;
                        if (page >= 0) {
                            mbar_arrive_expect_tx(&misc->full[s], S::kHead);
                            bulk_load(ring + s * S::kHead, a.cache + (page * a.kv_heads + k.h) * (int64_t)S::kHead, S::kHead, &misc->full[s]);
                        } else {
                            mbar_arrive(&misc->full[s]);
                        }
                    }
                }
                if (!ok) break;
            }
        } while (ok && k.next(a));
        // copies in flight end before the CTA does
        if (lane == 0)
            for (uint32_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i)
                if (!mbar_wait(&misc->full[i % S::kStages], i / S::kStages & 1)) break;
        return;
    }

    // ======================================================== consumers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsRegs));
    const int g = lane >> 2, t = lane & 3;
    const int tok0 = 4 * (g >> 1) + (g & 1);               // K rows g and g + 8 of the operand hold tokens tok0 and tok0 + 2
    const int blk = warp & 3;                              // block of the page
    const int col0 = GR == 2 ? (warp >> 2) * 8 * NB : 0;   // the warp's first column
    const int first_warp = GR == 2 ? warp & ~3 : 0;        // of those with the same columns
    constexpr int kSame = kConsumers / GR;                 // warps with the same columns
    uint32_t n = 0;                                        // stages before the piece
    bool ok = true;
    do {
        const int64_t row_of = k.w.row0;
        auto q_row = [&](int col, int& tok, int& hd) {     // column -> new token and query head; false behind the last row
            const int i = k.rb * COLS + col;
            tok = i / a.group;
            hd = k.h * a.group + i % a.group;
            return i < k.w.rows;
        };
        // ---- Q: each row times the power of two that puts its largest |q| in [2^14, 2^15), in operand order
        for (int col = warp; col < COLS; col += kConsumers) {
            int tok, hd;
            const bool live = q_row(col, tok, hd);
            const uint16_t* src = a.q + (row_of + tok) * a.q_tok + hd * a.q_head;
            constexpr int kWords = (D / 4 + 31) / 32;      // 4 dims a lane
            uint2 w[kWords];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int d = 4 * (lane + 32 * i);
                w[i] = live && d < D ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0, 0);
                // the largest finite magnitude, as bf16 bits
                const uint32_t m[4] = {w[i].x & 0x7fffu, w[i].x >> 16 & 0x7fffu, w[i].y & 0x7fffu, w[i].y >> 16 & 0x7fffu};
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max(top, m[j] < 0x7f80u ? m[j] : 0u);
            }
            top = __reduce_max_sync(0xffffffffu, top);
            const int e = q_exponent(top);
            const float up = pow2(e);
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int d = 4 * (lane + 32 * i);
                if (d < D) {
                    const int ks = d / 64 * 4 + d % 16 / 4, to = (col & 7) * 4 + d % 64 / 16;
                    qf[((col >> 3) * KS + ks) * 32 + to] = make_uint2(bf16x2_scaled_to_h2(w[i].x, up), bf16x2_scaled_to_h2(w[i].y, up));
                }
            }
            if (lane == 0) misc->c[col] = q_units(a.scale, e, 0x1.fffffep127f);
        }
        bar_sync<kConsBar, kConsumers * 32>();
        uint2 qr[S::kQRegs ? NB * KS : 1];
        if constexpr (S::kQRegs) {
#pragma unroll
            for (int i = 0; i < NB * KS; ++i) qr[i] = qf[((col0 >> 3) * KS + i) * 32 + lane];
        }
        float o[NB][D / 16][4];                            // O^T: dims 16 i + g and + 8, columns 8 nb + 2 t and + 1
        float ref[NB][2], ex[NB][2], sum[NB][2], c[NB][2];
        uint32_t see[NB][2];                               // positions that the column sees
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nb][i][j] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                ref[nb][j] = -INFINITY;
                ex[nb][j] = 0.f;                           // kFirst - exponent of the reference's values
                sum[nb][j] = 0.f;
                c[nb][j] = misc->c[col0 + 8 * nb + 2 * t + j];
                int tok, hd;
                q_row(col0 + 8 * nb + 2 * t + j, tok, hd);
                see[nb][j] = (uint32_t)max((int64_t)0, (int64_t)k.w.prefix + tok + 1);
            }
        }
        const uint32_t all_see = (uint32_t)max((int64_t)0, (int64_t)k.w.prefix + k.rb * COLS / a.group + 1);      // positions that every row of the block sees

        // with one half of columns, odd pages of the share are warps 4-7's
        for (int64_t p = k.page + (GR == 1 ? (warp >> 2 ^ n) & 1 : 0); p < k.end; p += 3 - GR) {
            const uint32_t m = n + (uint32_t)(p - k.page);
            const int s = m % S::kStages;
            if (ok && !wait_for(&misc->full[s], m / S::kStages & 1, abort_flag, a.b.wait_ns)) {
                timeout(2);
                ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (ok && misc->valid[s] && p * kPage + blk * kBlock < k.top) {
                const uint32_t pos = (uint32_t)p * kPage + blk * kBlock;    // of the block's first token; below seq_len (the block's last may not fit 31 bits)
                const uint8_t* head = ring + s * S::kHead;
                const float* scales = reinterpret_cast<const float*>(head + scale_at(D));
                const float k2 = pow2(scale_exponent(scales[blk]));
                const int ev = scale_exponent(scales[kBlocks + blk]);
                // ---- S^T
                float sc[NB][4];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[nb][j] = 0.f;
                const uint8_t* kr = head + (blk * kBlock + tok0) * D + 16 * t;
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    const uint4 x = *reinterpret_cast<const uint4*>(kr + 64 * h);
                    const uint4 y = *reinterpret_cast<const uint4*>(kr + 64 * h + 2 * D);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_h2(xs[w], a0, a2);
                        e4m3x4_h2(ys[w], a1, a3);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            uint2 b;
                            if constexpr (S::kQRegs) b = qr[nb * KS + h * 4 + w];
                            else b = qf[(((col0 >> 3) + nb) * KS + h * 4 + w) * 32 + lane];
                            mma_16816(sc[nb], a0, a1, a2, a3, b.x, b.y);
                        }
                    }
                }
                // ---- P^T: positions pos + tok0 (elements 0, 1) and + 2 (elements 2, 3)
                const bool masked = pos + kBlock > all_see;
                const uint32_t at = pos + tok0;
                bool outgrown = false;
                float x[NB][4];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sc[nb][j] *= k2;
                        x[nb][j] = fmaf(sc[nb][j] - ref[nb][j & 1], c[nb][j & 1], (float)ev + ex[nb][j & 1]);
                        if (masked && at + (j & 2) >= see[nb][j & 1]) x[nb][j] = -INFINITY;
                        outgrown |= x[nb][j] > kTop;
                    }
                if (__any_sync(0xffffffffu, outgrown)) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const bool in0 = !(masked && at >= see[nb][j]), in1 = !(masked && at + 2 >= see[nb][j]);
                            float top = fmaxf(in0 ? sc[nb][j] : -INFINITY, in1 ? sc[nb][2 + j] : -INFINITY);
                            bool mine = x[nb][j] > kTop || x[nb][2 + j] > kTop;
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                            mine = (__ballot_sync(0xffffffffu, mine) & (0x11111111u << t)) != 0;
                            if (mine) {
                                // a column without a reference has nothing to rescale
                                const bool fresh = ref[nb][j] == -INFINITY;
                                const float by = (ref[nb][j] - top) * c[nb][j], ne = kFirst - (float)ev;
                                const float f = fresh ? 0.f : exp2f(by - ex[nb][j] + ne), fs = fresh ? 0.f : exp2f(by);
                                sum[nb][j] *= fs;
#pragma unroll
                                for (int i = 0; i < D / 16; ++i) {
                                    o[nb][i][j] *= f;
                                    o[nb][i][2 + j] *= f;
                                }
                                ref[nb][j] = top;
                                ex[nb][j] = ne;
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (e ? in1 : in0) x[nb][2 * e + j] = fmaf(sc[nb][2 * e + j] - top, c[nb][j], kFirst);
                            }
                        }
                }
                uint32_t b0[NB], b1[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[nb][j] = ex2_approx(x[nb][j]);
                    // the sum's share of P: without the values' exponent and the reference's 2^kFirst
#pragma unroll
                    for (int j = 0; j < 2; ++j) sum[nb][j] = fmaf(x[nb][j] + x[nb][2 + j], minus_pow2((float)ev + ex[nb][j]), sum[nb][j]);
                    b0[nb] = transpose8(pack_h2(x[nb][0], x[nb][1]));
                    b1[nb] = transpose8(pack_h2(x[nb][2], x[nb][3]));
                }
                // ---- O^T
                const uint8_t* vr = head + v_at(D) + blk * kBlock * D + g * 16 + 4 * t;
                if (!masked) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_h2(*reinterpret_cast<const uint32_t*>(vr + i * 256), a0, a2);
                        e4m3x4_h2(*reinterpret_cast<const uint32_t*>(vr + i * 256 + 128), a1, a3);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_16816(o[nb][i], a0, a1, a2, a3, b0[nb], b1[nb]);
                    }
                } else {
                    // Tokens that no row of the block sees may hold anything, and a NaN counts for the
                    // rows that see it alone: 0 times NaN is none of the others' business.
                    const int seen = (int)min((int64_t)kBlock, k.top - pos);        // tokens that some row sees
                    uint32_t keep = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) keep |= 4 * t + j < seen ? 0xffu << (8 * j) : 0u;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t v[2] = {*reinterpret_cast<const uint32_t*>(vr + i * 256) & keep,
                                         *reinterpret_cast<const uint32_t*>(vr + i * 256 + 128) & keep};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t nan = nan_bytes(v[e]);
                            if (!__any_sync(0xffffffffu, nan != 0)) continue;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (nan >> j & 1) v[e] &= ~(0xffu << (8 * j));
                            nan <<= 4 * t;                                          // by token, of the four lanes of the dim
                            nan |= __shfl_xor_sync(0xffffffffu, nan, 1);
                            nan |= __shfl_xor_sync(0xffffffffu, nan, 2);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int64_t u = (int64_t)see[nb][j] - pos;    // the column's tokens of the block
                                    const uint32_t mine = u <= 0 ? 0u : u >= 16 ? 0xffffu : (1u << u) - 1;
                                    if (nan & mine) o[nb][i][2 * e + j] = __int_as_float(0x7fc00000);
                                }
                        }
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_h2(v[0], a0, a2);
                        e4m3x4_h2(v[1], a1, a3);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_16816(o[nb][i], a0, a1, a2, a3, b0[nb], b1[nb]);
                    }
                }
            }
            // A warp that gave up frees nothing: the stage's copy may still be under way, and a
            // second one onto it would be one arrival too many for its barrier.
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&misc->empty[s]);
        }
        n += (uint32_t)(k.end - k.page);

        // ---- the eight warps' columns are joined
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum[nb][j] += __shfl_xor_sync(0xffffffffu, sum[nb][j], d);
                if (g == 0) {
                    const int col = 8 * nb + 2 * t + j;
                    misc->ref[warp][col] = ref[nb][j];
                    misc->exp[warp][col] = kFirst - ex[nb][j];
                    misc->sum[warp][col] = sum[nb][j];
                }
            }
        bar_sync<kConsBar, kConsumers * 32>();
        // O_w counts 2^(e_w - kFirst) 2^(ref_w c): brought to the largest of these, the sums to the largest reference
        float f[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = 8 * nb + 2 * t + j;
                float base = -INFINITY, most = -INFINITY, total = 0.f;
#pragma unroll
                for (int w = first_warp; w < first_warp + kSame; ++w) base = fmaxf(base, misc->ref[w][col]);
#pragma unroll
                for (int w = first_warp; w < first_warp + kSame; ++w) {
                    const float by = (misc->ref[w][col] - base) * c[nb][j];
                    if (misc->ref[w][col] > -INFINITY) most = fmaxf(most, by + misc->exp[w][col]);
                    // a warp without a reference has seen nothing, or a NaN that is in its sum
                    if (misc->sum[w][col] != 0.f) total += misc->sum[w][col] * (misc->ref[w][col] > -INFINITY ? exp2f(by) : 1.f);
                }
                f[nb][j] = ref[nb][j] > -INFINITY ? exp2f((ref[nb][j] - base) * c[nb][j] + (kFirst - ex[nb][j]) - most) : 1.f;
                if (warp == first_warp && g == 0) {
                    misc->join[col0 + col][0] = base;
                    misc->join[col0 + col][1] = total != 0.f ? exp2f(most - kFirst) / total : 0.f;
                    misc->join[col0 + col][2] = total;
                }
            }
        const bool whole = k.page == 0 && k.end == k.pages;
        // the piece that goes on from an earlier share is its share's first partial, the one that the next share goes on with the second
        const int64_t slot = 2 * (int64_t)blockIdx.x + (k.page > 0 ? 0 : 1);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float* mine = red + (warp * 8 + 2 * t) * S::kRedStride + g;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) mine[(j & 1) * S::kRedStride + 16 * i + (j >> 1) * 8] = o[nb][i][j] * f[nb][j & 1];
            bar_sync<kConsBar, kConsumers * 32>();
            for (int i = tid; i < GR * 8 * D / 4; i += kConsumers * 32) {
                const int gr = i / (8 * D / 4), cc = i / (D / 4) % 8, d = i % (D / 4) * 4, col = gr * 8 * NB + 8 * nb + cc;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = gr * kSame; w < gr * kSame + kSame; ++w) {
                    const float4 y = *reinterpret_cast<const float4*>(red + (w * 8 + cc) * S::kRedStride + d);
                    v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                }
                const float by = misc->join[col][1];
                v.x *= by, v.y *= by, v.z *= by, v.w *= by;
                int tok, hd;
                const bool live = q_row(col, tok, hd);
                if (!whole) {
                    reinterpret_cast<float4*>(a.part_o)[((slot * COLS + col) * D + d) / 4] = v;
                } else if (live) {
                    const int64_t to = ((row_of + tok) * (a.kv_heads * a.group) + hd) * D + d;
                    if (a.out_f32) {
                        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = v;
                    } else {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    }
                }
            }
            bar_sync<kConsBar, kConsumers * 32>();
        }
        if (tid < COLS) {
            int tok, hd;
            const bool live = q_row(tid, tok, hd);
            const float base = misc->join[tid][0], total = misc->join[tid][2];
            if (!whole) a.part_ml[slot * COLS + tid] = make_float4(base, total, misc->c[tid], 0.f);
            else if (live && a.lse)
                a.lse[(row_of + tok) * (a.kv_heads * a.group) + hd] = total == 0.f ? -INFINITY : (base * misc->c[tid] + log2f(total)) * 0.69314718055994531f;
        }
        bar_sync<kConsBar, kConsumers * 32>();             // c is read before the next piece's Q is laid out
    } while (k.next(a));
}

// Joins the partials of the row blocks that shares have cut: one block for each share
// that is the first to go on with one (x) and part of its columns (y).
template <int D, int COLS>
__global__ void __launch_bounds__(128)
kv8_merge_kernel(const __grid_constant__ Args a, int G) {
    pdl_wait();
    pdl_trigger();
    const int g = blockIdx.x + 1;
    const Meta me = a.meta[g], prev = a.meta[g - 1];
    auto same = [&](const Meta& m) { return m.r == me.r && m.rb == me.rb && m.h == me.h; };
    if (me.r < 0 || !me.inside || (prev.inside && same(prev))) return;
    const Request w = request<COLS>(a, me.r);
    __shared__ int32_t s_end;
    if (threadIdx.x == 0) s_end = G;
    __syncthreads();
    for (int i = g + 1 + threadIdx.x; i < G; i += blockDim.x) {
        const Meta m = a.meta[i];
        if (!m.inside || !same(m)) atomicMin(&s_end, i);
    }
    __syncthreads();
    const int np = 1 + s_end - g;
    // the first piece is the last of the share before
    auto slot = [&](int i) { return i == 0 ? 2 * (int64_t)(g - 1) + 1 : 2 * (int64_t)(g - 1 + i); };
    constexpr int kQuads = D / 4, kBatch = 8;
    for (int i = blockIdx.y * 128 + threadIdx.x; i < COLS * kQuads; i += gridDim.y * 128) {
        const int col = i / kQuads, d = i % kQuads * 4, row = me.rb * COLS + col;
        if (row >= w.rows) continue;
        // in one pass, eight pieces' loads at a time: {reference, sum, log2 units of a score}, four dims
        float4 ml[kBatch], y[kBatch];
        auto load = [&](int q0) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                ml[q] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
                if (q0 + q < np) {
                    ml[q] = __ldcg(&a.part_ml[slot(q0 + q) * COLS + col]);
                    y[q] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + ((slot(q0 + q) * COLS + col) * D + d) / 4);
                }
            }
        };
        float base = -INFINITY, total = 0.f, c = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q0 = 0; q0 < np; q0 += kBatch) {
            load(q0);
            float top = base;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) top = fmaxf(top, ml[q].x);
            c = ml[0].z;
            const float old = base > -INFINITY ? exp2f((base - top) * c) : 1.f;
            total *= old;
            v.x *= old, v.y *= old, v.z *= old, v.w *= old;
            base = top;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (ml[q].y == 0.f) continue;              // nothing seen, or no piece
                const float f = ml[q].y * (ml[q].x > -INFINITY ? exp2f((ml[q].x - base) * c) : 1.f);
                total += f;
                v.x = fmaf(f, y[q].x, v.x), v.y = fmaf(f, y[q].y, v.y), v.z = fmaf(f, y[q].z, v.z), v.w = fmaf(f, y[q].w, v.w);
            }
        }
        const float inv = total != 0.f ? 1.f / total : 0.f;
        v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
        const int64_t at = (w.row0 + row / a.group) * (a.kv_heads * a.group) + me.h * a.group + row % a.group;
        if (a.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * D + d) = v;
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + d) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
        if (a.lse && d == 0) a.lse[at] = total == 0.f ? -INFINITY : (base * c + log2f(total)) * 0.69314718055994531f;
    }
}

dsa_status launch_prefill(const dsa_heads* q, const uint8_t* cache, const dsa_batch* b, int32_t heads, int32_t kv_heads, int32_t dim,
                          int32_t min_rows, float scale_log2, void* out, int out_f32, float* lse, void* ws, int32_t* st, cudaStream_t s);
size_t prefill_ws_bytes(int sms, const dsa_batch* b, int dim);
// Requests with more query rows than this are the prefill kernel's.
constexpr int kTcRows = 64;

// Query rows of a row block.
static int columns(int64_t max_rows, int dim) {
    if (max_rows <= 8) return 8;
    if (max_rows <= 16) return 16;
    return max_rows <= 32 || dim == 256 ? 32 : 64;
}

static int64_t longest_request(const dsa_batch* b, int group) { return std::min<int64_t>(b->max_q_len, b->total_q) * group; }

// The two kernels' parts of the workspace, one behind the other.
static size_t few_rows_ws_bytes(int sms, int dim) {
    const size_t cols = dim == 256 ? 32 : 64;
    return ((size_t)2 * sms * cols * (dim * 4 + 16) + (size_t)sms * sizeof(Meta) + 255) / 256 * 256;
}
static size_t ws_bytes(int sms, const dsa_batch* b, int group, int dim) {
    return few_rows_ws_bytes(sms, dim) + (longest_request(b, group) > kTcRows ? prefill_ws_bytes(sms, b, dim) : 0);
}

template <int D, int NB, int GR>
static dsa_status launch(Args a, int sms, int G, cudaStream_t s) {
    using S = Shape<D, NB, GR>;
    if (ensure_smem_limit(reinterpret_cast<const void*>(&kv8_attention_kernel<D, NB, GR>), S::kSmem) != DSA_OK) return DSA_ERR_CUDA;
    a.part_ml = reinterpret_cast<float4*>(a.part_o + (size_t)2 * sms * S::kCols * D);
    a.meta = reinterpret_cast<Meta*>(a.part_ml + (size_t)2 * sms * S::kCols);
    DSA_CHECK(launch_pdl(kv8_attention_kernel<D, NB, GR>, dim3((unsigned)G), dim3(kThreads), S::kSmem, s, 1, a));
    if (G > 1)
        DSA_CHECK(launch_pdl(kv8_merge_kernel<D, S::kCols>, dim3((unsigned)(G - 1), (unsigned)(S::kCols * D / 4 / 128)), dim3(128), 0, s, 1, a, G));
    return DSA_OK;
}

}  // namespace kv8
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_kv8_attention_workspace_size(const dsa_batch* b, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                                       size_t* bytes) {
    dsa_status vs = validate_batch(b);
    if (vs != DSA_OK) return vs;
    vs = kv8::check_shape(heads, kv_heads, head_dim);
    if (vs != DSA_OK) return vs;
    if (!bytes) return DSA_ERR_INVALID_ARGUMENT;
    *bytes = kv8::ws_bytes(device_sm_count(), b, heads / kv_heads, head_dim);
    return DSA_OK;
}

extern "C" dsa_status dsa_kv8_attention(const dsa_heads* q, const uint8_t* cache, const dsa_batch* b, int32_t heads,
                                        int32_t kv_heads, int32_t head_dim, float softmax_scale, void* out,
                                        int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                                        void* stream) {
    dsa_status vs = validate_batch(b);
    if (vs != DSA_OK) return vs;
    vs = kv8::check_shape(heads, kv_heads, head_dim);
    if (vs != DSA_OK) return vs;
    if (out_dtype != DSA_DTYPE_BF16 && out_dtype != DSA_DTYPE_F32) return DSA_ERR_INVALID_ARGUMENT;
    if (!(softmax_scale > 0.f) || softmax_scale > kv8::kMostScale) return DSA_ERR_INVALID_ARGUMENT;
    if (b->total_q * (heads / kv_heads) > 0x7fffff00LL) return DSA_ERR_UNSUPPORTED;          // 32-bit query rows of a request
    if (b->total_q == 0) return DSA_OK;
    if (!q || !cache || !out || !ws) return DSA_ERR_INVALID_ARGUMENT;
    if ((vs = kv8::check_heads(q)) != DSA_OK) return vs;
    if (!aligned16(cache) || !aligned16(out) || !aligned16(ws)) return DSA_ERR_ALIGNMENT;
    const int sms = device_sm_count();
    if (ws_bytes < kv8::ws_bytes(sms, b, heads / kv_heads, head_dim)) return DSA_ERR_WORKSPACE_TOO_SMALL;
    kv8::Args a = {};
    a.q = static_cast<const uint16_t*>(q->data);
    a.q_tok = q->token_stride, a.q_head = q->head_stride;
    a.cache = cache;
    a.b = to_dev(b);
    a.kv_heads = kv_heads, a.group = heads / kv_heads;
    a.scale = softmax_scale * 1.44269504088896341f;
    a.out = out;
    a.out_f32 = out_dtype == DSA_DTYPE_F32;
    a.lse = lse;
    a.part_o = static_cast<float*>(ws);
    a.st = dev_status;
    const cudaStream_t s = as_stream(stream);
    const int64_t longest = kv8::longest_request(b, a.group);
    a.max_rows = 0x7fffffff;
    // q's strides as a tensor map takes them; a q that does not lie so has its rows taken one by one
    const bool mapped = (heads == 1 || q->head_stride > 0) && (b->total_q == 1 || q->token_stride > 0) && q->head_stride < 1LL << 38 && q->token_stride < 1LL << 38;
    const bool prefill = longest > kv8::kTcRows && mapped;
    // a single request is the prefill kernel's however few of its rows there turn out to be
    const bool all = prefill && b->batch == 1;
    if (prefill) a.max_rows = kv8::kTcRows;
    const int64_t max_rows = std::min<int64_t>(longest, a.max_rows);
    const int cols = kv8::columns(max_rows, head_dim);
    // the pages of a CTA's share are counted in 32 bits
    if (!all && (b->total_q * a.group / cols + b->batch) * kv_heads > 0x7fffffffLL * sms / (((int64_t)b->max_seq_len + kPage - 1) / kPage) / 2)
        return DSA_ERR_UNSUPPORTED;
    if (prefill) {
        vs = kv8::launch_prefill(q, cache, b, heads, kv_heads, head_dim, all ? 0 : kv8::kTcRows + 1, a.scale, out, a.out_f32, lse,
                                 static_cast<uint8_t*>(ws) + kv8::few_rows_ws_bytes(sms, head_dim), dev_status, s);
        if (vs != DSA_OK || all) return vs;
    }
    // no more CTAs than pages
    const int64_t blocks = std::min<int64_t>(b->total_q * a.group / cols + b->batch, b->total_q * a.group);
    const int64_t pages = ((int64_t)b->max_seq_len + kPage - 1) / kPage;
    const int G = (int)std::min<int64_t>(sms, std::max<int64_t>(1, blocks) * kv_heads * pages);
    switch (1000 * head_dim + cols) {
        case 64008: return kv8::launch<64, 1, 1>(a, sms, G, s);
        case 64016: return kv8::launch<64, 2, 1>(a, sms, G, s);
        case 64032: return kv8::launch<64, 4, 1>(a, sms, G, s);
        case 64064: return kv8::launch<64, 4, 2>(a, sms, G, s);
        case 128008: return kv8::launch<128, 1, 1>(a, sms, G, s);
        case 128016: return kv8::launch<128, 2, 1>(a, sms, G, s);
        case 128032: return kv8::launch<128, 4, 1>(a, sms, G, s);
        case 128064: return kv8::launch<128, 4, 2>(a, sms, G, s);
        case 256008: return kv8::launch<256, 1, 1>(a, sms, G, s);
        case 256016: return kv8::launch<256, 2, 1>(a, sms, G, s);
        default: return kv8::launch<256, 2, 2>(a, sms, G, s);
    }
}
