// Attention of grouped heads over the KV8 cache, for requests with many query rows
// (prefill chunks): the tiles, the pipeline and the softmax of the packed prompts' kernel,
// on fp16 operands.
//   S = Q K^T      tcgen05.mma kind::f16, M = 128 rows (tokens x the group's heads), N = 128 keys
//   O += P V       P from TMEM, V as it lies in the cache, with a block's tokens side by side:
//                  a K-major operand
// Converter warps turn a step's 128 keys (two pages) into the 128-byte-swizzled stages that
// the MMAs read: 16 codes are one load, two stores of 16 bytes, and conversions only, as
// E4M3 is exact in fp16; a code's load for the next stage is under way while the others of
// this one are converted.  The blocks' scales stay out of the operands: the softmax takes a
// block's 16 scores times 2^ek, and P carries 2^ev.  With t = score + ev (log2 units), R
// the row's reference, a whole number, so that ev - R is exact,
//   P = 2^(t - R) <= 2^kTop in fp16,  O = sum P code_v,  l = sum 2^-ev P,  out = O / l
//
// Q comes by TMA as bf16 and is turned, in place, into fp16 by the softmax threads, each its
// own row: times the power of two that puts its largest |q| in [2^14, 2^15).
//
// Warps: softmax as there; then a warpgroup with one warp each for a tile's MMAs, the items and
// Q's copies; then the converters.
//
// What bounds it: 2048 tokens of 64 heads of 128 dims over 16384 take 984 to 993 us (1.05 PFLOP/s, 55 % of
// a library's product).  A step of both tiles is 4,300 cycles: of them 2,048 MMAs, 2,440 a tile's
// softmax (traced with the clock), and the converters, four warps with a stage's codes in their registers, are busy
// for 3,700.  Without their work the kernel takes 12 % less.  (Half of them for keys and half
// for values: 1563 us, as registers spill and a stage is held for a whole step while it is
// written.)  At 256 dims the converters bound it, 6,600 cycles a step: 512 rows of 32 heads over
// 32768 take 874 to 887 us (614 to 624 TFLOP/s; 936 with 104 registers a converter, which spill).  At 64
// dims 2048 tokens over 16384 take 770 us, no unit being more than 43 % busy.
#include <algorithm>

#include "grouped_tc.cuh"
#include "kv8.cuh"

namespace dsa {

int device_sm_count();

namespace kv8 {

using namespace sm100;
using namespace mlc;
using namespace gtc;

struct PrefillArgs {
    const uint8_t* cache;
    BatchDev b;
    int kv_heads, group, tokens;
    int run;                    // key heads laid out together
    uint32_t* dealt;            // items taken
    int min_rows;               // requests with fewer query rows are not this kernel's
    float scale;                // softmax scale * log2(e)
    void* out;
    int out_f32;
    float* lse;
    int32_t* st;
    Split split;
};

namespace {

constexpr float kNone = -3e38f;                            // reference of a row that has seen nothing so far: below any score
constexpr float kFirst = 7.0f, kTop = 15.0f;               // log2 of a new reference's P, and of the largest
// Scores (log2 units) up to here.  A score's product with its units is rounded once with the
// reference taken off, the reference on its own: they differ by half a step of the score, 1/2
// below 2^24, and P stays below 2^(kTop + 1/2), which fp16 holds.
constexpr float kMostScore = 16777216.0f;
constexpr int kMeta = 8;                                   // steps whose scales are kept: more than the ring holds

template <int D> struct TcShape {
    static constexpr int kDim = D;
    static constexpr int kTiles = D <= 128 ? 2 : 1;
    static constexpr int kSoft = kTiles * 4;
    static constexpr int kConv = D <= 128 ? 4 : 8;         // converter warps
    static constexpr int kConv0 = kSoft + 4;               // the first of them
    static constexpr int kThreads = 512;
    static constexpr int kSoftRegs = kTiles == 2 ? 184 : 232, kMmaRegs = 40, kConvRegs = kTiles == 2 ? 104 : 120;
    static_assert(kSoft * 32 * kSoftRegs + 128 * kMmaRegs + kConv * 32 * kConvRegs <= kThreads * 128, "more registers than the launch holds");
    static_assert(kSoftRegs >= 128 && kMmaRegs <= 128 && kConvRegs <= 128, "who takes and who gives");
    static constexpr int kPart = D < 128 ? D : 128;
    static constexpr int kParts = D / kPart;
    static constexpr int kStage = kBox * kPart / 64;
    static constexpr int kQ = kTiles * kBox * (D / 64);
    static constexpr int kStages = (232448 - 1024 - 2048 - kQ) / kStage < 10 ? (232448 - 1024 - 2048 - kQ) / kStage : 10;
    static constexpr int kSmem = kQ + kStages * kStage + 2048 + 1024;
    static constexpr uint32_t kIdQK = idesc_f16_f32(128, kKeys, false, false), kIdPV = idesc_f16_f32(128, kPart, false, false);
    static constexpr bool kValuesMn = false;
    static constexpr bool kCleans = false;                 // the converters do
    static constexpr bool kCut = true;
    static constexpr bool kTurns = false;                  // 2048 over 16384: 979 us without, 993 with it, 1024 over 8192 288 and 280, at 64 dims 769 and 719
    static constexpr uint32_t s(int i) { return 128 * i; }
    static constexpr uint32_t o(int i) { return 256 + 128 * i; }
};

struct Block {
    Pipe pipe;
    uint64_t q_raw[2];          // by tile: Q has come as bf16
    alignas(16) float k2[kMeta][8];   // scales of a step's blocks' keys
    alignas(16) float ev[kMeta][8];   // exponents of their values'
    int32_t far;                // some row's scores are beyond kMostScore
    uint32_t here[kMeta];       // bit h: the step's page h is in the cache
};
static_assert(sizeof(Block) <= 2048, "the block behind the ring");

__device__ __forceinline__ uint32_t nan_of(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

}  // namespace

template <int D>
__global__ void __launch_bounds__(TcShape<D>::kThreads, 1)
kv8_prefill_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap qmap) {
    using S = TcShape<D>;
    constexpr int kMmaWarp = S::kSoft, kItemWarp = kMmaWarp + 2, kQWarp = kMmaWarp + 3;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* q_smem = smem;
    uint8_t* ring = smem + S::kQ;
    Block* blk = reinterpret_cast<Block*>(ring + S::kStages * S::kStage);
    Pipe* pipe = &blk->pipe;
    // (a warp's number that the compiler knows for the warp's: its operands stay in uniform registers)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&pipe->kv_full[i], S::kConv);
            mbar_init(&pipe->kv_empty[i], S::kTiles);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&blk->q_raw[i], 1);
            mbar_init(&pipe->q_full[i], 4);
            mbar_init(&pipe->q_empty[i], 1);
            mbar_init(&pipe->s_full[i], 1);
            mbar_init(&pipe->o_done[i], 1);
            mbar_init(&pipe->drain[i], 1);
            mbar_init(&pipe->turn[i], 1);
            for (int h = 0; h < 2; ++h) mbar_init(&pipe->p_full[i][h], 4);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&pipe->item_full[i], 1);
            mbar_init(&pipe->item_empty[i], S::kSoft + S::kTiles + 1 + S::kConv);   // softmax, MMAs, Q's copies, converters
        }
        pipe->abort = 0;
        blk->far = 0;
        mbar_arrive(&pipe->turn[0]);                         // the first tile begins
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&pipe->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = 0;                               // all 512 columns are the CTA's
    pdl_wait();
    pdl_trigger();
    const BatchDev& b = a.b;
    const Role me = {pipe, b.wait_ns, a.st, warp, lane};

    // Registers by warpgroup, of 128 a thread at launch: a converter holds a stage's pieces of codes.
    // (Set within the roles' branches: behind a join, all roles get the fewest.)
    if (warp < S::kSoft) {
        more_registers<S::kSoftRegs>();
        // ======================================================== softmax: a thread a row
        const int x = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int tok_of = row / a.group, head_of = row % a.group;
        const int heads = a.kv_heads * a.group;
        uint32_t t = 0, q_items = 0, u0 = 0;               // the tile's steps, items with a Q and steps of the CTA so far
        Item it;
        bool ok = true;
        for (int k = 0; ok && me.take<S::kCut>(k, it); ++k) {
            const int count = it.count(x, a.tokens), steps = it.steps(x, a.tokens);
            const int most = max(it.steps(0, a.tokens), S::kTiles == 2 ? it.steps(1, a.tokens) : 0);
            const int tok = it.tok0 + x * a.tokens + tok_of;
            const bool live = tok_of < count;
            const int see = live ? it.see(tok) : INT32_MAX;
            float c = 0.f;                                 // log2 units of a score
            if (steps > 0) {
                ok = me.wait_all(&blk->q_raw[x], q_items++);
                if (!ok) break;
                {
                    // the row's chunks of 8 dims, swizzled
                    uint8_t* mine = q_smem + x * (D / 64) * kBox + row * 128;
                    uint32_t top = 0;
#pragma unroll 4
                    for (int j = 0; j < D / 8; ++j) {
                        const uint4 w = *reinterpret_cast<const uint4*>(mine + j / 8 * kBox + ((j ^ row) & 7) * 16);
                        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t lo = v[e] & 0x7fffu, hi = v[e] >> 16 & 0x7fffu;
                            if (lo < 0x7f80u) top = max(top, lo);          // of finite ones
                            if (hi < 0x7f80u) top = max(top, hi);
                        }
                    }
                    const int e = q_exponent(top);
                    const float up = pow2(e);
                    c = q_units(a.scale, e, 0x1p100f);     // times a key's scale, up to 2^24, it is finite
#pragma unroll 4
                    for (int j = 0; j < D / 8; ++j) {
                        uint4* p = reinterpret_cast<uint4*>(mine + j / 8 * kBox + ((j ^ row) & 7) * 16);
                        uint4 w = *p;
                        w.x = bf16x2_scaled_to_h2(w.x, up), w.y = bf16x2_scaled_to_h2(w.y, up);
                        w.z = bf16x2_scaled_to_h2(w.z, up), w.w = bf16x2_scaled_to_h2(w.w, up);
                        *p = w;
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&pipe->q_full[x]);
            }
            float ref = 0.f, sum = 0.f;                    // R, l
            float low = 0.f;                               // the first R: they only rise
            for (int i = 0; ok && i < steps; ++i, ++t) {
                const int s = S::kTiles == 2 ? x : t & 1;
                ok = me.wait_all(&pipe->s_full[s], S::kTiles == 2 ? t : t >> 1);
                if (!ok) break;
                tc_fence_after();
                uint32_t w[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(tmem + lanes + S::s(s) + 32 * q, w[q]);
                const int u = (u0 + i) % kMeta;
                const uint32_t here = blk->here[u];
                tmem_ld_wait();
                const int lim = see - (it.from + i) * kKeys;           // keys of the step that the row sees
                if (__any_sync(0xffffffffu, lim < kKeys) || here != 3u) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * q + j >= lim || !(here >> (q >> 1) & 1)) w[q][j] = 0xff800000u;
                }
                float top = -INFINITY;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const uint32_t* v = &w[g >> 1][16 * (g & 1)];
                    float m = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
                    for (int j = 2; j < 16; j += 2) m = max3(m, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                    top = fmaxf(top, fmaf(m, blk->k2[u][g] * c, blk->ev[u][g]));
                }
                const float fresh = top == -INFINITY ? kNone : rintf(top) - kFirst;
                if (i == 0) {
                    ref = low = fresh;
                } else if (__any_sync(0xffffffffu, top > ref + kTop)) {
                    const float to = top > ref + kTop ? fresh : ref, f = exp2f(ref - to);
                    ok = me.wait_all(&pipe->o_done[x], t - 1);
                    if (!ok) break;
                    tc_fence_after();
                    rescale_o<D>(tmem + lanes + S::o(x), f);
                    sum *= f;
                    if (ref == kNone) low = to;
                    ref = to;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int q = 2 * h; q < 2 * h + 2; ++q) {                  // 32 keys
                        uint32_t p[16];
#pragma unroll
                        for (int g = 2 * q; g < 2 * q + 2; ++g) {
                            const float ev = blk->ev[u][g], ck = blk->k2[u][g] * c;
                            const float2 c2 = make_float2(ck, ck), r2 = make_float2(ev - ref, ev - ref);
                            float2 sums = make_float2(0.f, 0.f);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t* v = &w[q][16 * (g & 1) + 2 * j];
                                float2 y = fma2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), c2, r2);
                                y.x = ex2_approx(y.x);
                                y.y = ex2_approx(y.y);
                                sums = add2(sums, y);
                                p[8 * (g & 1) + j] = pack_h2(y.x, y.y);
                            }
                            sum = fmaf(sums.x + sums.y, minus_pow2(ev), sum);
                        }
                        tmem_st_32x32b_x16(tmem + lanes + S::s(s) + 16 * q, p);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pipe->p_full[s][h]);
                }
            }
            u0 += most;
            // (asked here, of the first and the last reference: 1017 us when not asking took 996; of each in the
            // loop 1115, in the outputs' part 1023)
            if (live && ref != kNone && fmaxf(fabsf(low), fabsf(ref)) > kMostScore) blk->far = 1;
            // ---- the rows' outputs
            if (ok && steps > 0) {
                // each phase in turn, as one could be taken for the one after the next
                ok = S::kTiles == 2 || steps == 1 || me.wait(&pipe->o_done[x], t - 2);
                ok = __all_sync(0xffffffffu, ok && me.wait(&pipe->o_done[x], t - 1));
                tc_fence_after();
            }
            if (ok && count > 0) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const bool cut = it.slot >= 0;             // a piece's rows are its slot's
                const int64_t at = cut ? (int64_t)it.slot * (S::kTiles * 128) + x * 128 + row : (int64_t)(it.q_row + tok) * heads + it.h * a.group + head_of;
                void* const to = cut ? a.split.part_o : a.out;
                const bool odd = pipe->any_odd[k % kItems] != 0;
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    if (steps > 0) {
                        tmem_ld_32x32b_x32(tmem + lanes + S::o(x) + d, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0;
                    }
                    if (live) {
                        float y[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(o[j]) * inv;
                        if (odd) {
                            // NaN values of masked steps that this row sees
                            for (int e = 0; e < kMasked * kKeys; ++e) {
                                const int64_t key = ((int64_t)it.from + it.masked_from()) * kKeys + e;
                                if (!(pipe->odd[k % kItems][e / kKeys][e % kKeys / 32] >> (e & 31) & 1) || key >= see) continue;
                                const int64_t page = b.page_table[(int64_t)it.k_row * b.max_pages + key / kPage];
                                const uint8_t* v = a.cache + (page * a.kv_heads + it.h) * head_bytes(D) + v_at(D) + key % kPage / kBlock * (kBlock * D) +
                                                   d * kBlock + key % kBlock;
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if ((v[j * kBlock] & 0x7f) == 0x7f) y[j] = __int_as_float(0x7fc00000);
                            }
                        }
                        write_32(to, cut || a.out_f32, at * D + d, y);
                    }
                    __syncwarp();
                }
                if (live && cut) a.split.part_ml[at] = make_float2(ref, sum);
                else if (live && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
            }
            tc_fence_before();                             // O is read before the next item's first P says so
            me.done_with(k);
        }
    } else if (warp < S::kConv0) {
        fewer_registers<S::kMmaRegs>();
        if (warp < kItemWarp) {
            if (warp - kMmaWarp < S::kTiles) issue_mmas<S>(me, warp - kMmaWarp, smem_addr(q_smem), smem_addr(ring), a.tokens);
        } else if (warp == kItemWarp) {
            lay_out_items(
                me, b.batch, a.kv_heads, a.run, a.tokens, S::kTiles, a.split, a.dealt,
                [&](int r, int& qs, int& qn) {
                    qs = b.q_start[r];
                    qn = (int)max((int64_t)0, min((int64_t)b.q_start[r + 1], b.total_q) - qs);
                    if ((int64_t)qn * a.group < a.min_rows) qn = 0;
                },
                [&](int r, Item& it, bool first) {
                    const int len = b.seq_len[r];
                    const int64_t room = (int64_t)b.max_pages * kPage;
                    it.k_row = r;
                    it.len = len - (b.q_start[r + 1] - it.q_row) + it.n;
                    it.cap = (int)min((int64_t)INT32_MAX, room);
                    if (first && lane == 0 && it.h == 0 && it.tok0 == 0) {
                        if (it.len < it.n) record_error(a.st, DSA_DEVERR_INDEX_RANGE, it.len - it.n);
                        else if (len > room) record_error(a.st, DSA_DEVERR_INDEX_RANGE, len);
                    }
                });
        } else if (warp == kQWarp) {
            // ======================================================== Q's copies, by one thread
            uint32_t items[2] = {0, 0};
            bool ok = true;
            Item it;
            for (int k = 0; me.take<S::kCut>(k, it); ++k) {
                me.done_with(k);
#pragma unroll
                for (int x = 0; x < S::kTiles; ++x) {
                    if (lane != 0 || !ok || it.steps(x, a.tokens) == 0) continue;
                    if (items[x] > 0) ok = me.wait(&pipe->q_empty[x], items[x] - 1);
                    if (!ok) continue;
                    ++items[x];
                    mbar_arrive_expect_tx(&blk->q_raw[x], (uint32_t)(D * 2 * a.tokens * a.group));
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(q_smem + (x * (D / 64) + c) * kBox, &qmap, 64 * c, it.h * a.group, it.q_row + it.tok0 + x * a.tokens, &blk->q_raw[x]);
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            }
            if (lane == 0)                                 // copies in flight end before the CTA does
                for (int x = 0; x < S::kTiles; ++x)
                    if (items[x] > 0) mbar_wait(&blk->q_raw[x], (items[x] - 1) & 1);
        }
    } else {
        fewer_registers<S::kConvRegs>();
        // ======================================================== converters
        constexpr int kThr = S::kConv * 32;
        constexpr int kUnits = kKeys * S::kPart / 16 / kThr;                   // 16-byte pieces of a stage, a thread
        const int ct = tid - S::kConv0 * 32;
        uint32_t n = 0, u = 0;                             // stages and steps so far
        bool ok = true;
        Item it;
        for (int k = 0; ok && me.take<S::kCut>(k, it); ++k) {
            const int most = max(it.steps(0, a.tokens), S::kTiles == 2 ? it.steps(1, a.tokens) : 0), masked = it.masked_from();
            int last = it.n - 1;                           // the item's last token
            last = min(last, it.tok0 + a.tokens * S::kTiles - 1);
            const int top = it.see(last);                  // keys that some row of the item sees
            const bool tells = it.h == 0 && last == it.n - 1 && ct == 0;       // one item of a request records its pages
            const int32_t* table = b.page_table + (int64_t)it.k_row * b.max_pages;
            // Page h of step i: its id as the table has it, -1 behind what the item sees; then its
            // part of the head, NULL where there is none.  Ids are loaded three steps ahead, scales and
            // codes one step ahead of their use.
            auto page_at = [&](int i, int h) { return 2 * ((int64_t)it.from + i) + h; };
            auto id_of = [&](int i, int h) {
                const int64_t p = page_at(i, h);
                return p * kPage < top ? __ldg(table + p) : -1;
            };
            auto head_of_page = [&](int32_t id, int i, int h) -> const uint8_t* {
                if (id >= 0 && id < b.num_pages) return a.cache + ((int64_t)id * a.kv_heads + it.h) * head_bytes(D);
                if (tells && page_at(i, h) * kPage < top) record_error(a.st, DSA_DEVERR_PAGE_RANGE, id);
                return nullptr;
            };
            // Piece e of part p of a step's keys (v = 0): 16 dims of a token, or values: a block's 16 tokens of
            // a dim.  Neighbouring threads take neighbouring pieces, the first half of a thread's are of the
            // first page.
            constexpr int kHalf = kUnits / 2;
            constexpr int kPer = S::kPart / 16, kTokens = kThr / kPer;         // pieces of a token, tokens of a piece of all threads
            constexpr int kDims = kThr / S::kPart;                             // blocks of a piece of all threads
            const uint32_t k_from = ct / kPer * D + ct % kPer * 16, v_from = v_at(D) + ct / S::kPart * (kBlock * D) + ct % S::kPart * 16;
            auto piece = [&](const uint8_t* x0, const uint8_t* x1, int v, int p, int e) {
                const uint8_t* x = e < kHalf ? x0 : x1;
                const uint32_t off = v ? v_from + e % kHalf * kDims * (kBlock * D) + p * S::kPart * 16 : k_from + e % kHalf * kTokens * D + p * S::kPart;
                return x ? ldg_pinned(reinterpret_cast<const uint4*>(x + off)) : make_uint4(0, 0, 0, 0);
            };
            // ... and its place: the first 16 of its 32 bytes; the others' is the neighbour's
            const uint32_t k_to = ct % kPer / 4 * kBox + ct / kPer * 128 + ((2 * (ct % kPer % 4)) ^ (ct / kPer & 7)) * 16;
            auto place = [&](int v, int e) -> uint32_t {
                if (!v) return k_to + e * kTokens * 128;
                const int block = ct / S::kPart + e * kDims, d = ct % S::kPart;
                return block / 4 * (S::kPart * 128) + d * 128 + ((2 * (block % 4)) ^ (d & 7)) * 16;
            };
            static_assert(kTokens % 8 == 0 && kUnits % 2 == 0, "a thread's pieces have one swizzle and are half of each page's");
            // scales of block ct of a step: keys', values'
            auto scales_of = [&](const uint8_t* x0, const uint8_t* x1) {
                const uint8_t* x = ct < kBlocks ? x0 : x1;
                if (ct >= 8 || !x) return make_float2(1.f, 1.f);
                const float* sc = reinterpret_cast<const float*>(x + scale_at(D)) + ct % kBlocks;
                return make_float2(__ldg(sc), __ldg(sc + kBlocks));
            };
            // Pages of this step, the next and the one after; pieces under way, of the keys and of the values
            // to be converted next, loaded again as soon as they are used; the next keys' step's scales.
            const uint8_t *h0 = nullptr, *h1 = nullptr, *n0 = nullptr, *n1 = nullptr, *m0 = nullptr, *m1 = nullptr;
            uint4 w[2][S::kParts * kUnits];
            float2 sc = make_float2(1.f, 1.f);
            // Turns step i's keys (v = 0) or values, codes of pages x0 and x1, into their stages; the next ones
            // are z0's and z1's.
            auto convert = [&](auto kind, int i, const uint8_t* x0, const uint8_t* x1, const uint8_t* z0, const uint8_t* z1) {
                constexpr int v = decltype(kind)::value;
#pragma unroll
                for (int p = 0; p < S::kParts; ++p) {
                    const int s = n % S::kStages;
                    if (ok && n >= S::kStages) ok = me.wait_all(&pipe->kv_empty[s], n / S::kStages - 1);
                    if (!ok) return;
                    const uint32_t base = smem_addr(ring + s * S::kStage);
#pragma unroll
                    for (int e = 0; e < kUnits; ++e) {
                        uint4 c = w[v][p * kUnits + e];
                        if (v == 1 && i >= masked) {
                            // tokens that no row sees become zeros; a NaN joins the rows that see it in the end
                            const int block = ct / S::kPart + e * kDims;
                            const int seen = top - (it.from + i) * kKeys - block * kBlock;
                            uint32_t* q = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int left = seen - 4 * y;
                                q[y] &= left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1;
                                const uint32_t nan = nan_of(q[y]);
                                if (nan) {
                                    q[y] &= ~nan;
                                    for (int z = 0; z < 4; ++z)
                                        if (nan >> (8 * z) & 1) {
                                            const int key = block * kBlock + 4 * y + z;
                                            atomicOr(&pipe->odd[k % kItems][i - masked][key >> 5], 1u << (key & 31));
                                        }
                                    pipe->any_odd[k % kItems] = 1;
                                }
                            }
                        }
                        uint32_t h[8];
                        e4m3x4_h2(c.x, h[0], h[1]);
                        e4m3x4_h2(c.y, h[2], h[3]);
                        e4m3x4_h2(c.z, h[4], h[5]);
                        e4m3x4_h2(c.w, h[6], h[7]);
                        const uint32_t to = base + place(v, e);
                        st_shared_v4(to, h[0], h[1], h[2], h[3]);
                        st_shared_v4(to ^ 16, h[4], h[5], h[6], h[7]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pipe->kv_full[s]);
#pragma unroll
                    for (int e = 0; e < kUnits; ++e) w[v][p * kUnits + e] = piece(z0, z1, v, p, e);
                    ++n;
                }
            };
            // Step i's keys, of pages x0 and x1, and what the softmax has to know of it.
            auto keys = [&](int i, const uint8_t* x0, const uint8_t* x1, const uint8_t* z0, const uint8_t* z1) {
                if (ct < 8) {
                    const int at = (u + i) % kMeta;
                    blk->k2[at][ct] = pow2(scale_exponent(sc.x));
                    blk->ev[at][ct] = (float)scale_exponent(sc.y);
                    if (ct == 0) blk->here[at] = (x0 ? 1u : 0u) | (x1 || (2 * ((int64_t)it.from + i) + 1) * kPage >= top ? 2u : 0u);
                }
                sc = scales_of(z0, z1);
                convert(Constant<0>(), i, x0, x1, z0, z1);
            };
            if (most > 0) {
                const int32_t i0 = id_of(0, 0), i1 = id_of(0, 1), j0 = id_of(1, 0), j1 = id_of(1, 1), k0 = id_of(2, 0), k1 = id_of(2, 1);
                h0 = head_of_page(i0, 0, 0), h1 = head_of_page(i1, 0, 1);
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int e = 0; e < S::kParts * kUnits; ++e) w[v][e] = piece(h0, h1, v, e / kUnits, e % kUnits);
                sc = scales_of(h0, h1);
                n0 = head_of_page(j0, 1, 0), n1 = head_of_page(j1, 1, 1);
                m0 = head_of_page(k0, 2, 0), m1 = head_of_page(k1, 2, 1);
                if (S::kTiles == 1) keys(0, h0, h1, n0, n1);
            }
            for (int i = 0; ok && i < most; ++i) {
                const int32_t r0 = id_of(i + 3, 0), r1 = id_of(i + 3, 1);
                if (S::kTiles == 2) keys(i, h0, h1, n0, n1);
                else if (i + 1 < most) keys(i + 1, n0, n1, m0, m1);
                convert(Constant<1>(), i, h0, h1, n0, n1);
                h0 = n0, h1 = n1;
                n0 = m0, n1 = m1;
                m0 = head_of_page(r0, i + 3, 0), m1 = head_of_page(r1, i + 3, 1);
                // (8 x 96 tokens over 60,000, more than the L2 holds: 1487 us without, 1393 with; 2048 over
                // 16384, which it holds: 984 without, 994 with)
                if (ct == 0 && n0) prefetch_l2(n0, (uint32_t)head_bytes(D));
                if (ct == 32 && n1) prefetch_l2(n1, (uint32_t)head_bytes(D));
            }
            u += most;
            me.done_with(k);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && blk->far) record_error(a.st, DSA_DEVERR_FP16_RANGE, 0);
    if (warp == 0) tmem_dealloc(pipe->tmem_base, 512);
}

template <int D>
static dsa_status launch_tc(PrefillArgs a, int64_t longest, const CUtensorMap& q, cudaStream_t s) {
    using S = TcShape<D>;
    if (ensure_smem_limit(reinterpret_cast<const void*>(&kv8_prefill_kernel<D>), S::kSmem) != DSA_OK) return DSA_ERR_CUDA;
    const int64_t most = most_items(a.b.total_q, a.b.batch, a.kv_heads, a.tokens * S::kTiles);
    if (most > 0x7fff0000LL) return DSA_ERR_UNSUPPORTED;
    const unsigned G = a.split.slots ? (unsigned)a.split.ctas : (unsigned)std::min<int64_t>(a.split.ctas, most);
    if (!deals(most, longest, G)) a.dealt = nullptr;
    else DSA_CHECK(launch_pdl(clear_count, dim3(1), dim3(1), 0, s, 1, a.dealt));
    DSA_CHECK(launch_pdl(kv8_prefill_kernel<D>, dim3(G), dim3(S::kThreads), S::kSmem, s, 1, a, q));
    if (a.split.slots) {
        // items of the last round, at most; a block for every two rows, as long as the blocks are few
        const unsigned x = (unsigned)std::min<int64_t>(G, most), rows = S::kTiles * 128;
        const unsigned y = std::max(rows / 16, std::min(rows / kJoinRows, 2048 / x));
        DSA_CHECK(launch_pdl(join_kernel<D>, dim3(x, y), dim3(kJoinRows * kJoinWarps * 32), 0, s, 1, a.split, a.group, a.kv_heads, (int)rows, a.out,
                             a.out_f32, a.lse));
    }
    return DSA_OK;
}

// Slots of partial outputs: two a CTA where some request may be long enough for two pieces of an item.
static int slots(int sms, const dsa_batch* b) { return b->max_seq_len >= 2 * kMinSteps * kKeys ? 2 * sms : 0; }
static int64_t item_rows(int dim) { return dim <= 128 ? 256 : 128; }

size_t prefill_ws_bytes(int sms, const dsa_batch* b, int dim) {
    const size_t n = slots(sms, b);
    return (n * item_rows(dim) * (dim * 4 + 8) + sms * sizeof(Cut) + sizeof(uint32_t) + 255) / 256 * 256;
}

// The requests of the batch with at least min_rows query rows.
dsa_status launch_prefill(const dsa_heads* q, const uint8_t* cache, const dsa_batch* b, int32_t heads, int32_t kv_heads, int32_t dim,
                          int32_t min_rows, float scale_log2, void* out, int out_f32, float* lse, void* ws, int32_t* st, cudaStream_t s) {
    PrefillArgs a = {};
    a.cache = cache;
    a.b = to_dev(b);
    a.kv_heads = kv_heads, a.group = heads / kv_heads, a.tokens = 128 / a.group;
    a.run = heads_of_run(kv_heads, b->max_seq_len * (int64_t)dim * 2);
    a.min_rows = min_rows;
    a.scale = scale_log2;
    a.out = out, a.out_f32 = out_f32, a.lse = lse, a.st = st;
    a.split.ctas = device_sm_count();
    a.split.slots = slots(a.split.ctas, b);
    const size_t rows = a.split.slots * item_rows(dim);
    a.split.part_o = static_cast<float*>(ws);
    a.split.part_ml = reinterpret_cast<float2*>(a.split.part_o + rows * dim);
    a.split.cut = reinterpret_cast<Cut*>(a.split.part_ml + rows);
    a.dealt = reinterpret_cast<uint32_t*>(a.split.cut + a.split.ctas);
    CUtensorMap qm;
    if (!make_heads_map(q, dim, heads, b->total_q, (unsigned)a.group, (unsigned)a.tokens, &qm)) return DSA_ERR_CUDA;
    if (dim == 64) return launch_tc<64>(a, b->max_seq_len, qm, s);
    if (dim == 128) return launch_tc<128>(a, b->max_seq_len, qm, s);
    return launch_tc<256>(a, b->max_seq_len, qm, s);
}

}  // namespace kv8
}  // namespace dsa
