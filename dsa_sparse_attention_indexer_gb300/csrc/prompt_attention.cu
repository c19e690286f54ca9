// Causal attention of packed prompts with grouped heads, on bf16 keys and values:
//   S_tj = scale <q_t, k_j>,  out_t = sum_j softmax(S_t)_j v_j,  j <= k_len - q_len + t
// in one pass over the keys with a running reference and sum per row; S and P never
// leave the SM.
//
// Tiles: the 128 rows of an MMA are neighbouring tokens times the heads of a group, so
// that a group's keys and values are read once for all its heads, short prompts fill the
// rows and the diagonal cuts off less.  128 keys a step:
//   S = Q K^T      tcgen05.mma kind::f16, M = 128 rows, N = 128 keys, K = dim
//   O += P V       M = 128 rows, N = dim, K = 128 keys; P, in bf16, comes from TMEM, where
//                  it takes the place of its S; V is read MN-major as it lies
// Up to 128 dims a CTA holds two such tiles of rows (S and O of both fill the 512 TMEM
// columns): one's softmax runs beside the other's products.  At 256 dims it holds one,
// with two S.  Keys and values come by TMA, 128 keys x 128 dims a stage, in the 128-byte
// swizzle that both products read.
//
// Warps: 0-3 and 4-7 a tile's softmax each, a thread a row; then one warp each to issue
// a tile's MMAs, to issue the copies and to lay out the CTA's items (a request's, head's
// and tile pair's rows).  A row's probability of a key that it does not see is 0, and 0
// times an infinite or NaN value would not be: in a step that some rows see in part the
// softmax threads take those values out of shared memory before the MMA, and they join
// the rows that see them in the end.  (The first tile's threads do it for both tiles, 4 x ~2048
// tokens of 64 dims 66 us; each tile for itself 71.  They wait for the values' copy themselves
// where there are two tiles; told by the MMA warp, as with one, 72.)
//
// O is rescaled only when a row's largest score passes its reference by 2^8.
//
// What bounds it: the chain of a tile's softmax and MMAs, which overlaps the other tile's in
// part.  1 x 8192 tokens of 64 heads of 128 dims take 781 to 786 us (1.40 PFLOP/s, 73 % of a
// library's product), a step of both tiles about 3,300 cycles of which 2,048 are MMAs
// (tensor pipe 57 % busy).  At 64 dims a step's softmax is as long beside half of the MMAs: 4 x
// ~2048 tokens of 16 heads 66 us (tensor pipe and exponentials 26 % busy each).  At 256 dims
// there is one tile, whose softmax and MMAs follow one another but for S of the next step; 2 x
// ~4096 tokens of 64 heads 975 to 987 us (1.05 PFLOP/s).  Short prompts are bound by an item's two
// ends, about 4,000 cycles: 16 of up to 512 tokens 81 us, one of 129 10.0 on the GPU.  A few
// queries behind long keys leave SMs idle, as items are not cut along the keys: one query of 8
// key heads behind 8192 keys 87 us.
#include <algorithm>

#include <cudaTypedefs.h>

#include "grouped_tc.cuh"
#include "kv8.cuh"

namespace dsa {

int device_sm_count();

namespace gtc {
bool make_heads_map(const dsa_heads* h, int dim, int64_t heads, int64_t rows, unsigned bh, unsigned br, CUtensorMap* out) {
    const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    // the stride of an axis of one entry says nothing
    const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? h->head_stride : dim) * 2, (cuuint64_t)(rows > 1 ? h->token_stride : dim * heads) * 2};
    const cuuint32_t box[3] = {64, bh, br}, estr[3] = {1, 1, 1};
    return encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(h->data), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace gtc

namespace prompt {

using namespace sm100;
using namespace mlc;
using namespace gtc;

struct Args {
    const uint16_t* v;          // for values that are not finite
    int64_t v_tok, v_head;
    const int32_t *q_start, *k_start;
    int64_t total_q, total_k;
    int batch, kv_heads, group;
    int run;                    // key heads laid out together
    uint32_t* dealt;            // items taken
    int tokens;                 // of a tile: 128 / group
    float scale;                // softmax scale * log2(e)
    void* out;
    int out_f32;
    float* lse;
    uint64_t wait_ns;
    int32_t* st;
};

constexpr float kGrow = 8.0f;                              // log2 of how far a score may pass its reference

// kind::f16 with bf16 operands, fp32 sums.
constexpr uint32_t idesc_bf16(int M, int N, bool b_mn) { return idesc_f16_f32(M, N, false, b_mn) | (1u << 7) | (1u << 10); }

template <int D> struct Shape {
    static constexpr int kDim = D;
    static constexpr int kTiles = D <= 128 ? 2 : 1;        // tiles of rows of a CTA
    static constexpr int kSoft = kTiles * 4;               // softmax warps
    static constexpr int kThreads = (kSoft + 4) * 32;
    static constexpr int kPart = D < 128 ? D : 128;        // dims of a stage
    static constexpr int kParts = D / kPart;               // stages of a step's keys (or values)
    static constexpr int kStage = kBox * kPart / 64;
    static constexpr int kQ = kTiles * kBox * (D / 64);
    static constexpr int kStages = (232448 - 1024 - 2048 - kQ) / kStage < 10 ? (232448 - 1024 - 2048 - kQ) / kStage : 10;
    static constexpr int kSmem = kQ + kStages * kStage + 2048 + 1024;
    static constexpr uint32_t kIdQK = idesc_bf16(128, kKeys, false), kIdPV = idesc_bf16(128, kPart, true);
    static constexpr bool kValuesMn = true;
    static constexpr bool kCleans = true;
    // TMEM columns
    static constexpr bool kCut = false;
    static constexpr bool kTurns = true;
    static constexpr uint32_t s(int i) { return 128 * i; }
    static constexpr uint32_t o(int i) { return 256 + 128 * i; }
};

static_assert(sizeof(Pipe) <= 2048, "the block behind the ring");

// A 16-bit pair of bf16 holds an infinity or a NaN.
__device__ __forceinline__ uint32_t odd2(uint32_t w) { return __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u); }

// Takes infinite and NaN values of a masked step's keys from `from` on out of its stages and
// notes their keys; by the 128 threads of a tile, before their P says that the step's values
// may be read.  Masked is what some row of the item does not see.  The steps that the first
// tile sees are its threads' work, for which both tiles' MMAs wait: none reads what has not been
// taken out, and a row gets such a value in the end whether its P was 0 or not.
template <class S>
__device__ __noinline__ void clean_values(Pipe* m, uint8_t* ring, Place<S> vp, int from, int masked, int k, int thread) {
    for (int p = 0; p < S::kParts; ++p, vp.next()) {
        uint8_t* stage = ring + vp.stage * S::kStage;
        bool found = false;
#pragma unroll 4
        for (int e = thread; e < (kKeys - from) * (S::kPart / 8); e += 128) {  // a key's 8 pieces of 16 bytes of each 64 dims
            const int key = from + (e >> 3) % (kKeys - from), box = (e >> 3) / (kKeys - from);
            uint4* at = reinterpret_cast<uint4*>(stage + box * kBox + key * 128 + (e & 7) * 16);
            const uint4 w = *at;
            const uint4 o = make_uint4(odd2(w.x), odd2(w.y), odd2(w.z), odd2(w.w));
            if (o.x | o.y | o.z | o.w) {
                if (masked < kMasked) atomicOr(&m->odd[k % kItems][masked][key >> 5], 1u << (key & 31));
                m->any_odd[k % kItems] = 1;
                *at = make_uint4(w.x & ~o.x, w.y & ~o.y, w.z & ~o.z, w.w & ~o.w);
                found = true;
            }
        }
        if (found) fence_proxy_async_smem();
    }
    __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
prompt_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<D>;
    constexpr int kMmaWarp = S::kSoft, kTmaWarp = kMmaWarp + 2, kItemWarp = kMmaWarp + 3;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* q_smem = smem;
    uint8_t* ring = smem + S::kQ;
    Pipe* misc = reinterpret_cast<Pipe*>(ring + S::kStages * S::kStage);
    // (a warp's number that the compiler knows for the warp's: its operands stay in uniform registers)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&misc->kv_full[i], 1);
            mbar_init(&misc->kv_empty[i], S::kTiles);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&misc->q_full[i], 1);
            mbar_init(&misc->q_empty[i], 1);
            mbar_init(&misc->s_full[i], 1);
            mbar_init(&misc->o_done[i], 1);
            mbar_init(&misc->drain[i], 1);
            mbar_init(&misc->turn[i], 1);
            for (int h = 0; h < 2; ++h) mbar_init(&misc->p_full[i][h], 4);
        }
        mbar_init(&misc->here, 1);
        for (int i = 0; i < kCleans; ++i) mbar_init(&misc->clean[i], 4);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&misc->item_full[i], 1);
            mbar_init(&misc->item_empty[i], S::kSoft + S::kTiles + 1);  // the softmax warps and those of the MMAs and the copies
        }
        misc->abort = 0;
        mbar_arrive(&misc->turn[0]);                         // the first tile begins
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&misc->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = 0;                               // all 512 columns are the CTA's
    pdl_wait();
    pdl_trigger();
    const Role me = {misc, a.wait_ns, a.st, warp, lane};

    // Registers: 168 a thread at launch (65,536 / 384, in eights); 256 x 216 + 128 x 72 = 384 x 168.
    // (Set within the roles' branches: behind a join, all roles get the fewest.)
    if (warp < S::kSoft) {
        if constexpr (S::kTiles == 2) more_registers<216>();
        // ======================================================== softmax: a thread a row
        const int x = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int tok_of = row / a.group, head_of = row % a.group;
        const int heads = a.kv_heads * a.group;
        uint32_t t = 0, cleaned = 0;                       // steps, and of them those whose values its threads clean, so far
        Ring<S> at;                                        // where the steps' values are
        Item it;
        bool ok = true;
        for (int k = 0; ok && me.take<S::kCut>(k, it); ++k) {
            const int most = max(it.steps(0, a.tokens), S::kTiles == 2 ? it.steps(1, a.tokens) : 0);
            const int all_see = it.see(it.tok0), clean_from = it.cleans_from(x, a.tokens);       // keys that all of the item's rows see
            const int count = it.count(x, a.tokens), steps = it.steps(x, a.tokens);
            const int tok = it.tok0 + x * a.tokens + tok_of;
            const bool live = tok_of < count;              // tok_of < a.tokens too
            const int see = live ? it.see(tok) : INT32_MAX;
            float refc = 0.f, sum = 0.f;                   // reference in log2 units, sum of P
            Place<S> vp, np;
            if (most > 0) at.take();
            for (int i = 0; ok && i < steps; ++i, ++t) {
                at.step(i + 1 < most, vp, np);
                const int s = S::kTiles == 2 ? x : t & 1;
                if (i >= clean_from) {
                    // The step's values have to be there.  A wait for some of a stage's phases only takes the one before the
                    // last for the one that it is for, unless the last one has been.  With two tiles it has when the
                    // scores of the step before, or of the first, are there: the MMA warp has waited for every stage up
                    // to their keys.  With one tile the last phase may be the values of the step before, of which no
                    // score tells; the MMA warp, which waits for each phase, does.
                    if (S::kTiles == 1) {
                        ok = me.wait_all(&misc->here, cleaned);
                    } else {
                        static_assert(S::kTiles == 1 || (S::kParts == 1 && S::kStages >= 3), "a step's values are three stages behind the keys of the step before");
                        ok = (i > 0 || me.wait_all(&misc->s_full[s], t)) && me.wait_all(&misc->kv_full[vp.stage], vp.phase);
                    }
                    if (!ok) break;
                    clean_values<S>(misc, ring, vp, max(0, all_see - i * kKeys), i - it.masked_from(), k, (warp & 3) * 32 + lane);
                    if (S::kTiles == 2 && x == 0 && lane == 0) mbar_arrive(&misc->clean[cleaned % kCleans]);
                    ++cleaned;
                }
                ok = me.wait_all(&misc->s_full[s], S::kTiles == 2 ? t : t >> 1);
                if (!ok) break;
                tc_fence_after();
                uint32_t w[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tmem + lanes + S::s(s) + 32 * c, w[c]);
                tmem_ld_wait();
                const int lim = see - i * kKeys;           // keys of the step that the row sees
                if (__any_sync(0xffffffffu, lim < kKeys)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * c + j >= lim) w[c][j] = 0xff800000u;
                }
                float m[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    m[c] = fmaxf(__uint_as_float(w[c][0]), __uint_as_float(w[c][1]));
#pragma unroll
                    for (int j = 2; j < 32; j += 2) m[c] = max3(m[c], __uint_as_float(w[c][j]), __uint_as_float(w[c][j + 1]));
                }
                const float top = max3(fmaxf(m[0], m[1]), m[2], m[3]) * a.scale;
                if (i == 0) {
                    refc = top == -INFINITY ? -3e38f : top;      // (no score so far: whatever comes is above)
                } else if (__any_sync(0xffffffffu, top > refc + kGrow)) {
                    // O counts from a new reference
                    const float to = top > refc + kGrow ? top : refc, f = exp2f(refc - to);
                    ok = me.wait_all(&misc->o_done[x], t - 1);
                    if (!ok) break;
                    tc_fence_after();
                    rescale_o<D>(tmem + lanes + S::o(x), f);
                    sum *= f;
                    refc = to;
                }
                const float2 c2 = make_float2(a.scale, a.scale), r2 = make_float2(-refc, -refc);
                float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int e = 64 * h + 2 * j;
                        float2 y = fma2(make_float2(__uint_as_float(w[e >> 5][e & 31]), __uint_as_float(w[e >> 5][(e & 31) + 1])), c2, r2);
                        y.x = ex2_approx(y.x);
                        y.y = ex2_approx(y.y);
                        sums[j & 1] = add2(sums[j & 1], y);
                        p[j] = pack_bf2(y.x, y.y);
                    }
                    tmem_st_32x32b_x32(tmem + lanes + S::s(s) + 32 * h, p);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&misc->p_full[s][h]);
                }
                sums[0] = add2(sums[0], sums[1]);
                sum += sums[0].x + sums[0].y;
            }
            for (int i = steps; i < most; ++i) at.step(i + 1 < most, vp, np);
            // ---- the rows' outputs
            if (ok && steps > 0) {
                // With two S the last step's products began before the ones of the step before had
                // ended: each phase is waited for, so that none is taken for the one after it.
                ok = S::kTiles == 2 || steps == 1 || me.wait(&misc->o_done[x], t - 2);
                ok = __all_sync(0xffffffffu, ok && me.wait(&misc->o_done[x], t - 1));
                tc_fence_after();
            }
            if (ok && count > 0) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int64_t at = (int64_t)(it.q_row + tok) * heads + it.h * a.group + head_of;
                const bool odd = misc->any_odd[k % kItems] != 0;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    if (steps > 0) {
                        tmem_ld_32x32b_x32(tmem + lanes + S::o(x) + c, o);
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
                            // infinite and NaN values of masked steps that this row sees
                            for (int e = 0; e < kMasked * kKeys; ++e) {
                                const int64_t key = (int64_t)it.masked_from() * kKeys + e;
                                if (!(misc->odd[k % kItems][e / kKeys][e % kKeys / 32] >> (e & 31) & 1) || key >= see) continue;
                                const uint16_t* v = a.v + (it.k_row + key) * a.v_tok + it.h * a.v_head + c;
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    const float z = bf16_bits_to_f32(v[j]);
                                    if (!(fabsf(z) < INFINITY)) y[j] += z;
                                }
                            }
                        }
                        write_32(a.out, a.out_f32, at * D + c, y);
                    }
                    __syncwarp();
                }
                if (live && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (refc + log2f(sum)) * 0.69314718055994531f;
            }
            tc_fence_before();                             // O is read before the next item's first P says so
            me.done_with(k);
        }
    } else {
        if constexpr (S::kTiles == 2) fewer_registers<72>();
        if (warp < kTmaWarp) {
            if (warp - kMmaWarp < S::kTiles) issue_mmas<S>(me, warp - kMmaWarp, smem_addr(q_smem), smem_addr(ring), a.tokens);
        } else if (warp == kTmaWarp) {
            // ======================================================== copies, by one thread
            uint32_t n = 0, items[2] = {0, 0};             // stages, and items with a Q of each tile, so far
            bool ok = true;
            Item it;
            for (int k = 0; me.take<S::kCut>(k, it); ++k) {
                me.done_with(k);
                const int steps[2] = {it.steps(0, a.tokens), S::kTiles == 2 ? it.steps(1, a.tokens) : 0};
                const int most = max(steps[0], steps[1]);
                if (lane == 0 && ok) {
                    auto load = [&](int i, int v) {        // a step's keys or values
                        for (int p = 0; p < S::kParts && ok; ++p, ++n) {
                            const int s = n % S::kStages;
                            if (n >= S::kStages) ok = me.wait(&misc->kv_empty[s], n / S::kStages - 1);
                            if (!ok) break;
                            mbar_arrive_expect_tx(&misc->kv_full[s], S::kStage);
#pragma unroll
                            for (int c = 0; c < S::kPart / 64; ++c)
                                tma_load_3d(ring + s * S::kStage + c * kBox, v ? &vmap : &kmap, p * S::kPart + 64 * c, it.h,
                                            it.k_row + i * kKeys, &misc->kv_full[s]);
                        }
                    };
                    if (most > 0) load(0, 0);
#pragma unroll
                    for (int x = 0; x < S::kTiles; ++x) {  // Q behind the first keys, which have room earlier
                        if (!ok || steps[x] == 0) continue;
                        if (items[x] > 0) ok = me.wait(&misc->q_empty[x], items[x] - 1);
                        if (!ok) continue;
                        ++items[x];
                        mbar_arrive_expect_tx(&misc->q_full[x], (uint32_t)(D * 2 * a.tokens * a.group));
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(q_smem + (x * (D / 64) + c) * kBox, &qmap, 64 * c, it.h * a.group,
                                        it.q_row + it.tok0 + x * a.tokens, &misc->q_full[x]);
                    }
                    for (int i = 0; i < most && ok; ++i) {
                        if (S::kTiles == 1 && i + 1 < most) load(i + 1, 0);
                        if (ok) load(i, 1);
                        if (S::kTiles == 2 && ok && i + 1 < most) load(i + 1, 0);
                    }
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            }
            if (lane == 0) {                                   // copies in flight end before the CTA does
                for (uint32_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i)
                    if (!mbar_wait(&misc->kv_full[i % S::kStages], i / S::kStages & 1)) break;
                for (int x = 0; x < S::kTiles; ++x)
                    if (items[x] > 0) mbar_wait(&misc->q_full[x], (items[x] - 1) & 1);
            }
        } else if (warp == kItemWarp) {
            lay_out_items(
                me, a.batch, a.kv_heads, a.run, a.tokens, S::kTiles, Split{}, a.dealt,
                [&](int r, int& qs, int& qn) {
                    qs = a.q_start[r];
                    qn = (int)max((int64_t)0, min((int64_t)a.q_start[r + 1], a.total_q) - qs);
                },
                [&](int r, Item& it, bool) {
                    it.k_row = a.k_start[r];
                    it.len = it.cap = (int)max((int64_t)0, min((int64_t)a.k_start[r + 1], a.total_k) - it.k_row);
                });
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(misc->tmem_base, 512);
}

template <int D>
static dsa_status launch(Args a, int64_t longest, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    using S = Shape<D>;
    if (ensure_smem_limit(reinterpret_cast<const void*>(&prompt_kernel<D>), S::kSmem) != DSA_OK) return DSA_ERR_CUDA;
    const int64_t most = most_items(a.total_q, a.batch, a.kv_heads, a.tokens * S::kTiles);
    if (most > 0x7fff0000LL) return DSA_ERR_UNSUPPORTED;
    const unsigned G = (unsigned)std::min<int64_t>(device_sm_count(), most);
    if (!deals(most, longest, G)) a.dealt = nullptr;
    else DSA_CHECK(launch_pdl(clear_count, dim3(1), dim3(1), 0, s, 1, a.dealt));
    DSA_CHECK(launch_pdl(prompt_kernel<D>, dim3(G), dim3(S::kThreads), S::kSmem, s, 1, a, q, k, v));
    return DSA_OK;
}

static dsa_status check_prompt(const dsa_prompt* b) {
    if (!b || b->batch < 1 || b->max_q_len < 0 || b->max_k_len < 0 || b->total_q < 0 || b->total_k < 0 || b->reserved != 0) return DSA_ERR_INVALID_ARGUMENT;
    if (!b->q_start || !b->k_start) return DSA_ERR_INVALID_ARGUMENT;
    if (b->total_q > (int64_t)b->batch * b->max_q_len || b->total_k > (int64_t)b->batch * b->max_k_len) return DSA_ERR_INVALID_ARGUMENT;
    if (b->total_q > 0x7fffff00LL || b->total_k > 0x7fffff00LL || b->batch > 65535) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

}  // namespace prompt
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_prompt_attention_workspace_size(const dsa_prompt* b, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                                          size_t* bytes) {
    dsa_status vs = prompt::check_prompt(b);
    if (vs != DSA_OK) return vs;
    vs = kv8::check_shape(heads, kv_heads, head_dim);
    if (vs != DSA_OK) return vs;
    if (!bytes) return DSA_ERR_INVALID_ARGUMENT;
    *bytes = 256;
    return DSA_OK;
}

extern "C" dsa_status dsa_prompt_attention(const dsa_heads* q, const dsa_heads* k, const dsa_heads* v, const dsa_prompt* b,
                                           int32_t heads, int32_t kv_heads, int32_t head_dim, float softmax_scale, void* out,
                                           int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                                           void* stream) {
    dsa_status vs = prompt::check_prompt(b);
    if (vs != DSA_OK) return vs;
    vs = kv8::check_shape(heads, kv_heads, head_dim);
    if (vs != DSA_OK) return vs;
    if (out_dtype != DSA_DTYPE_BF16 && out_dtype != DSA_DTYPE_F32) return DSA_ERR_INVALID_ARGUMENT;
    if (!(softmax_scale > 0.f) || softmax_scale > kv8::kMostScale) return DSA_ERR_INVALID_ARGUMENT;
    if (b->total_q == 0) return DSA_OK;
    if (!q || !out || !ws || (b->total_k > 0 && (!k || !v))) return DSA_ERR_INVALID_ARGUMENT;
    const dsa_heads* kk = b->total_k > 0 ? k : q;           // without keys nothing is read of them
    const dsa_heads* vv = b->total_k > 0 ? v : q;
    struct { const dsa_heads* h; int64_t heads, rows; } in[3] = {{q, heads, b->total_q}, {kk, kv_heads, b->total_k}, {vv, kv_heads, b->total_k}};
    for (auto& i : in) {
        if ((vs = kv8::check_heads(i.h)) != DSA_OK) return vs;
        if ((i.heads > 1 && i.h->head_stride == 0) || (i.rows > 1 && i.h->token_stride == 0)) return DSA_ERR_UNSUPPORTED;
        if (i.h->head_stride >= 1LL << 38 || i.h->token_stride >= 1LL << 38) return DSA_ERR_UNSUPPORTED;
    }
    if (!aligned16(out) || !aligned16(ws)) return DSA_ERR_ALIGNMENT;
    if (ws_bytes < 256) return DSA_ERR_WORKSPACE_TOO_SMALL;
    prompt::Args a = {};
    a.v = static_cast<const uint16_t*>(vv->data);
    a.v_tok = vv->token_stride, a.v_head = vv->head_stride;
    a.q_start = b->q_start, a.k_start = b->k_start;
    a.total_q = b->total_q, a.total_k = b->total_k;
    a.batch = b->batch;
    a.kv_heads = kv_heads, a.group = heads / kv_heads;
    a.tokens = 128 / a.group;
    a.run = gtc::heads_of_run(kv_heads, (int64_t)b->max_k_len * head_dim * 4);
    a.scale = softmax_scale * 1.44269504088896341f;
    a.out = out;
    a.out_f32 = out_dtype == DSA_DTYPE_F32;
    a.lse = lse;
    a.dealt = static_cast<uint32_t*>(ws);
    a.wait_ns = wait_limit_ns();
    a.st = dev_status;
    CUtensorMap qm, km, vm;
    const int64_t rows = std::max<int64_t>(1, b->total_k);
    if (!gtc::make_heads_map(q, head_dim, heads, b->total_q, (unsigned)a.group, (unsigned)a.tokens, &qm) ||
        !gtc::make_heads_map(kk, head_dim, kv_heads, rows, 1, gtc::kKeys, &km) || !gtc::make_heads_map(vv, head_dim, kv_heads, rows, 1, gtc::kKeys, &vm))
        return DSA_ERR_CUDA;
    const cudaStream_t s = as_stream(stream);
    if (head_dim == 64) return prompt::launch<64>(a, b->max_k_len, qm, km, vm, s);
    if (head_dim == 128) return prompt::launch<128>(a, b->max_k_len, qm, km, vm, s);
    return prompt::launch<256>(a, b->max_k_len, qm, km, vm, s);
}
