// Device helpers that the tensor-core attention kernels on grouped heads share:
// their items of work, MMAs with an operand in TMEM, packed fp32 arithmetic.
#pragma once
#include <algorithm>

#include "dsa_internal.cuh"
#include "kv8.cuh"
#include "mla_common.cuh"
#include "sm100.cuh"

namespace dsa {
namespace gtc {

using namespace sm100;

constexpr int kKeys = 128;                                 // of a step
constexpr int kBox = kKeys * 128;                          // bytes of 128 rows of 64 16-bit values

// What a CTA does at a time: neighbouring tokens of a sequence with the heads of one
// key head, in one or two tiles of 128 rows.
struct Item {
    int32_t q_row, tok0, n;     // the sequence's first row of q, the item's first token, the sequence's tokens; n < 0: no more items
    int32_t k_row, len, h;      // its first row of k (of a paged cache: its request), the sequence's keys, the key head
    int32_t cap;                // keys that there are
    int32_t from, to;           // the steps of this piece of it: [from, to)
    int32_t slot;               // of the piece's partial outputs; -1: it is whole
    int32_t pad;
    // keys that token t sees
    __device__ __forceinline__ int see(int t) const { return max(0, min(cap, len - n + t + 1)); }
    // tokens of tile x, and its steps, of the whole item and of this piece
    __device__ __forceinline__ int count(int x, int tokens) const { return max(0, min(tokens, n - tok0 - x * tokens)); }
    __device__ __forceinline__ int all_steps(int x, int tokens) const {
        const int c = count(x, tokens);
        const int last = c ? see(tok0 + x * tokens + c - 1) : 0;
        return last / kKeys + (last % kKeys != 0);         // (rounding up first would pass 2^31 with the longest contexts)
    }
    __device__ __forceinline__ int steps(int x, int tokens) const { return max(0, min(all_steps(x, tokens), to) - from); }
    // the first step that some row of the item sees in part or not at all, counted from the piece's first
    __device__ __forceinline__ int masked_from() const { return see(tok0) / kKeys - from; }
    // The first step whose values tile x's threads clean: of masked steps, the first tile's that it has, the second's the others.
    __device__ __forceinline__ int cleans_from(int x, int tokens) const { return x == 0 ? masked_from() : max(masked_from(), steps(0, tokens)); }
};

// MMAs and commits of one lane, `lead`, of a warp that runs them together: in control flow
// that the whole warp takes, the operands are kept and added to in uniform registers, and an
// MMA is issued every 64 cycles (128 x 128 x 16, as fast as it runs).  Behind a branch that
// one lane takes each operand is moved there for each MMA: 100 cycles, and the thread that
// issues bounds the kernel (1 x 8192 tokens of 64 heads: 938 us).
// D[tmem] (+)= A[smem] B[smem].
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead) : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A holds two 16-bit values a column.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead) : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
    asm volatile("{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
                 ::"r"(smem_addr(bar)), "r"(lead) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// 32 bytes, a sector of memory: in one store where the address allows it.
__device__ __forceinline__ void store_32_bytes(void* to, bool wide, const uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
    } else {
        static_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
// 32 dims of an output row, of outputs that begin at a multiple of 16 bytes.  A thread holds a
// row, so that a warp's stores go to 32 places: half as many as with 16 bytes each.
__device__ __forceinline__ void write_32(void* out, int f32, int64_t at, const float (&y)[32]) {
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    uint32_t w[8];
    if (f32) {
        float* to = static_cast<float*>(out) + at;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(y[j + e]);
            store_32_bytes(to + j, wide, w);
        }
    } else {
        uint16_t* to = static_cast<uint16_t*>(out) + at;
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack_bf2(y[j + 2 * e], y[j + 2 * e + 1]);
            store_32_bytes(to + j, wide, w);
        }
    }
}
// O's TMEM columns [o, o + D) of the warp's rows times f.
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t o_tmem, float f) {
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(o_tmem + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        tmem_st_32x32b_x32(o_tmem + c, o);
    }
}

// Items of a call, at most; the kernels count them in 32 bits.
inline int64_t most_items(int64_t total_q, int batch, int kv_heads, int per) { return std::min(total_q, total_q / per + batch) * kv_heads; }

// Key heads whose items are laid out together: as many as have their keys and values in half of
// the L2, where the CTAs that work on them find them.  2 x 4096 tokens of 64 key heads of 256
// dims (270 MB a prompt) 1039 us with all heads together, which read 2.0 GB of 0.4 from DRAM,
// 939 in runs of 64 MB, 951 of 32, 965 of 16; 8 key heads of 128 dims on 8192 tokens (34 MB)
// 797 in one run and 807 in runs of 16 MB.
constexpr int64_t kRunBytes = 64 << 20;
inline int heads_of_run(int kv_heads, int64_t bytes) { return (int)std::max<int64_t>(1, std::min<int64_t>(kv_heads, kRunBytes / std::max<int64_t>(1, bytes))); }

// Which calls deal their items out as they go: those of many rounds, and those whose CTAs have
// many steps each.  The launch that clears the count takes 2 us, and an item that is known late
// has its first copies late.  Dealt and not, in us: 16 prompts of up to 512 tokens (14 rounds)
// 76.4, 81.9; 2 x 4096 tokens of 256 dims (27 rounds) 939, 972; 2048 tokens over 16384 in the cache (3.4
// rounds, 430 steps a CTA) 993, 1041; 4 x 2048 tokens of 64 dims (3.5 rounds, 55 steps) 68.8, 64.8.
// Between these, in a graph: 2 x 4096 of 2 key heads (3.4 rounds, 108 steps) 129, 148; 8 x 512 (6.7
// rounds) 68.8, 69.5; 2 x 1024 (3.4, 27) 48.7, 52.1 and 4 x 2048 of 64 dims of equal lengths (3.4, 54) 72.4,
// 78.4, which the rule has wrong; 1 x 4096 of 2 key heads (1.7, 54) 77.0, 57.8.
constexpr int kDealtRounds = 4, kDealtSteps = 100;
inline bool deals(int64_t items, int64_t longest, int64_t ctas) {
    return items > ctas && (items > kDealtRounds * ctas || items * (longest / kKeys) > kDealtSteps * ctas);
}
static __global__ void clear_count(uint32_t* dealt) {
    pdl_wait();
    pdl_trigger();
    *dealt = 0;
}

// bf16 rows of heads as [rows, heads, dim], boxes of 64 dims x bh heads x br rows.
bool make_heads_map(const dsa_heads* h, int dim, int64_t heads, int64_t rows, unsigned bh, unsigned br, CUtensorMap* out);

template <int R> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// ---------------------------------------------------------------- the pipeline
// Barriers and items of a CTA.  A stage of the ring holds 128 keys x up to 128 dims of a
// step's keys or values; the stages of an item are its steps' keys and values in turn.
constexpr int kMaxStages = 10;
constexpr int kItems = 2;                                  // laid out ahead
constexpr int kMasked = 4;                                 // steps of an item that some rows see in part, at most
// Barriers of the first tile's masked steps, in turn: its softmax is up to two steps ahead of the second tile's MMAs,
// and a barrier must not be in its next but one phase when a wait for one is made.
constexpr int kCleans = 4;

struct Pipe {
    uint64_t q_full[2], q_empty[2];                        // by tile
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
    uint64_t s_full[2], o_done[2];                         // by S, by tile
    uint64_t p_full[2][2];                                 // by S: the first 64 keys' P, the others'
    uint64_t turn[2];                                      // by tile: its warp may issue a step's last MMAs
    uint64_t here;                                         // with one tile: a masked step's values are there
    uint64_t clean[kCleans];                               // with two: ... and are finite
    uint64_t drain[2];
    uint64_t item_full[kItems], item_empty[kItems];
    Item item[kItems];
    uint32_t odd[kItems][kMasked][4];                      // keys of an item's masked steps whose values are not all finite
    uint32_t any_odd[kItems];
    uint32_t tmem_base;
    int32_t abort;
};

// One role's view of it.  Every wait is bounded; one that gives up is recorded and ends the
// CTA's work.  What it was for may still be under way: nothing is freed behind it.
struct Role {
    Pipe* m;
    uint64_t wait_ns;
    int32_t* st;
    int warp, lane;
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
        const volatile int32_t* gone = &m->abort;
        if (mbar_test_wait(bar, parity & 1)) return true;
        // Without a time to sleep: a thread that is to be suspended for long wakes late, and a step's waits
        // follow one another (1 x 8192 tokens: 812 us with 20 us of it).
        const uint64_t t0 = wait_ns ? globaltimer_ns() : 0;
        for (uint32_t it = 1; wait_ns != 0; ++it) {
            if (mbar_try_wait(bar, parity & 1)) return true;
            if ((it & 255u) == 0u && (*gone || globaltimer_ns() - t0 > wait_ns)) break;
        }
        record_error(st, DSA_DEVERR_TIMEOUT, warp);
        *const_cast<volatile int32_t*>(gone) = 1;
        return false;
    }
    __device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) const { return __all_sync(0xffffffffu, wait(bar, parity)); }
    // Item k of the CTA, read by a whole warp; false when there is none.
    // (Cut: items may be pieces.)
    template <bool Cut> __device__ __forceinline__ bool take(int k, Item& it) const {
        if (!wait_all(&m->item_full[k % kItems], k / kItems)) return false;
        it = m->item[k % kItems];
        if (!Cut) it.from = 0, it.to = INT32_MAX, it.slot = -1;
        return it.n >= 0;
    }
    __device__ __forceinline__ void done_with(int k) const {
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->item_empty[k % kItems]);
    }
};

template <int I> struct Constant { static constexpr int value = I; };

// A place in the ring: stage and the parity of its phase.
template <class S>
struct Place {
    uint32_t stage = 0, phase = 0;
    __device__ __forceinline__ void next(int by = 1) {
        stage += by;
        if (stage >= S::kStages) stage -= S::kStages, phase ^= 1;
    }
    __device__ __forceinline__ Place then(int by) const {
        Place p = *this;
        p.next(by);
        return p;
    }
};

// The stages of an item, in the order in which the MMAs take them: the first step's keys, then
// of each step its values and the next one's keys; with one tile (two S) the next one's keys
// come first, as their S is formed while this step's P is.  (In the other order, the next keys'
// copy waits for values that are not read before it: 2 x 4096 tokens of 256 dims 1356 us.)
template <class S>
struct Ring {
    Place<S> at;
    __device__ __forceinline__ Place<S> take() {
        const Place<S> p = at;
        at.next(S::kParts);
        return p;
    }
    // values of a step, and keys of the next if there are more
    __device__ __forceinline__ void step(bool more, Place<S>& values, Place<S>& keys) {
        if (S::kTiles == 1 && more) keys = take();
        values = take();
        if (S::kTiles == 2 && more) keys = take();
    }
};

// The warp that issues tile x's MMAs.  S: kDim, kTiles, kPart, kParts, kStage, kStages, s(i) and
// o(i) (TMEM columns), kIdQK and kIdPV, kValuesMn (values lie with their dims side by side: an
// MN-major operand; else their tokens), kTurns, kCut (items may be pieces), kCleans (the
// softmax threads take values that are not finite out of masked steps, before MMAs read them).
// A warp a tile, as its own waits and the time that operands take to uniform registers (an MMA of
// 128 x 128 x 16 runs 64 cycles and is issued in 80 to 100) would bound the kernel if one warp
// issued for both.  With kTurns the tiles take turns with a step's last MMAs, which keeps them out
// of step: one's softmax runs beside the other's MMAs (1 x 8192 tokens: 892 us without, 812 with).
// TMEM is the kernel's alone: all 512 columns, from column 0.
template <class S>
__device__ __forceinline__ void issue_mmas(const Role& me, int x, uint32_t q0, uint32_t r0, int tokens) {
    static_assert(S::kStages <= kMaxStages && 2 * S::kParts < S::kStages, "a step's values and the next one's keys are held at once");
    Pipe* m = me.m;
    const uint32_t lead = me.lane == 0;
    uint32_t t = 0, items = 0, turns = 0, cleaned = 0;     // the tile's steps, items with a Q, turns and the first tile's masked steps, so far
    Ring<S> ring;
    bool ok = true;
    Item it;
    for (int k = 0; ok && me.take<S::kCut>(k, it); ++k) {
        me.done_with(k);
        auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };      // so that the compiler knows it for the warp's
        const int steps = same(it.steps(x, tokens));
        const int most = S::kTiles == 2 ? same(max(it.steps(0, tokens), it.steps(1, tokens))) : steps;
        const int masked = S::kCleans ? same(it.masked_from()) : 0, cleaned_to = S::kCleans && S::kTiles == 2 && x == 1 ? same(it.steps(0, tokens)) : 0;
        auto full = [&](Place<S> p) {
#pragma unroll
            for (int i = 0; i < S::kParts; ++i, p.next()) ok = ok && me.wait_all(&m->kv_full[p.stage], p.phase);
            tc_fence_after();
        };
        auto free_stages = [&](Place<S> p) {
#pragma unroll
            for (int i = 0; i < S::kParts; ++i, p.next())
                if (ok) commit(lead, &m->kv_empty[p.stage]);
        };
        auto qk = [&](int s, Place<S> p) {                 // S[s] = Q[x] K^T
            uint32_t part[S::kParts];
#pragma unroll
            for (int i = 0; i < S::kParts; ++i, p.next()) part[i] = r0 + p.stage * S::kStage;
            const uint32_t d = S::s(0) + 128 * s;
#pragma unroll
            for (int c = 0; c < S::kDim / 64; ++c) {
                const uint64_t dq = desc_kmajor_sw128(q0 + (x * (S::kDim / 64) + c) * kBox);
                const uint64_t dk = desc_kmajor_sw128(part[c * 64 / S::kPart] + c * 64 % S::kPart / 64 * kBox);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma_ss(lead, d, dq + (uint64_t)(kk * 32 >> 4), dk + (uint64_t)(kk * 32 >> 4), S::kIdQK, c + kk > 0);
            }
            commit(lead, &m->s_full[s]);
        };
        // 64 keys of O[x] (+)= P[s] V: half h
        auto pv = [&](int s, Place<S> p, int h, bool first) {
            const uint32_t a = S::s(0) + 128 * s + 32 * h;
#pragma unroll
            for (int i = 0; i < S::kParts; ++i, p.next()) {
                // 16 keys on: 16 rows of 128 bytes, or 32 bytes in the rows of 64 keys
                const uint32_t v0 = r0 + p.stage * S::kStage + h * (S::kValuesMn ? 4 * 2048 : S::kPart * 128);
                const uint64_t dv = S::kValuesMn ? desc_mnmajor_sw128(v0, kBox) : desc_kmajor_sw128(v0);
                const uint32_t d = S::o(0) + 128 * x + i * S::kPart;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts(lead, d, a + kk * 8, dv + (uint64_t)((S::kValuesMn ? kk * 2048 : kk * 32) >> 4), S::kIdPV, kk > 0 || !first);
            }
        };
        if (steps > 0) ok = ok && me.wait_all(&m->q_full[x], items++);
        Place<S> vp, np;
        if (ok && most > 0) {
            np = ring.take();
            full(np);
            if (ok && steps > 0) qk(S::kTiles == 2 ? x : t & 1, np);
            free_stages(np);
            if (ok && steps == 1) commit(lead, &m->q_empty[x]);
        }
        for (int i = 0; i < most && ok; ++i) {
            const bool more = i + 1 < most;
            ring.step(more, vp, np);
            if constexpr (S::kTiles == 2) {
                full(vp);
                if (more) full(np);
                if (S::kCleans && i >= masked && i < cleaned_to) {     // the second tile's, by the first one's threads
                    ok = ok && me.wait_all(&m->clean[cleaned % kCleans], cleaned / kCleans);
                    ++cleaned;
                }
                if (i < steps) {
                    ok = ok && me.wait_all(&m->p_full[x][0], t);
                    tc_fence_after();
                    if (ok) pv(x, vp, 0, i == 0);
                    ok = ok && me.wait_all(&m->p_full[x][1], t);
                    tc_fence_after();
                    if (S::kTurns) ok = ok && me.wait_all(&m->turn[x], turns);
                    if (ok) {
                        pv(x, vp, 1, false);
                        commit(lead, &m->o_done[x]);
                        if (i + 1 < steps) qk(x, np);
                    }
                    ++t;
                } else if (S::kTurns) {
                    ok = ok && me.wait_all(&m->turn[x], turns);
                }
                ++turns;
                if (S::kTurns && ok && lead) mbar_arrive(&m->turn[1 - x]);
                // a tile with fewer steps than the other lets the stages go by
                free_stages(vp);
                if (more) free_stages(np);
            } else {
                // with two S, the next step's is formed while this one's P is
                if (more) {
                    full(np);
                    if (ok) qk((t + 1) & 1, np);
                    free_stages(np);
                }
                full(vp);
                if (S::kCleans && i >= masked && ok && lead) mbar_arrive(&m->here);
                for (int h = 0; h < 2; ++h) {
                    ok = ok && me.wait_all(&m->p_full[t & 1][h], t >> 1);
                    tc_fence_after();
                    if (ok) pv(t & 1, vp, h, i == 0 && h == 0);
                }
                if (ok) commit(lead, &m->o_done[x]);
                free_stages(vp);
                ++t;
            }
            if (ok && i + 2 == steps) commit(lead, &m->q_empty[x]);
        }
    }
    __syncwarp();
    commit(lead, &m->drain[x]);                            // MMAs in flight end before TMEM is given back
    mbar_wait(&m->drain[x], 0);
}

// Items are dealt out to the CTAs in rounds.  The last round's, which would leave CTAs without
// work, may be cut along the keys into equal pieces, as many as fill the CTAs best, that leave
// partial outputs for a second kernel: one request's 512 items of 128 steps on 152 CTAs take
// 3.4 rounds so and 4 else, and a chunk of 100 tokens over a long cache has few items at all.
constexpr int kMinSteps = 8;                               // of a piece: beginning and end cost about five steps
constexpr int kMaxPieces = 160;

struct Split {
    float* part_o;              // [slots][rows of an item][D]: normalised
    float2* part_ml;            // [slots][rows of an item]: reference in log2 units, sum
    struct Cut* cut;            // [CTAs]: the last round's items
    int slots;                  // 0: no item is cut
    int ctas;
};
struct Cut {
    int32_t q_row, tok0, count, h, slot, pieces, pad[2];   // first row of q and token, tokens; pieces < 2: nothing to join
};

// How many pieces each of `rest` items is cut into: the smallest number of CTAs' turns, in
// units of an item.  Asked of a whole warp.
__device__ __forceinline__ uint32_t pieces_of(uint32_t rest, uint32_t ctas, uint32_t slots) {
    if (rest == 0) return 1;
    const uint32_t most = min(slots / rest, (uint32_t)kMaxPieces);
    uint32_t best = 0xffffffffu;
    for (uint32_t p = 1 + (threadIdx.x & 31); p <= most; p += 32) best = min(best, ((rest * p + ctas - 1) / ctas * 65536u / p) << 8 | p);
    best = __reduce_min_sync(0xffffffffu, best);
    return best == 0xffffffffu ? 1 : best & 255u;
}
static_assert(kMaxPieces < 256, "pieces in a byte");

// The items of a call in order, 32 requests at a time, one a lane; asked of a whole warp, for
// items in ascending order.
template <class Rows>
struct Finder {
    Rows rows;
    int batch, kv_heads, run, per, lane;
    int c0 = -32;
    uint32_t base = 0, all = 0;                            // items before the 32 requests, and theirs (the host bounds them)
    uint32_t upto = 0;                                     // and of those up to the lane's
    int qs = 0, qn = 0, blocks = 0;
    __device__ __forceinline__ bool next() {
        if (c0 + 32 >= batch) return false;
        base += all;
        c0 += 32;
        qs = qn = 0;
        if (c0 + lane < batch) rows(c0 + lane, qs, qn);
        blocks = (qn + per - 1) / per;
        upto = (uint32_t)(blocks * kv_heads);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        all = __shfl_sync(0xffffffffu, upto, 31);
        return true;
    }
    // Item i without its keys; returns its request, -1 when there is none.
    __device__ __forceinline__ int find(uint32_t i, Item& it) {
        it = Item{};
        it.n = -1;
        while (i >= base + all)
            if (!next()) return -1;
        const int at = __ffs(__ballot_sync(0xffffffffu, i < base + upto)) - 1;
        const int b = __shfl_sync(0xffffffffu, blocks, at);
        const uint32_t j = i - base - __shfl_sync(0xffffffffu, upto - (uint32_t)(blocks * kv_heads), at);
        it.q_row = __shfl_sync(0xffffffffu, qs, at);
        it.n = __shfl_sync(0xffffffffu, qn, at);
        const int first = (int)(j / (uint32_t)(b * run)) * run, heads = min(run, kv_heads - first);
        const uint32_t e = j - (uint32_t)(b * first);
        it.tok0 = (b - 1 - (int)(e / (uint32_t)heads)) * per;
        it.h = first + (int)(e % (uint32_t)heads);
        return c0 + at;
    }
};

// Lays out the CTA's items, of `tiles` tiles of `tokens` tokens: `rows(r, qs, qn)` gives a
// request's first row and tokens, `keys(r, it, first)` sets an item's keys (first: it is the
// item's first piece).  The items of a request come in runs of `run` heads, longest first.  A
// CTA's first item is its number's; the others go to the CTAs as they get there, by the count
// `dealt` (0 at the start), or, without one, there and back over them.  What an item's outputs
// are does not depend on who takes it.
template <class Rows, class Keys>
__device__ __forceinline__ void lay_out_items(const Role& me, int batch, int kv_heads, int run, int tokens, int tiles, const Split& split, uint32_t* dealt, Rows rows, Keys keys) {
    Pipe* m = me.m;
    const int per = tokens * tiles;
    uint32_t whole = 0xffffffffu, pieces = 1;              // items before the last round; pieces of its items
    auto pieces_now = [&](const Item& it) {                // of one of them
        int most = it.all_steps(0, tokens);
        if (tiles == 2) most = max(most, it.all_steps(1, tokens));
        return max(1, min((int)pieces, most / kMinSteps));
    };
    if (split.slots > 0) {
        Finder<Rows> count{rows, batch, kv_heads, run, per, me.lane};
        while (count.next()) {}
        const uint32_t items = count.base + count.all, rest = items % gridDim.x;
        whole = items - rest;
        pieces = pieces_of(rest, gridDim.x, (uint32_t)split.slots);
        // The joining kernel's list: written before any wait, so that it is there whatever else happens.
        Cut cut = {};
        if (blockIdx.x < rest) {
            Finder<Rows> one{rows, batch, kv_heads, run, per, me.lane};
            Item it;
            const int r = one.find(whole + blockIdx.x, it);
            if (r >= 0) {
                keys(r, it, false);
                cut.q_row = it.q_row, cut.tok0 = it.tok0, cut.count = min(per, it.n - it.tok0), cut.h = it.h;
                cut.slot = (int)(blockIdx.x * pieces), cut.pieces = pieces_now(it);
            }
        }
        if (me.lane == 0) split.cut[blockIdx.x] = cut;
    }
    Finder<Rows> finder{rows, batch, kv_heads, run, per, me.lane};
    uint32_t turn = 0;
    for (uint32_t k = 0;; ++k) {
        if (k >= kItems && !me.wait_all(&m->item_empty[k % kItems], k / kItems - 1)) break;
        Item it;
        int r;
        bool nothing;
        do {
            uint32_t i = blockIdx.x;
            if (turn > 0) {
                if (dealt) i = __shfl_sync(0xffffffffu, me.lane == 0 ? gridDim.x + atomicAdd(dealt, 1u) : 0u, 0);
                else i = turn * gridDim.x + (turn & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            }
            ++turn;
            const uint32_t piece = i < whole ? 0 : (i - whole) % pieces;
            r = finder.find(i < whole ? i : whole + (i - whole) / pieces, it);
            it.from = 0, it.to = INT32_MAX, it.slot = -1;
            nothing = false;
            if (r < 0) break;
            keys(r, it, piece == 0);
            if (i >= whole && pieces > 1) {
                const int n = pieces_now(it);
                nothing = (int)piece >= n;
                if (n > 1) {
                    const int64_t most = max(it.all_steps(0, tokens), tiles == 2 ? it.all_steps(1, tokens) : 0);
                    it.from = (int)(most * piece / n), it.to = (int)(most * (piece + 1) / n);
                    it.slot = (int)(i - whole);
                }
            }
        } while (nothing);
        if (me.lane < kMasked * 4) m->odd[k % kItems][me.lane >> 2][me.lane & 3] = 0;
        __syncwarp();
        if (me.lane == 0) {
            m->item[k % kItems] = it;
            m->any_odd[k % kItems] = 0;
            mbar_arrive(&m->item_full[k % kItems]);
        }
        if (r < 0) break;
    }
}

// Joins the partial outputs of the items that were cut: (R, l) of a piece: out = sum 2^R l
// out_piece / sum 2^R l.  Four warps a row, each a quarter of its pieces, as what bounds it
// is the loads' latency (100 pieces one after another by one warp: 80 us for 100 tokens over
// 100,000); a lane takes D / 32 dims.
constexpr int kJoinRows = 2, kJoinWarps = 4;               // rows of a block at a time, warps of a row
template <int D>
__global__ void __launch_bounds__(kJoinRows * kJoinWarps * 32)
join_kernel(const __grid_constant__ Split split, int group, int kv_heads, int item_rows, void* out, int out_f32, float* lse) {
    pdl_wait();
    pdl_trigger();
    __shared__ float part[kJoinRows][kJoinWarps][D + 1];
    const Cut cut = split.cut[blockIdx.x];
    if (cut.pieces < 2) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp / kJoinWarps, w = warp % kJoinWarps;
    const int tokens = 128 / group;                        // of a tile
    for (int row0 = blockIdx.y * kJoinRows; row0 < item_rows; row0 += gridDim.y * kJoinRows) {
        const int row = row0 + mine, tok = row / 128 * tokens + row % 128 / group;
        const bool live = row % 128 < tokens * group && tok < cut.count;
        float top = -INFINITY, total = 0.f, v[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) v[j] = 0.f;
        if (live) {
            const float2* ml_at = split.part_ml + (int64_t)cut.slot * item_rows + row;
            const float* o_at = split.part_o + ((int64_t)cut.slot * item_rows + row) * D + lane * (D / 32);
            for (int p = lane; p < cut.pieces; p += 32) {
                const float2 ml = __ldcg(ml_at + (int64_t)p * item_rows);
                if (ml.y != 0.f) top = fmaxf(top, ml.x);   // 0: the row sees nothing there
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll 8
            for (int p = w; p < cut.pieces; p += kJoinWarps) {
                const float2 ml = __ldcg(ml_at + (int64_t)p * item_rows);
                float y[D / 32];
#pragma unroll
                for (int j = 0; j < D / 32; j += 2) {
                    const float2 two = __ldcg(reinterpret_cast<const float2*>(o_at + (int64_t)p * item_rows * D + j));
                    y[j] = two.x, y[j + 1] = two.y;
                }
                const float f = ml.y != 0.f ? ml.y * exp2f(ml.x - top) : 0.f;
                total += f;
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    if (ml.y != 0.f) v[j] = fmaf(f, y[j], v[j]);               // (a NaN counts whatever its share)
            }
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) part[mine][w][lane + 32 * j] = v[j];
        if (lane == 0) part[mine][w][D] = total;
        __syncthreads();
        if (live && w == 0) {
#pragma unroll
            for (int i = 1; i < kJoinWarps; ++i) {
                total += part[mine][i][D];
#pragma unroll
                for (int j = 0; j < D / 32; ++j) v[j] += part[mine][i][lane + 32 * j];
            }
            const float inv = total != 0.f ? 1.f / total : 0.f;
            const int64_t at = (int64_t)(cut.q_row + cut.tok0 + tok) * (kv_heads * group) + cut.h * group + row % 128 % group;
#pragma unroll
            for (int j = 0; j < D / 32; j += 2) {
                const int64_t to = at * D + lane * (D / 32) + j;
                if (out_f32) *reinterpret_cast<float2*>(static_cast<float*>(out) + to) = make_float2(v[j] * inv, v[j + 1] * inv);
                else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + to) = pack_bf2(v[j] * inv, v[j + 1] * inv);
            }
            if (lse && lane == 0) lse[at] = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.69314718055994531f;
        }
        __syncthreads();
    }
}

}  // namespace gtc
}  // namespace dsa
