// Device helpers that the tensor-core attention kernels on grouped heads share:
// their items of work, MMAs with an operand in TMEM, packed fp32 arithmetic.
#pragma once
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
    int32_t cap, pad;           // keys that there are
    // keys that token t sees
    __device__ __forceinline__ int see(int t) const { return max(0, min(cap, len - n + t + 1)); }
    // tokens of tile x, and its steps
    __device__ __forceinline__ int count(int x, int tokens) const { return max(0, min(tokens, n - tok0 - x * tokens)); }
    __device__ __forceinline__ int steps(int x, int tokens) const {
        const int c = count(x, tokens);
        return c ? (see(tok0 + x * tokens + c - 1) + kKeys - 1) / kKeys : 0;
    }
    // the first step that some row of the item sees in part or not at all
    __device__ __forceinline__ int masked_from() const { return see(tok0) / kKeys; }
};

// D[tmem] (+)= A[tmem] B[smem]: A holds two 16-bit values a column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
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
// 32 dims of an output row.
__device__ __forceinline__ void write_32(void* out, int f32, int64_t at, const float (&y)[32]) {
    if (f32) {
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
        for (int j = 0; j < 8; ++j) to[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
    } else {
        uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            to[j] = make_uint4(pack_bf2(y[8 * j], y[8 * j + 1]), pack_bf2(y[8 * j + 2], y[8 * j + 3]),
                               pack_bf2(y[8 * j + 4], y[8 * j + 5]), pack_bf2(y[8 * j + 6], y[8 * j + 7]));
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

// bf16 rows of heads as [rows, heads, dim], boxes of 64 dims x bh heads x br rows.
bool make_heads_map(const dsa_heads* h, int dim, int64_t heads, int64_t rows, unsigned bh, unsigned br, CUtensorMap* out);

template <int R> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// ---------------------------------------------------------------- the pipeline
// Barriers and items of a CTA.  A stage of the ring holds 128 keys x up to 128 dims of a
// step's keys or values; the stages of an item are its steps' keys and values in turn.
constexpr int kMaxStages = 10;
constexpr int kItems = 2;                                  // laid out ahead
constexpr int kCleaned = 8;                                // masked steps that may be looked through before their MMA: more than the ring holds
constexpr int kMasked = 4;                                 // steps of an item that some rows see in part, at most

struct Pipe {
    uint64_t q_full, q_empty;
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
    uint64_t s_full[2], p_full[2], o_done[2];
    uint64_t v_clean[kCleaned], drain;
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
        if (kv8::wait_for(bar, parity & 1, gone, wait_ns)) return true;
        record_error(st, DSA_DEVERR_TIMEOUT, warp);
        *const_cast<volatile int32_t*>(gone) = 1;
        return false;
    }
    __device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) const { return __all_sync(0xffffffffu, wait(bar, parity)); }
    // Item k of the CTA, read by a whole warp; false when there is none.
    __device__ __forceinline__ bool take(int k, Item& it) const {
        if (!wait_all(&m->item_full[k % kItems], k / kItems)) return false;
        it = m->item[k % kItems];
        return it.n >= 0;
    }
    __device__ __forceinline__ void done_with(int k) const {
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->item_empty[k % kItems]);
    }
};

// S: kDim, kTiles, kPart, kParts, kStage, kStages, s(i) and o(i) (TMEM columns), kIdQK and
// kIdPV, kValuesMn (values lie with their dims side by side: an MN-major operand; else their
// tokens), kCleans (masked steps' values are looked through first).
template <class S>
__device__ __forceinline__ void issue_mmas(const Role& me, uint32_t tmem, uint32_t q0, uint32_t r0, int tokens) {
    Pipe* m = me.m;
    uint32_t n = 0, cleaned = 0, t[2] = {0, 0};            // stages, masked steps and the tiles' steps so far
    uint32_t items = 0;                                    // with a Q
    bool ok = true;
    Item it;
    for (int k = 0; me.take(k, it); ++k) {
        me.done_with(k);
        const int steps[2] = {it.steps(0, tokens), S::kTiles == 2 ? it.steps(1, tokens) : 0};
        const int most = max(steps[0], steps[1]), masked = it.masked_from();
        if (me.lane == 0 && most > 0 && ok) {
            // stage of part p of step i's keys (v = 0) or values (v = 1)
            auto stage = [&](int i, int v, int p) { return (n + (2 * i + v) * S::kParts + p) % S::kStages; };
            auto full = [&](int i, int v) {
#pragma unroll
                for (int p = 0; p < S::kParts; ++p)
                    ok = ok && me.wait(&m->kv_full[stage(i, v, p)], (n + (2 * i + v) * S::kParts + p) / S::kStages);
                tc_fence_after();
            };
            auto free_stages = [&](int i, int v) {
#pragma unroll
                for (int p = 0; p < S::kParts && ok; ++p) mma_commit(&m->kv_empty[stage(i, v, p)]);
            };
            auto free_q = [&]() {
                if (ok) mma_commit(&m->q_empty);
            };
            auto qk = [&](int x, int s, int i) {           // S[s] = Q[x] K_i^T
#pragma unroll
                for (int c = 0; c < S::kDim / 64; ++c) {
                    const uint64_t dq = desc_kmajor_sw128(q0 + (x * (S::kDim / 64) + c) * kBox);
                    const uint64_t dk = desc_kmajor_sw128(r0 + stage(i, 0, c * 64 / S::kPart) * S::kStage + c * 64 % S::kPart / 64 * kBox);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16(tmem + S::s(s), dq + (uint64_t)(kk * 32 >> 4), dk + (uint64_t)(kk * 32 >> 4), S::kIdQK, c + kk > 0);
                }
                mma_commit(&m->s_full[s]);
            };
            auto pv = [&](int x, int s, int i) {           // O[x] += P[s] V_i
#pragma unroll
                for (int p = 0; p < S::kParts; ++p) {
                    const uint32_t v0 = r0 + stage(i, 1, p) * S::kStage;
                    const uint64_t dv = S::kValuesMn ? desc_mnmajor_sw128(v0, kBox) : desc_kmajor_sw128(v0);
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk) {
                        // 16 keys on: 16 rows of 128 bytes, or 32 bytes in the rows of 64 keys
                        const uint64_t at = S::kValuesMn ? kk * 2048 : kk / 4 * (S::kPart * 128) + kk % 4 * 32;
                        mma_f16_ts(tmem + S::o(x) + p * S::kPart, tmem + S::s(s) + kk * 8, dv + (at >> 4), S::kIdPV, i > 0 || kk > 0);
                    }
                }
                mma_commit(&m->o_done[x]);
            };
            auto values = [&](int i) {
                full(i, 1);
                if (S::kCleans && i >= masked) {
                    ok = ok && me.wait(&m->v_clean[cleaned % kCleaned], cleaned / kCleaned);
                    ++cleaned;
                }
            };
            ok = ok && me.wait(&m->q_full, items++);
            full(0, 0);
            if constexpr (S::kTiles == 2) {
                for (int x = 0; x < 2 && ok; ++x)
                    if (steps[x] > 0) qk(x, x, 0);
                free_stages(0, 0);
                if (most == 1) free_q();
                for (int i = 0; i < most && ok; ++i) {
                    values(i);
                    bool have = false;                     // the next keys
                    for (int x = 0; x < 2 && ok; ++x) {
                        if (i >= steps[x]) continue;
                        ok = ok && me.wait(&m->p_full[x], t[x]++);
                        tc_fence_after();
                        if (ok) pv(x, x, i);
                        if (ok && i + 1 < steps[x]) {
                            if (!have) full(i + 1, 0);
                            have = true;
                            if (ok) qk(x, x, i + 1);
                        }
                    }
                    if (!ok) break;
                    free_stages(i, 1);
                    if (i + 1 < most) free_stages(i + 1, 0);
                    if (i + 2 == most) free_q();
                }
            } else {
                if (ok) qk(0, t[0] & 1, 0);
                free_stages(0, 0);
                if (most == 1) free_q();
                for (int i = 0; i < most && ok; ++i) {
                    const uint32_t u = t[0]++;
                    if (i + 1 < most) {
                        full(i + 1, 0);
                        if (ok) qk(0, (u + 1) & 1, i + 1);
                        free_stages(i + 1, 0);
                        if (i + 2 == most) free_q();
                    }
                    values(i);
                    ok = ok && me.wait(&m->p_full[u & 1], u >> 1);
                    tc_fence_after();
                    if (ok) pv(0, u & 1, i);
                    free_stages(i, 1);
                }
            }
            n += 2 * most * S::kParts;
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
    }
    if (me.lane == 0) {                                    // MMAs in flight end before TMEM is given back
        mma_commit(&m->drain);
        mbar_wait(&m->drain, 0);
    }
}

// Lays out the CTA's items, `per` tokens each, 32 requests at a time, one a lane: `rows(r, qs,
// qn)` gives a request's first row and tokens, `keys(r, it)` sets an item's keys.  The items of
// a request come longest first, and go there and back over the CTAs.
template <class Rows, class Keys>
__device__ __forceinline__ void lay_out_items(const Role& me, int batch, int kv_heads, int per, Rows rows, Keys keys) {
    Pipe* m = me.m;
    int c0 = -32;
    int64_t base = 0, all = 0;                             // items before the 32 requests, and theirs
    int64_t upto = 0;                                      // and of those up to the lane's
    int qs = 0, qn = 0, blocks = 0;
    for (int k = 0;; ++k) {
        const int64_t i = (int64_t)k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        while (i >= base + all && c0 + 32 < batch) {
            base += all;
            c0 += 32;
            qs = qn = 0;
            if (c0 + me.lane < batch) rows(c0 + me.lane, qs, qn);
            blocks = (qn + per - 1) / per;
            upto = (int64_t)blocks * kv_heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (me.lane >= o) upto += y;
            }
            all = __shfl_sync(0xffffffffu, upto, 31);
        }
        Item it = {};
        it.n = -1;
        const uint32_t past = __ballot_sync(0xffffffffu, i < base + upto);
        if (past) {
            const int at = __ffs(past) - 1;
            const int b = __shfl_sync(0xffffffffu, blocks, at);
            const int64_t j = i - base - __shfl_sync(0xffffffffu, upto - (int64_t)blocks * kv_heads, at);
            it.q_row = __shfl_sync(0xffffffffu, qs, at);
            it.n = __shfl_sync(0xffffffffu, qn, at);
            it.tok0 = (b - 1 - (int)(j / kv_heads)) * per;
            it.h = (int)(j % kv_heads);
            keys(c0 + at, it);
        }
        if (k >= kItems && !me.wait_all(&m->item_empty[k % kItems], k / kItems - 1)) break;
        if (me.lane < kMasked * 4) m->odd[k % kItems][me.lane >> 2][me.lane & 3] = 0;
        __syncwarp();
        if (me.lane == 0) {
            m->item[k % kItems] = it;
            m->any_odd[k % kItems] = 0;
            mbar_arrive(&m->item_full[k % kItems]);
        }
        if (it.n < 0) break;
    }
}

}  // namespace gtc
}  // namespace dsa
