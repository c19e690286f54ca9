// New tokens of grouped heads enter the KV8 cache: rotation by position, one scale
// for each block of 16 tokens and head, E4M3 codes; queries are rotated beside them.
//
//   (a, b) -> (a cos - b sin, a sin + b cos), angle p f_i, for the pairs of dims
//   e_new  = max(e of what the block already holds, smallest e: amax <= 448 2^e)
//   code   = E4M3(x 2^-e_new)
//
// Work split: a block of tokens and a head are one warp's: 16 x dim values fit its
// registers, the largest comes by shuffles, and no warp waits for another.  The
// warps of a thread block share the cosines and sines of the block's positions.
// A thread takes 16 dims of a token at a time, both dims of each pair among them, so
// queries and keys may be rotated in place.  Values lie with a block's 16 tokens side
// by side in the cache; a warp turns them over in shared memory and writes (or, where
// the block is not all new, reads, mends and writes) them as whole 16-byte pieces.
//
// What bounds it: 7 x 1024 tokens of 64 + 8 + 8 heads take 62 us, 4.5 TB/s, 67 % of a copy's
// rate: two thread blocks an SM, each loading, then computing, then storing, with the load and
// store pipe's wavefronts at 68 % of their peak (at 128 dims 60 bytes a thread spill at the 128
// registers that two blocks leave).  One token takes 5.0 us on the GPU, 128 of as many requests
// 6.2: a chain of loads (length, page, scale, codes).
//
// An angle is a whole number: f_i / 2 pi as a 64-bit fraction of a turn, times the
// position, modulo 2^64.  The fraction is formed from 106 bits of f_i / 2 pi, so that it
// is right to 2^-63 of a turn for any f_i up to 2^32, and the angle to 2^-32 at any
// position (an fp64 quotient's 53 bits would leave 2^-25 at position 2^31, 2^-15 with
// f_i = 1000).  It takes four integer products where fp64 would take twice as long
// (two fp64 operations a cycle and SM).
#include <algorithm>
#include <cmath>

#include "kv8.cuh"

namespace dsa {

int device_sm_count();

namespace kv8 {

// Heads of 256 dims take twice the registers and shared memory of a warp.
template <int D> constexpr int kThreads = D == 256 ? 128 : 256;
constexpr int kMaxPairs = 128;

struct Turns {
    uint64_t f[kMaxPairs];      // f_i / 2 pi in units of 2^-64 turns
};

// 1 / 2 pi as a sum of two fp64 numbers.
constexpr double kTurnHi = 0x1.45f306dc9c883p-3, kTurnLo = -0x1.6b01ec5417056p-57;

// A number of turns, less its whole ones, in units of 2^-64.
__host__ __device__ inline uint64_t turn_fraction(double x) {
    const double rest = x - rint(x);                        // exact, in [-1/2, 1/2]
    return rest == 0.5 ? 1ull << 63 : (uint64_t)(int64_t)rint(rest * 18446744073709551616.0);
}
__host__ __device__ inline uint64_t turn_fraction(double hi, double lo) { return turn_fraction(hi) + turn_fraction(lo); }

// x y, x and y sums of two fp64 numbers, to 2^-103 of itself.
struct Two { double hi, lo; };
inline Two times(Two x, Two y) {
    const double p = x.hi * y.hi, e = std::fma(x.hi, y.hi, -p) + std::fma(x.hi, y.lo, x.lo * y.hi);
    const double hi = p + e;
    return {hi, e - (hi - p)};
}
// f_i = base^(-2i / dims) = q^i with q^(dims / 2) = 1 / base: q is fp64's power and one step of
// Newton's method, q + q (1 - base q^n) / n, whose error is the square of fp64's.
inline void turns_of_base(double base, int dims, uint64_t* f) {
    const int n = dims / 2;
    const double q0 = std::pow(base, -1.0 / n);
    Two power = {base, 0.0};
    for (int i = 0; i < n; ++i) power = times(power, Two{q0, 0.0});
    const double step = q0 * ((1.0 - power.hi) - power.lo) / n;
    const Two q = {q0 + step, step - ((q0 + step) - q0)};
    Two x = {kTurnHi, kTurnLo};
    for (int i = 0; i < n; ++i, x = times(x, q)) f[i] = turn_fraction(x.hi, x.lo);
}

struct AppendArgs {
    const uint16_t *k, *v, *q;
    int64_t k_tok, k_head, v_tok, v_head, q_tok, q_head;   // strides in elements
    BatchDev b;
    int heads, kv_heads;
    int rope, halves;
    const float* inv_freq;
    uint8_t* cache;
    uint16_t *q_out, *k_out;
    int32_t* st;
    int rows_per;               // batch rows of a thread block: it takes the blocks that begin among them
    Turns turns;
};

// 16 dims of a token: two runs of 8.  The pairs of the rotation lie within them.
template <int D>
__device__ __forceinline__ void item_dims(int item, int rope, int halves, int& o1, int& o2) {
    const bool split = halves && item * 16 < rope;
    o1 = split ? item * 8 : item * 16;
    o2 = split ? rope / 2 + item * 8 : item * 16 + 8;
}

__device__ __forceinline__ void unpack8(uint4 w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float2 c) {
    const float a0 = a, b0 = b;
    a = a0 * c.x - b0 * c.y;
    b = a0 * c.y + b0 * c.x;
}
// Rotates item `item` of a token; cs: the token's cosines and sines.
__device__ __forceinline__ void rotate(float (&x)[16], int item, int rope, int halves, const float2* cs) {
    if (item * 16 >= rope) return;
    cs += item * 8;
    if (halves) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[i], x[8 + i], cs[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], cs[i]);
    }
}

// The exponent of a block whose largest value is amax: smallest e with amax <= 448 2^e.
__device__ __forceinline__ int exponent_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);       // 448 = 1.75 * 2^8
    return max(-kMaxExp, min(kMaxExp, e));
}

// Four codes of values scaled by 2^down.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float down) {
    const float2 a = e4m3x2_to_f32x2((uint16_t)codes), b = e4m3x2_to_f32x2((uint16_t)(codes >> 16));
    return f32x2_to_e4m3x2(a.x * down, a.y * down) | (uint32_t)f32x2_to_e4m3x2(b.x * down, b.y * down) << 16;
}
__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
    uint2 r;
    r.x = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv) | (uint32_t)f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16;
    r.y = f32x2_to_e4m3x2(x[4] * inv, x[5] * inv) | (uint32_t)f32x2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16;
    return r;
}

// Place of the 16 bytes of dim d in the warp's turned-over block: neighbouring items'
// dims (16 apart) fall into different banks.
__device__ __forceinline__ int turned(int d) { return ((d & ~7) | ((d ^ (d >> 4)) & 7)) * 16; }

// One warp: keys (V = false) or values of one block and head.  row0: batch row of the
// block's first new token, at place `held` of the block; n new tokens.  head: the page's
// part of this head, NULL when there is no page.
template <int D, bool V>
__device__ __forceinline__ void append_block(const AppendArgs& a, int h, int64_t row0, int held, int n, int at, uint8_t* head,
                                             const float2* cs, uint8_t* tile, int lane) {
    constexpr int kItems = D / 16;                          // of a token
    constexpr int kPer = kBlock * kItems / 32;              // of a lane
    constexpr float kBig = 448.0f * 16777216.0f;     // 448 * 2^24
    const uint16_t* src = (V ? a.v + h * a.v_head : a.k + h * a.k_head) + row0 * (V ? a.v_tok : a.k_tok);
    const int64_t tok = V ? a.v_tok : a.k_tok;
    float x[kPer][16];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int t = (lane + 32 * j) / kItems, item = (lane + 32 * j) % kItems;
        int o1, o2;
        item_dims<D>(item, V ? 0 : a.rope, a.halves, o1, o2);
        uint4 w1 = make_uint4(0, 0, 0, 0), w2 = w1;
        if (t < n) {
            w1 = *reinterpret_cast<const uint4*>(src + t * tok + o1);
            w2 = *reinterpret_cast<const uint4*>(src + t * tok + o2);
        }
        unpack8(w1, x[j]);
        unpack8(w2, x[j] + 8);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int t = (lane + 32 * j) / kItems, item = (lane + 32 * j) % kItems;
        if (!V && t < n) {
            rotate(x[j], item, a.rope, a.halves, cs + t * (a.rope / 2));
            if (a.k_out) {
                int o1, o2;
                item_dims<D>(item, a.rope, a.halves, o1, o2);
                uint16_t* out = a.k_out + ((row0 + t) * a.kv_heads + h) * D;
                *reinterpret_cast<uint4*>(out + o1) = pack8(x[j]);
                *reinterpret_cast<uint4*>(out + o2) = pack8(x[j] + 8);
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float m = fabsf(x[j][i]);
            if (m <= kBig) amax = fmaxf(amax, m);
            else x[j][i] = __int_as_float(0x7fc00000);
        }
    }
    if (!head) return;
    amax = warp_max(amax);
    float* scale = reinterpret_cast<float*>(head + scale_at(D)) + (V ? kBlocks : 0) + at;
    int e = exponent_for(amax);
    float down = 1.f;
    if (held) {
        const int was = scale_exponent(*scale);
        e = max(e, was);
        down = pow2(was - e);
    }
    const float inv = pow2(-e);
    __syncwarp();                                           // every lane has read the scale
    if (lane == 0) *scale = pow2(e);
    if (!V) {
        uint8_t* rows = head + at * kBlock * D;
        if (down != 1.f)
            for (int i = lane; i < held * (D / 16); i += 32) {
                uint4* p = reinterpret_cast<uint4*>(rows) + i;
                uint4 w = *p;
                w.x = rescale4(w.x, down), w.y = rescale4(w.y, down), w.z = rescale4(w.z, down), w.w = rescale4(w.w, down);
                *p = w;
            }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int t = (lane + 32 * j) / kItems, item = (lane + 32 * j) % kItems;
            int o1, o2;
            item_dims<D>(item, a.rope, a.halves, o1, o2);
            if (t < n) {
                *reinterpret_cast<uint2*>(rows + (held + t) * D + o1) = codes8(x[j], inv);
                *reinterpret_cast<uint2*>(rows + (held + t) * D + o2) = codes8(x[j] + 8, inv);
            }
        }
    } else {
        uint4* piece = reinterpret_cast<uint4*>(head + v_at(D) + at * kBlock * D);     // a dim's 16 tokens
        if (n < kBlock) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int d = lane + 32 * i;
                uint4 w = piece[d];
                if (down != 1.f) {
                    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int k = min(4, max(0, held - 4 * c));                   // bytes of earlier tokens
                        const uint32_t m = k == 4 ? 0xffffffffu : (1u << (8 * k)) - 1;
                        u[c] = (rescale4(u[c], down) & m) | (u[c] & ~m);
                    }
                }
                *reinterpret_cast<uint4*>(tile + turned(d)) = w;
            }
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int t = (lane + 32 * j) / kItems, item = (lane + 32 * j) % kItems;
            if (t < n) {
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const uint16_t two = f32x2_to_e4m3x2(x[j][i] * inv, x[j][i + 1] * inv);
                    tile[turned(item * 16 + i) + held + t] = (uint8_t)two;
                    tile[turned(item * 16 + i + 1) + held + t] = (uint8_t)(two >> 8);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < D / 32; ++i) piece[lane + 32 * i] = *reinterpret_cast<const uint4*>(tile + turned(lane + 32 * i));
        __syncwarp();
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads<D>, 2)
append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kThreads = kv8::kThreads<D>, kWarps = kThreads / 32;
    __shared__ alignas(16) uint8_t tiles[kWarps][kBlock * D];
    __shared__ float2 cs[kBlock * kMaxPairs];
    __shared__ uint64_t turn[kMaxPairs];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pairs = a.rope / 2;
    pdl_wait();
    pdl_trigger();
    const BatchDev& b = a.b;
    const int64_t rows = min((int64_t)b.q_start[b.batch], b.total_q);
    const int64_t begin = (int64_t)blockIdx.x * a.rows_per, end = min(begin + a.rows_per, rows);
    if (begin >= end) return;
    for (int i = tid; i < pairs; i += kThreads) {
        uint64_t f = a.turns.f[i];
        if (a.inv_freq) {
            const double x = a.inv_freq[i], hi = x * kTurnHi;
            f = turn_fraction(hi, fma(x, kTurnLo, fma(x, kTurnHi, -hi)));
        }
        turn[i] = f;
    }
    int r = row_request(b.q_start, b.batch, begin);
    for (int64_t row = begin; row < end;) {
        while (row >= b.q_start[r + 1]) ++r;               // row < q_start[B]
        const int64_t first = b.q_start[r], len = b.seq_len[r];
        const int64_t p = len - (b.q_start[r + 1] - row);
        const int held = (int)(((p % kBlock) + kBlock) % kBlock);
        if (row > first && held != 0) {                    // inside a block that begins before: on to the next
            row = min(row + kBlock - held, (int64_t)b.q_start[r + 1]);
            continue;
        }
        const int n = (int)min((int64_t)(kBlock - held), min((int64_t)b.q_start[r + 1], rows) - row);
        __syncthreads();                                   // turn is complete; the last block's cosines have been read
        for (int i = tid; i < n * pairs; i += kThreads) {
            const uint64_t angle = turn[i % pairs] * (uint64_t)(p + i / pairs);
            // The nearest quarter of a turn is taken off in whole numbers: what is left, at most a
            // quarter of half a turn, keeps 2^-27 of one as fp32, where the whole angle would keep 2^-25.
            const uint32_t quarter = (uint32_t)((angle + (1ull << 61)) >> 62);
            const int32_t rest = (int32_t)((int64_t)(angle - ((uint64_t)quarter << 62)) >> 30);
            float s, c;
            sincospif((float)rest * 1.1641532182693481e-10f, &s, &c);          // 2^-33
            const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;       // cos(a + 90) = -sin a, sin(a + 90) = cos a
            cs[i] = make_float2(quarter + 1 & 2 ? -x : x, quarter & 2 ? -y : y);
        }
        __syncthreads();
        uint8_t* page = nullptr;
        if (p < 0 || p / kPage >= b.max_pages) {
            if (tid == 0 && blockIdx.y == 0) record_error(a.st, DSA_DEVERR_INDEX_RANGE, p);
        } else {
            const int64_t id = b.page_table[(int64_t)r * b.max_pages + p / kPage];
            if (id < 0 || id >= b.num_pages) {
                if (tid == 0 && blockIdx.y == 0) record_error(a.st, DSA_DEVERR_PAGE_RANGE, id);
            } else {
                page = a.cache + id * a.kv_heads * head_bytes(D);
            }
        }
        const int at = (int)(p >= 0 ? p % kPage / kBlock : 0);
        const int step = gridDim.y * kWarps, me = blockIdx.y * kWarps + warp;
        for (int job = me; job < 2 * a.kv_heads; job += step) {
            const int h = job >> 1;
            uint8_t* head = page ? page + h * head_bytes(D) : nullptr;
            if (job & 1) append_block<D, true>(a, h, row, held, n, at, head, cs, tiles[warp], lane);
            else append_block<D, false>(a, h, row, held, n, at, head, cs, tiles[warp], lane);
        }
        if (a.q) {
            // queries: a thread takes 16 dims of a head, of four tokens at a time
            constexpr int kItems = D / 16;
            for (int i = blockIdx.y * kThreads + tid; i < a.heads * kItems; i += gridDim.y * kThreads) {
                const int item = i % kItems, h = i / kItems;
                int o1, o2;
                item_dims<D>(item, a.rope, a.halves, o1, o2);
                const uint16_t* src = a.q + row * a.q_tok + h * a.q_head;
                uint16_t* out = a.q_out + (row * a.heads + h) * D;
                for (int t0 = 0; t0 < n; t0 += 4) {
                    uint4 w[4][2];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        if (t0 + t < n) {
                            w[t][0] = *reinterpret_cast<const uint4*>(src + (t0 + t) * a.q_tok + o1);
                            w[t][1] = *reinterpret_cast<const uint4*>(src + (t0 + t) * a.q_tok + o2);
                        }
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        if (t0 + t < n) {
                            float x[16];
                            unpack8(w[t][0], x);
                            unpack8(w[t][1], x + 8);
                            rotate(x, item, a.rope, a.halves, cs + (t0 + t) * pairs);
                            *reinterpret_cast<uint4*>(out + (int64_t)(t0 + t) * a.heads * D + o1) = pack8(x);
                            *reinterpret_cast<uint4*>(out + (int64_t)(t0 + t) * a.heads * D + o2) = pack8(x + 8);
                        }
                }
            }
        }
        row += n;
    }
}

}  // namespace kv8
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_kv8_append(const dsa_heads* k, const dsa_heads* v, const dsa_heads* q, const dsa_batch* b,
                                     int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t rope_dims,
                                     int32_t rope_style, float rope_base, const float* inv_freq, uint8_t* cache,
                                     void* q_out, void* k_out, int32_t* dev_status, void* stream) {
    dsa_status vs = validate_batch(b);
    if (vs != DSA_OK) return vs;
    vs = kv8::check_shape(heads, kv_heads, head_dim);
    if (vs != DSA_OK) return vs;
    if (rope_style != DSA_ROPE_INTERLEAVED && rope_style != DSA_ROPE_HALVES) return DSA_ERR_INVALID_ARGUMENT;
    if (rope_dims < 0 || rope_dims > head_dim || !(rope_base > 0.f) || std::isinf(rope_base)) return DSA_ERR_INVALID_ARGUMENT;
    if (rope_dims % 16 != 0) return DSA_ERR_UNSUPPORTED;
    if (b->total_q == 0) return DSA_OK;
    if (!k || !v || !cache || !q != !q_out) return DSA_ERR_INVALID_ARGUMENT;
    for (const dsa_heads* h : {k, v, q})
        if (h && (vs = kv8::check_heads(h)) != DSA_OK) return vs;
    if (!aligned16(cache) || !aligned16(q_out) || !aligned16(k_out)) return DSA_ERR_ALIGNMENT;

    kv8::AppendArgs a = {};
    a.k = static_cast<const uint16_t*>(k->data);
    a.v = static_cast<const uint16_t*>(v->data);
    a.k_tok = k->token_stride, a.k_head = k->head_stride;
    a.v_tok = v->token_stride, a.v_head = v->head_stride;
    if (q) {
        a.q = static_cast<const uint16_t*>(q->data);
        a.q_tok = q->token_stride, a.q_head = q->head_stride;
    }
    a.b = to_dev(b);
    a.heads = heads, a.kv_heads = kv_heads;
    a.rope = rope_dims, a.halves = rope_style == DSA_ROPE_HALVES;
    a.inv_freq = inv_freq;
    a.cache = cache;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.k_out = static_cast<uint16_t*>(k_out);
    a.st = dev_status;
    if (!inv_freq) {
        // the last rotation's frequencies, by host thread: forming them takes longer than the rest of the call
        static thread_local struct { int32_t dims = -1; float base = 0.f; kv8::Turns turns; } last;
        if (last.dims != rope_dims || last.base != rope_base) {
            kv8::turns_of_base(rope_base, rope_dims, last.turns.f);
            last.dims = rope_dims, last.base = rope_base;
        }
        a.turns = last.turns;
    }
    // A thread block for each row where rows are few, so that a decode batch spreads over the
    // SMs (one that does not begin a block of tokens ends at once), for 16 rows where they are
    // many; several share a block of tokens' heads, eight to an SM where there are heads enough.
    a.rows_per = b->total_q <= 2048 ? 1 : kv8::kBlock;
    const int64_t groups = (b->total_q + a.rows_per - 1) / a.rows_per;
    const int64_t blocks = std::min<int64_t>(groups, (b->total_q + kv8::kBlock - 1) / kv8::kBlock + b->batch);
    const int threads = head_dim == 256 ? kv8::kThreads<256> : kv8::kThreads<128>, warps = threads / 32;
    const int64_t jobs = std::max<int64_t>((2 * (int64_t)kv_heads + warps - 1) / warps, (int64_t)heads * head_dim / 16 / threads);
    const int64_t share = std::max<int64_t>(1, std::min<int64_t>(jobs, (8 * device_sm_count() + blocks - 1) / blocks));
    const dim3 grid((unsigned)groups, (unsigned)std::min<int64_t>(share, 65535));
    auto* kernel = head_dim == 64 ? kv8::append_kernel<64> : head_dim == 128 ? kv8::append_kernel<128> : kv8::append_kernel<256>;
    DSA_CHECK(launch_pdl(kernel, grid, dim3((unsigned)threads), 0, as_stream(stream), 1, a));
    return DSA_OK;
}
