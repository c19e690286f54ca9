// MLA over a whole context of the paged latent cache: a sliding window with the
// context's first tokens (sinks), and trees of drafted tokens.
//   S_hj = scale * <q_h, [c_j * s_j | r_j]>,  out_h = sum_j softmax_j(S_hj) c_j
// over the positions j that the query row sees, 64 heads of 576 dims.
#include "dsa_internal.cuh"
#include "indexer_common.cuh"

namespace dsa {

int device_sm_count();

namespace mld {

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
    int32_t* st;
};

// One row's visible positions: j < sink_end or first <= j < end, and new token
// u at position prefix + u when bit u of mask is set.  They lie in `tiles`
// pages: the first sink_pages, then those from first_page on.
struct Row {
    int32_t r;                  // request
    int32_t sink_end, first, end;
    int32_t prefix;
    uint64_t mask;
    int32_t sink_pages, first_page, tiles;
    __device__ __forceinline__ int page(int tile) const { return tile < sink_pages ? tile : first_page + tile - sink_pages; }
    __device__ __forceinline__ bool sees(int j) const {
        if (j < sink_end || (j >= first && j < end)) return true;
        const unsigned u = (unsigned)(j - prefix);
        return u < 64u && (mask >> u & 1u);
    }
};

// Row `row` of the batch.  A row that sees nothing keeps one (empty) tile, so
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
    w.tiles = 1;
    if (L <= 0 || w.prefix < 0) return w;
    if (v.tree) {
        const int known = min(qn, 64);
        w.mask = v.tree[row] & (known >= 64 ? ~0ull : (1ull << known) - 1);
        w.end = min(w.prefix, L);
        const int64_t last = w.mask ? (int64_t)w.prefix + 64 - __clzll((long long)w.mask) : w.end;
        if (last > L) w.mask = L > w.prefix ? w.mask & ((1ull << (L - w.prefix)) - 1) : 0;
        w.tiles = max(1, (int)((min(last, (int64_t)L) + kPage - 1) / kPage));
        return w;
    }
    const int end = (int)min((int64_t)w.prefix + (row - qs) + 1, (int64_t)L);
    w.end = end;
    w.first = max(0, w.prefix + (int)(row - qs) + 1 - v.window);
    w.sink_end = min(v.sinks, end);
    w.sink_pages = w.sink_end / kPage + (w.sink_end % kPage != 0);
    w.first_page = max(w.sink_pages, w.first / kPage);
    w.tiles = max(1, w.sink_pages + max(0, (end + kPage - 1) / kPage - w.first_page));
    return w;
}

// The plain kernel: one block per (row, 8 heads), a warp per head.  16 tokens at a
// time are dequantised into shared memory; each warp keeps its head's query and
// output in registers with a running maximum and sum.
constexpr int kThreads = 256;
constexpr int kTok = 16;

__global__ void __launch_bounds__(kThreads)
dense_mla_kernel(Args a) {
    __shared__ float k[kTok][576];
    __shared__ int seen[kTok];
    const int64_t row = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y * 8 + warp;
    const BatchDev& b = a.b;
    const Row w = row_view(b, a.view, row, blockIdx.y == 0 && threadIdx.x == 0 ? a.st : nullptr);
    if (w.tiles == 0) return;
    float q[18], o[16] = {}, m = -INFINITY, l = 0.f;
    for (int i = 0; i < 18; ++i) q[i] = bf16_bits_to_f32(a.q[(row * 64 + h) * 576 + lane + 32 * i]) * a.scale;
    for (int t = 0; t < w.tiles; ++t) {
        const int lp = w.page(t);
        const int64_t pg = lp < b.max_pages ? b.page_table[(int64_t)w.r * b.max_pages + lp] : -1;
        for (int base = 0; base < kPage; base += kTok) {
            __syncthreads();
            if (threadIdx.x < kTok) {
                const int j = lp * kPage + base + threadIdx.x;
                int s = w.sees(j) ? 1 : 0;
                if (s && (pg < 0 || pg >= b.num_pages)) {
                    if (blockIdx.y == 0) record_error(a.st, DSA_DEVERR_PAGE_RANGE, pg);
                    s = 0;
                }
                seen[threadIdx.x] = s;
            }
            __syncthreads();
            for (int e = threadIdx.x; e < kTok * 576; e += kThreads) {
                const int tk = e / 576, d = e % 576;
                float x = 0.f;
                if (seen[tk]) {
                    const uint8_t* rp = a.kv + pg * kKvPageBytes + (int64_t)(base + tk) * kKvTokenBytes;
                    if (d < 512) {
                        const float sc = reinterpret_cast<const float*>(rp + 512)[d >> 7];
                        x = e4m3x2_to_f32x2(rp[d]).x * sc;
                    } else {
                        x = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(rp + 528)[d - 512]);
                    }
                }
                k[tk][d] = x;
            }
            __syncthreads();
            for (int tk = 0; tk < kTok; ++tk) {
                if (!seen[tk]) continue;
                float s = 0.f;
                for (int i = 0; i < 18; ++i) s += q[i] * k[tk][lane + 32 * i];
                s = warp_sum(s);
                const float mn = fmaxf(m, s);
                const float al = expf(m - mn), p = expf(s - mn);
                l = l * al + p;
                for (int i = 0; i < 16; ++i) o[i] = o[i] * al + p * k[tk][lane + 32 * i];
                m = mn;
            }
        }
    }
    for (int i = 0; i < 16; ++i) {
        const float v = l > 0.f ? o[i] / l : 0.f;
        const int64_t at = (row * 64 + h) * 512 + lane + 32 * i;
        if (a.out_f32) static_cast<float*>(a.out)[at] = v;
        else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    }
    if (a.lse && lane == 0) a.lse[row * 64 + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

static size_t ws_bytes(int G) {
    const size_t n = (size_t)2 * G * 64 * (512 + 2) * 4 + (size_t)G * 16;
    return (n + 255) / 256 * 256;
}

static dsa_status launch(const void* q, const uint8_t* kv, const dsa_batch* b, View view, float softmax_scale, void* out,
                         int32_t out_dtype, float* lse, void* ws, size_t bytes, int32_t* st, void* stream) {
    if (out_dtype != DSA_DTYPE_BF16 && out_dtype != DSA_DTYPE_F32) return DSA_ERR_INVALID_ARGUMENT;
    if (!(softmax_scale > 0.f) || softmax_scale > 3.0e38f) return DSA_ERR_INVALID_ARGUMENT;
    if (b->num_pages * DSA_PAGE_TOKENS > 0x7fffffffLL) return DSA_ERR_UNSUPPORTED;        // int32 cache slots
    if (b->total_q == 0) return DSA_OK;
    if (!q || !kv || !out) return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(q) || !aligned16(kv) || !aligned16(out)) return DSA_ERR_ALIGNMENT;
    if (!ws) return DSA_ERR_INVALID_ARGUMENT;
    if (bytes < ws_bytes(device_sm_count())) return DSA_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(ws)) return DSA_ERR_ALIGNMENT;
    Args a = {};
    a.q = static_cast<const uint16_t*>(q);
    a.kv = kv;
    a.b = to_dev(b);
    a.view = view;
    a.scale = softmax_scale;
    a.out = out;
    a.out_f32 = out_dtype == DSA_DTYPE_F32;
    a.lse = lse;
    a.st = st;
    dense_mla_kernel<<<dim3((unsigned)b->total_q, 8), kThreads, 0, as_stream(stream)>>>(a);
    DSA_CHECK_LAUNCH();
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
