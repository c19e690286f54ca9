// The KV8 cache: grouped heads' keys and values in E4M3, one power-of-two scale
// for each block of 16 tokens and head (layout in dsa.h).
#pragma once
#include "dsa_internal.cuh"
#include "indexer_common.cuh"
#include "mla_common.cuh"

namespace dsa {
namespace kv8 {

constexpr int kBlock = DSA_KV8_BLOCK;
constexpr int kBlocks = kPage / kBlock;                    // of a page
constexpr int kMaxExp = DSA_KV8_MAX_EXP;

// Bytes of one head in a page, and where its parts begin.
__host__ __device__ constexpr int64_t head_bytes(int dim) { return 2 * kPage * dim + 32; }
__host__ __device__ constexpr int v_at(int dim) { return kPage * dim; }
__host__ __device__ constexpr int scale_at(int dim) { return 2 * kPage * dim; }

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // e in [-126, 127]
// 2^-d for a whole d in [-126, 126].
__device__ __forceinline__ float minus_pow2(float d) { return __int_as_float(__float_as_int(8388608.0f + 127.0f - d) << 23); }
// The exponent of a stored scale.  Whatever the word holds, it is one of the cache's.
__device__ __forceinline__ int scale_exponent(float s) {
    return max(-kMaxExp, min(kMaxExp, (int)((__float_as_uint(s) >> 23) & 0xffu) - 127));
}

// Four codes -> their values as fp16, exactly.
__device__ __forceinline__ void e4m3x4_h2(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}" : "=r"(lo), "=r"(hi) : "r"(four));
}

// The power of two by which a row of q becomes fp16: it puts its largest |q| (`top`, bf16 bits of a finite
// number) in [2^14, 2^15), or a number below 2^-112 as near to that as 2^126 takes it.
__device__ __forceinline__ int q_exponent(uint32_t top) { return top ? min(126, 14 - ((int)(top >> 7) - 127)) : 0; }
// Log2 units of a score of such a row, neither 0 nor infinite, as scores of -inf and differences of 0 are
// multiplied by them.  A score without its units is below 2^56, so with 2^-102 or less it is nothing beside 1;
// two of them differ by 2^-57 or not at all, so with 2^100 or more a row's best has all of the weight.
// `most`: what the caller's products allow.
__device__ __forceinline__ float q_units(float scale, int e, float most) { return fminf(fmaxf(scale * pow2(-e), 0x1p-102f), most); }

// A wait of these kernels' pipelines: within the limit, and not beyond another role's
// timeout.  A limit of 0 takes what has happened already, and is not suspended for it.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const volatile int32_t* abort_flag, uint64_t limit_ns) {
    return limit_ns == 0 ? sm100::mbar_test_wait(bar, parity) : mlc::wait_ab(bar, parity, abort_flag, limit_ns);
}

// The largest softmax scale of the attention calls: log2(e) times it is finite.
constexpr float kMostScale = 2.0e38f;

// Checks that the calls on grouped heads share.
inline dsa_status check_shape(int32_t heads, int32_t kv_heads, int32_t dim) {
    if (heads < 1 || kv_heads < 1) return DSA_ERR_INVALID_ARGUMENT;
    if (dim != 64 && dim != 128 && dim != 256) return DSA_ERR_UNSUPPORTED;
    if (heads % kv_heads != 0 || heads / kv_heads > 128 || heads > 65535) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}
inline dsa_status check_heads(const dsa_heads* h) {
    if (!h->data || h->token_stride < 0 || h->head_stride < 0) return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(h->data) || h->token_stride % 8 != 0 || h->head_stride % 8 != 0) return DSA_ERR_ALIGNMENT;
    return DSA_OK;
}

}  // namespace kv8
}  // namespace dsa
