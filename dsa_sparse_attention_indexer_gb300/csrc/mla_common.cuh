// Device helpers shared by the MLA kernels: bounded waits, conversions of latent
// rows and queries to fp16, and a transposing warp reduction.
#pragma once
#include "dsa_internal.cuh"
#include "sm100.cuh"

namespace dsa {
namespace mlc {

using namespace sm100;

// Named barriers of a role's threads; bar_any also reduces a predicate.
template <int BAR, int NT>
__device__ __forceinline__ void bar_sync() {
    asm volatile("bar.sync %0, %1;" ::"n"(BAR), "n"(NT) : "memory");
}
template <int BAR, int NT>
__device__ __forceinline__ bool bar_any(bool pred) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n"
                 " selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(r) : "r"((uint32_t)pred), "n"(BAR), "n"(NT) : "memory");
    return r != 0;
}

// mbarrier wait that also gives up when another role has set the abort flag.
__device__ __forceinline__ bool wait_ab(uint64_t* bar, uint32_t parity, const volatile int32_t* abort_flag,
                                        uint64_t limit_ns = 2000000000ull) {
    if (mbar_try_wait(bar, parity)) return true;
    if (limit_ns == 0) return false;                       // no waiting at all
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
        if ((it & 63u) == 0u && (*abort_flag || globaltimer_ns() - t0 > limit_ns)) return false;
    }
}

// 16-byte read-only load that stays where it is written (a prefetch a tile
// ahead must not be sunk to its first use).
__device__ __forceinline__ uint4 ldg_pinned(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// 16 (4) bytes from global to shared memory without a register; the thread that
// issued them sees them after cp_async_wait_all.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 2^x by the hardware approximation (subnormal results flush to 0): its error
// is far below the fp16 rounding that P gets next.
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (a + b) * s for two values in two instructions.
__device__ __forceinline__ float2 add_scale2(float2 a, float2 b, float2 s) {
    float2 r;
    asm("{\n .reg .b64 a, b, s;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 s, {%6, %7};\n"
        " add.rn.f32x2 a, a, b;\n mul.rn.f32x2 a, a, s;\n mov.b64 {%0, %1}, a;\n}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(s.x), "f"(s.y));
    return r;
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t e4m3x2_scaled_h2(uint32_t two, __half2 sc2) {
    __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);   // exact
    const __half2 p = __hmul2(*reinterpret_cast<__half2*>(&h), sc2);                     // * 2^e: exact
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t bf16x2_to_h2(uint32_t w) {
    return pack_h2(bf16_bits_to_f32(w & 0xffffu), bf16_bits_to_f32(w >> 16));
}
// Two bf16 key RoPE values -> two fp16.  A magnitude of 2^16 or more (inf and
// NaN included) does not fit fp16: it is clamped to +-65280 (the largest bf16
// below fp16's maximum), so the scores stay finite, and bad is set.  Every
// other bf16 value converts exactly, except those below 2^-17, whose error
// (under 2^-25 absolute) is far below the attention tolerance.
__device__ __forceinline__ uint32_t rope_bf16x2_to_h2(uint32_t w, uint32_t& bad) {
    const uint32_t over = __vcmpgeu2(w & 0x7fff7fffu, 0x47804780u);   // per half: |x| >= 2^16
    bad |= over;
    return bf16x2_to_h2((w & ~over) | (over & ((w & 0x80008000u) | 0x477f477fu)));
}
// The same with cvt's saturation to the largest finite fp16 (a caller that checks
// the magnitudes itself).
__device__ __forceinline__ uint32_t bf16x2_to_h2_sat(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(__uint_as_float(w & 0xffff0000u)), "f"(__uint_as_float(w << 16)));
    return h;
}
template <int OFF = 0>
__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0 + %5], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d), "n"(OFF) : "memory");
}
// Four E4M3 codes times a power of two (as two equal fp16), exact: (lo, hi) pairs of fp16.
__device__ __forceinline__ void e4m3x4_scaled_h2(uint32_t four, uint32_t sc2, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n .reg .b32 x, y;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 x, a;\n cvt.rn.f16x2.e4m3x2 y, b;\n"
        " mul.rn.f16x2 %0, x, %3;\n mul.rn.f16x2 %1, y, %3;\n}"
        : "=r"(lo), "=r"(hi) : "r"(four), "r"(sc2));
}
// A query pair multiplied by the row's power of two `sc` (exact in fp32) ->
// two fp16.  After that scaling no |value| reaches 2^15, so nothing
// overflows; values more than 2^39 below the row's largest are rounded to
// fp16's subnormal grid (absolute error under 2^-25 after the scaling).
__device__ __forceinline__ uint32_t bf16x2_scaled_to_h2(uint32_t w, float sc) {
    return pack_h2(bf16_bits_to_f32(w & 0xffffu) * sc, bf16_bits_to_f32(w >> 16) * sc);
}

// Reduce 32 values across the 32 lanes of a warp: afterwards lane l holds the
// result for index l in v[0] (31 shuffles instead of 160).
template <bool kMax>
__device__ __forceinline__ void xreduce32(float (&v)[32], int lane) {
#pragma unroll
    for (int s = 16, n = 16; s >= 1; s >>= 1, n >>= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n];
            const float keep = up ? v[i + n] : v[i];
            const float recv = __shfl_xor_sync(0xffffffffu, send, s);
            v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
        }
    }
}

// Reduce 16 values across the 32 lanes of a warp: afterwards lanes l and l + 16
// hold the result for index l in v[0].
template <bool kMax>
__device__ __forceinline__ void xreduce16(float (&v)[16], int lane) {
#pragma unroll
    for (int s = 8, n = 8; s >= 1; s >>= 1, n >>= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n];
            const float keep = up ? v[i + n] : v[i];
            const float recv = __shfl_xor_sync(0xffffffffu, send, s);
            v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
        }
    }
    const float recv = __shfl_xor_sync(0xffffffffu, v[0], 16);
    v[0] = kMax ? fmaxf(v[0], recv) : v[0] + recv;
}

}  // namespace mlc
}  // namespace dsa
