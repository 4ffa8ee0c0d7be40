// tcgen05 pieces that the paged cache's kernels share: e4m3 MMAs and the
// shared-memory layouts of their operands, and the row arithmetic of a sink.
#pragma once

#include <math.h>

#include <cuda_fp16.h>

#include "common.cuh"

namespace sattn {

constexpr uint32_t B_E5M2 = 1u << 10;  // in such a descriptor: B is e5m2
// kind::f8f6f4, e4m3 x e4m3 -> f32; a_mn, b_mn: A is stored with its M index, B with its
// N index contiguous.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N, uint32_t a_mn,
                                                          uint32_t b_mn) {
    return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Shared-memory descriptor of rows of W bytes (16, 32, 64, 128) under W-byte
// swizzle (16: none), in atoms of 8 rows that follow one another. Rows are the M or
// N index with K contiguous, or K with one such atom's M or N contiguous.
template <int W> __device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(W == 16 ? 8 : 1) << 16;  // unswizzled: 8-row groups of K 128 bytes apart
    d |= (uint64_t)(8 * W >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(W == 128 ? 2 : W == 64 ? 4 : W == 32 ? 6 : 0) << 61;
    return d;
}
// Byte offset of 16-byte unit u of row r in such a tile: the address bits from 4
// up are XORed with those from 7 up.
template <int W> __device__ __forceinline__ uint32_t sw_offset(uint32_t r, uint32_t u) {
    const uint32_t a = r * W + (u << 4);
    return W == 16 ? a : a ^ ((a >> 3) & (W - 16));
}
__device__ __forceinline__ float tmem_ld1(uint32_t a) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(a));
    tc_wait_ld();
    return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t a, float v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(a),
                 "r"(__float_as_uint(v))
                 : "memory");
    tc_wait_st();
}
constexpr int TIMED_OUT = 2;

// mbar_wait in as few instructions as it takes: it stands at dozens of places of
// kernels whose roles share the instruction cache, and code that does not fit
// there costs more than anything else in a short call. The limit is taken in 32 bits of
// nanoseconds (4 s at most).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const DevCtx &ctx,
                                         volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t limit = (uint32_t)min(ctx.wait_ns, (uint64_t)4000000000u);
    uint32_t t0, t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
#pragma unroll 1
    do {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    } while (t - t0 <= limit);
    *abort = TIMED_OUT;  // recorded at the kernel's end
    return false;
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile(
        "{\n\t.reg .b64 st;\n\t"
        "mbarrier.arrive.release.cta.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
        "r"(n)
        : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Two f16 to two e4m3 codes, nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t difference_f16x2(uint32_t a, uint32_t b) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&a),
                              *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&d);
}
// F (a - b) of two f16 pairs.
template <int F> __device__ __forceinline__ uint32_t times_difference(uint32_t a, uint32_t b) {
    const __half2 d = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&a),
                                      *reinterpret_cast<const __half2 *>(&b)),
                              __float2half2_rn((float)F));
    return *reinterpret_cast<const uint32_t *>(&d);
}
// Two f16 in [0, 2^15] as N e5m2 each, t[0] + t[1] / 8 + t[2] / 64 (+ t[3] / 512), in the upper
// bytes of t's halves. A term is the upper byte of what the ones before leave (times 8
// each time), which an f16 holds: four have 3 + 3 + 3 + 2 bits, all of them; for three the
// f16 are first rounded to 9 bits (to 2^-22 below 2^-14). A NaN is not kept.
template <int N> __device__ __forceinline__ void e5m2_terms(uint32_t x, uint32_t (&t)[N]) {
    static_assert(N == 3 || N == 4, "9 or 11 bits");
    if constexpr (N == 3) x = (x + 0x00020002u) & 0xfffcfffcu;
#pragma unroll
    for (int k = 0; k < N - 1; ++k) {
        t[k] = x & 0xff00ff00u;
        x = times_difference<8>(x, t[k]);
    }
    t[N - 1] = x;
}

// x = keep ? x : -inf. Volatile so that it stays behind the branch it is written in:
// the compiler otherwise turns a branch around many selections into selections that
// every tile pays for (3 ALU operations a score where whole tiles need none).
__device__ __forceinline__ void hide_unless(uint32_t &x, bool keep) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tselp.b32 %0, %0, 0xff800000, p;\n\t}"
        : "+r"(x)
        : "r"((uint32_t)keep));
}

// The null logit joins a row's denominator.
__device__ __forceinline__ void with_null_sink(float sink, float &lse2, float &inv) {
    const float top = fmaxf(lse2, sink);
    if (top == -INFINITY) return;
    const float all = top + __log2f(ex2(lse2 - top) + ex2(sink - top));
    inv *= ex2(lse2 - all);
    lse2 = lse2 != lse2 ? lse2 : all;
}

}  // namespace sattn
