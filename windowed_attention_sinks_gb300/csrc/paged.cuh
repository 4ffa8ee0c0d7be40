// Device helpers of the paged FP8 cache kernels: which sequence a token
// belongs to, whether that sequence is well formed, and the e4m3 coding.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>

#include "common.cuh"

namespace sattn {

// One sequence of a ragged batch: its new tokens are rows [t0, t0 + n) of the
// packed arrays and the last n of the `len` positions its pages hold.
struct PagedSeq {
    int t0, n, len;
};

// The largest b in [0, B) with start(b) <= x, for a non-decreasing start with
// start(0) <= x; called by a whole warp. Each round loads 32 pivots at once, so
// a batch of 1024 takes two dependent loads where a bisection takes ten.
template <typename F> __device__ __forceinline__ int warp_find(int B, long long x, F start) {
    const int lane = threadIdx.x & 31;
    int lo = 0, count = B;  // the answer lies in [lo, lo + count)
    while (count > 1) {
        const int step = (count + 31) >> 5;
        const int at = lo + lane * step;
        const bool le = lane == 0 || (lane * step < count && start(at) <= x);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));
        count = min(step, count - last * step);
        lo += last * step;
    }
    return lo;
}

// Loads sequence b and checks it against the packed arrays: cu_seqlens starts at
// 0 and never falls, its rows lie in [0, T), its positions fit the page table.
__device__ __forceinline__ bool load_seq(const int32_t *cu, const int32_t *kv_lens, int b, int T,
                                         long long capacity, PagedSeq &s) {
    s.t0 = __ldg(cu + b);
    const int t1 = __ldg(cu + b + 1);
    s.len = __ldg(kv_lens + b);
    s.n = t1 - s.t0;
    return __ldg(cu) == 0 && s.t0 >= 0 && t1 >= s.t0 && t1 <= T && s.len >= 0 && s.len <= capacity;
}

// Two values to two e4m3 codes (the first in the low byte), nearest even,
// saturating at +-448, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | e4m3x2(c, d) << 16;
}
// Two codes to their values, exactly (f16 holds every e4m3 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
    const uint32_t h = e4m3x2_to_f16x2(codes);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The least power of two s >= 2^-64 with amax <= 448 s: 448 = 1.75 x 2^8, so the
// exponent of amax less 8, one more where its mantissa is above 1.75. An
// infinite amax counts as the largest finite one.
constexpr float LEAST_SCALE = 5.421010862427522e-20f;  // 2^-64
__device__ __forceinline__ float pow2_scale(float amax) {
    const uint32_t b = min(__float_as_uint(amax), 0x7f7fffffu);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < 63 ? LEAST_SCALE : __uint_as_float((uint32_t)e << 23);
}

// A sink in log2 units. The largest finite values stay finite (the factor would
// take them to infinity): key 0 alone has weight 1 whatever its bias.
__device__ __forceinline__ float sink_log2(float s) {
    return isinf(s) ? s : fminf(fmaxf(s * 1.4426950408889634f, -3e38f), 3e38f);
}

}  // namespace sattn
