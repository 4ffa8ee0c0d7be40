// Attention over a paged e4m3 cache, one warp per query row (token, head).
//
// Serves fp32 queries. Each lane holds d/32 neighbouring columns of the query and of the
// accumulator; the row walks its visible positions lo .. hi with an online
// softmax in the log2 domain. A key's logit is <q, codes> * k_scale * scale, a
// value counts codes * v_scale, in terms of the power of two of the largest v_scale so
// far (exact), so that sums of values near fp32's largest do not overflow.
//
// Bound by the one-key-at-a-time chain (table entry, scale, codes, a reduction over the
// warp, an exponential) rather than by memory, and each head of a KV group reads the
// codes again: it is the exact fp32 form, the bf16 kernels are the fast ones. 32 requests
// of 301 .. 8192 positions, 32 heads on 8, d = 128: 9.7 ms against their 54 us.
#include <math.h>

#include "internal.h"
#include "paged.cuh"

namespace sattn {
namespace {

constexpr int kWarps = 4;

template <int E> __device__ __forceinline__ void load_codes(const uint8_t *p, float (&v)[E]) {
    uint32_t w;
    if (E == 4) w = __ldg(reinterpret_cast<const uint32_t *>(p));
    else w = __ldg(reinterpret_cast<const uint16_t *>(p));
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float2 f = e4m3x2_to_f32(w >> (8 * e));
        v[e] = f.x, v[e + 1] = f.y;
    }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) paged_simt_kernel(PagedArgs a, DevCtx ctx) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (long long)a.T * a.H) return;
    const int t = (int)(row / a.H), h = (int)(row % a.H), g = h / (a.H / a.Hkv);
    const int b = warp_find(a.B, t, [&](int i) { return (long long)__ldg(a.cu_seqlens + i); });
    PagedSeq s;
    if (!load_seq(a.cu_seqlens, a.kv_lens, b, a.T, (long long)a.max_pages * a.page, s)) {
        if (lane == 0) record_error(ctx, DEVERR_SEQLENS);
        return;
    }
    if (t - s.t0 < 0 || t - s.t0 >= s.n) return;  // behind the last sequence
    const int pos = s.len - s.n + (t - s.t0);
    const int hi = a.causal ? pos : s.len - 1;
    const int lo = a.window_left < 0 ? 0 : max(0, pos - a.window_left);
    const float qs = a.scale * LOG2E;
    const float sink = a.sinks ? sink_log2(__ldg(a.sinks + h)) : 0.f;
    float q[E], acc[E];
    const float *qrow = static_cast<const float *>(a.q) + (size_t)t * a.q_stride + (size_t)h * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = qrow[e] * qs;
        acc[e] = 0.f;
    }
    float m = a.sink_mode == 2 ? sink : -INFINITY, l = a.sink_mode == 2 ? 1.f : 0.f;
    float unit = 7.888609052210118e-31f, per_unit = 1.f / unit;  // 2^-100
    const int32_t *pages = a.page_table + (size_t)b * a.max_pages;
    bool bad = false;
    for (int j = lo; j <= hi; ++j) {
        const int pid = __ldg(pages + j / a.page);
        if (pid < 0 || pid >= a.num_pages) {
            bad = true;
            continue;
        }
        const size_t ph = (size_t)pid * a.Hkv + g;
        const size_t at = (ph * a.page + j % a.page) * D + lane * E;
        float kv[E];
        load_codes<E>(a.k_cache + at, kv);
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x += q[e] * kv[e];
        x = warp_sum(x) * __ldg(a.k_scale + ph);
        if (a.sink_mode == 1 && j == 0) x += sink;
        if (x == -INFINITY) continue;  // weight 0, whatever the running maximum
        const float mn = fmaxf(m, x);
        const float alpha = m == -INFINITY ? 0.f : ex2(m - mn), p = ex2(x - mn);
        load_codes<E>(a.v_cache + at, kv);
        const float vs = __ldg(a.v_scale + ph);
        if (vs >= 2.f * unit) {
            const float larger = __uint_as_float(__float_as_uint(vs) & 0x7f800000u);
            per_unit = 1.f / larger;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= unit * per_unit;
            unit = larger;
        }
        const float pv = p * (vs * per_unit);
        l = l * alpha + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * alpha + pv * kv[e];
        m = mn;
    }
    if (bad && lane == 0) record_error(ctx, DEVERR_INDEX);
    // l > 0 unless the row saw nothing; a NaN logit makes l NaN and goes out as NaN
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float *orow = static_cast<float *>(a.o) + (size_t)row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) orow[e] = acc[e] * inv * unit;
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

}  // namespace

cudaError_t launch_paged_simt(const PagedArgs &a, const DevInfo &dev, cudaStream_t s) {
    const long long blocks = ((long long)a.T * a.H + kWarps - 1) / kWarps;
    const DevCtx ctx = make_ctx(dev);
    if (a.d == 64) paged_simt_kernel<64><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a, ctx);
    else paged_simt_kernel<128><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a, ctx);
    return cudaGetLastError();
}

}  // namespace sattn
