// Cross attention to encoder states and its key weights, one warp a query row and one
// thread a key: every type, fp32 throughout.
//
// cross_simt: each lane holds d / 32 neighbouring columns of the query and of the
// accumulator; the row walks its states with an online softmax in the log2 domain.
// weights_simt: a block takes 128 keys of a sequence and KV head, a thread each, the key in
// registers; the rows of the group pass through shared memory, 16 at a time.
//
// Bound by the chain of one key at a time and by fp32 arithmetic: the exact fp32 form, the
// bf16 kernels are the fast ones (16 prompts of 17 to 900 queries over 257 to 4100 states, 32 heads
// on 8, d = 128: 47 ms against 0.18; 64 single tokens over 257 to 6404 4.8 against 0.15, their key
// weights 1.1 against 0.09). bf16 comes here without states, where no tensor map can be
// made, and the weights also without queries.
#include <math.h>

#include "internal.h"
#include "paged.cuh"
#include "states.cuh"

namespace sattn {
namespace {

constexpr int kWarps = 4;
constexpr int KEYS = 128, STAGED = 16;

template <typename T, int E> __device__ __forceinline__ void load(const T *p, float (&v)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = to_f32<T>(p[e]);
}

// Reports malformed sequences, those without queries too. A block.
__device__ __noinline__ void report_bad(const CrossArgs &a, const DevCtx &ctx) {
    StateSeq s;
    bool bad = false;
    for (int b = threadIdx.x; b < a.B; b += kWarps * 32)
        bad |= !load_states(a.cu_seqlens, a.kv_starts, a.kv_lens, b, a.T, a.S, s);
    if (bad) record_error(ctx, DEVERR_SEQLENS);
}

// The first good sequence that has token t, or -1: where cu_seqlens falls, a search misses some.
// A warp.
__device__ __noinline__ int first_with(const CrossArgs &a, int t) {
    const int lane = threadIdx.x & 31;
    StateSeq s;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const bool has = b0 + lane < a.B &&
                         load_states(a.cu_seqlens, a.kv_starts, a.kv_lens, b0 + lane, a.T, a.S, s) &&
                         t >= s.t0 && t - s.t0 < s.n;
        const uint32_t found = __ballot_sync(0xffffffffu, has);
        if (found) return b0 + __ffs(found) - 1;
    }
    return -1;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) cross_simt_kernel(CrossArgs a, DevCtx ctx) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0) report_bad(a, ctx);
    const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (long long)a.T * a.H) return;
    const int t = (int)(row / a.H), h = (int)(row % a.H), g = h / (a.H / a.Hkv);
    const int b = warp_find(a.B, t, [&](int i) { return (long long)__ldg(a.cu_seqlens + i); });
    StateSeq s;
    if (!load_states(a.cu_seqlens, a.kv_starts, a.kv_lens, b, a.T, a.S, s) || t < s.t0 ||
        t - s.t0 >= s.n) {
        const int other = first_with(a, t);
        if (other < 0) return;  // of no sequence, or of one that is skipped
        load_states(a.cu_seqlens, a.kv_starts, a.kv_lens, other, a.T, a.S, s);
    }
    const float sink = a.sinks ? state_sink(__ldg(a.sinks + h)) : 0.f;
    float q[E], acc[E], kv[E];
    load<T, E>(static_cast<const T *>(a.q) + (size_t)t * a.q_stride + (size_t)h * D + lane * E, q);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] *= a.scale * LOG2E;
        acc[e] = 0.f;
    }
    float m = a.sink_mode == 2 ? sink : -INFINITY, l = a.sink_mode == 2 && sink != -INFINITY;
    const T *k = static_cast<const T *>(a.k) + (size_t)s.s0 * a.k_stride + (size_t)g * D + lane * E;
    const T *v = static_cast<const T *>(a.v) + (size_t)s.s0 * a.v_stride + (size_t)g * D + lane * E;
    for (int j = 0; j < s.len; ++j, k += a.k_stride, v += a.v_stride) {
        load<T, E>(k, kv);
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x += q[e] * kv[e];
        x = warp_sum(x);
        if (a.sink_mode == 1 && j == 0) x += sink;
        load<T, E>(v, kv);
        // (weight 0 for -inf, whatever the running maximum; times a NaN value it is NaN)
        const float mn = fmaxf(m, x);
        const float alpha = m == -INFINITY ? 0.f : ex2(m - mn);
        const float p = x == -INFINITY ? 0.f : ex2(x - mn);
        l = l * alpha + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * alpha + p * kv[e];
        m = mn;
    }
    // l > 0 unless the row saw nothing; a NaN logit makes l NaN and goes out as NaN
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *orow = static_cast<T *>(a.o) + (size_t)row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) orow[e] = from_f32<T>(acc[e] * inv);
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

template <typename T, int D>
__global__ void __launch_bounds__(KEYS) weights_simt_kernel(KeyWeightArgs a, DevCtx ctx) {
    __shared__ float rows[STAGED][D], lse2[STAGED], sinks[STAGED];
    const int G = a.H / a.Hkv;
    long long unit = blockIdx.x;  // of all sequences' (head, key tile)
    for (int b = 0; b < a.B; ++b) {
        StateSeq s;
        if (!load_states(a.cu_seqlens, a.kv_starts, a.kv_lens, b, a.T, a.S, s)) {
            if (blockIdx.x == 0 && threadIdx.x == 0) record_error(ctx, DEVERR_SEQLENS);
            continue;
        }
        const int tiles = (s.len + KEYS - 1) / KEYS;
        const long long units = (long long)tiles * a.Hkv;
        for (; unit < units; unit += gridDim.x) {
            const int h = (int)(unit / tiles), key = (int)(unit % tiles) * KEYS + threadIdx.x;
            const bool in = key < s.len;
            float k[D], w = 0.f;
            load<T, D>(static_cast<const T *>(a.k) + (size_t)(s.s0 + min(key, s.len - 1)) * a.k_stride +
                           (size_t)h * D, k);
            const long long n = (long long)s.n * G;
            for (long long r0 = 0; r0 < n; r0 += STAGED) {
                __syncthreads();
                for (int e = threadIdx.x; e < STAGED * D; e += KEYS) {
                    const long long r = r0 + e / D;
                    const int t = (int)(r / G), g = (int)(r % G);
                    rows[e / D][e % D] = r < n ? a.scale * LOG2E *
                        to_f32<T>(static_cast<const T *>(a.q)[(size_t)(s.t0 + t) * a.q_stride +
                                                              (size_t)(h * G + g) * D + e % D]) : 0.f;
                }
                if (threadIdx.x < STAGED) {
                    const long long r = r0 + threadIdx.x;
                    const int head = h * G + (int)(r % G);
                    float x = INFINITY;  // a row without a denominator weighs nothing
                    if (r < n) x = a.lse[(size_t)(s.t0 + r / G) * a.H + head] * LOG2E;
                    lse2[threadIdx.x] = x == -INFINITY ? INFINITY : x;
                    sinks[threadIdx.x] = a.sinks ? state_sink(__ldg(a.sinks + head)) : 0.f;
                }
                __syncthreads();
                const int c = (int)min((long long)STAGED, n - r0);
                for (int r = 0; r < c; ++r) {
                    float x = 0.f;
#pragma unroll
                    for (int e = 0; e < D; ++e) x += rows[r][e] * k[e];
                    if (a.sink_mode == 1 && key == 0) x += sinks[r];
                    x -= lse2[r];
                    if (x > 0.f) x = 0.f;  // (by the rounding of a large lse; a NaN stays)
                    w += lse2[r] == INFINITY ? 0.f : ex2(x);
                }
            }
            if (in) {
                float *at = a.weights + (size_t)h * a.S + s.s0 + key;
                *at = a.accumulate ? *at + w : w;
            }
        }
        unit -= units;
    }
}

}  // namespace

cudaError_t launch_cross_simt(const CrossArgs &a, const DevInfo &dev, cudaStream_t s) {
    const unsigned blocks = (unsigned)(((long long)a.T * a.H + kWarps - 1) / kWarps);
    const DevCtx ctx = make_ctx(dev);
    if (a.dtype == SATTN_F32) {
        if (a.d == 64) cross_simt_kernel<float, 64><<<blocks, kWarps * 32, 0, s>>>(a, ctx);
        else cross_simt_kernel<float, 128><<<blocks, kWarps * 32, 0, s>>>(a, ctx);
    } else {
        if (a.d == 64) cross_simt_kernel<__nv_bfloat16, 64><<<blocks, kWarps * 32, 0, s>>>(a, ctx);
        else cross_simt_kernel<__nv_bfloat16, 128><<<blocks, kWarps * 32, 0, s>>>(a, ctx);
    }
    return cudaGetLastError();
}

cudaError_t launch_weights_simt(const KeyWeightArgs &a, const DevInfo &dev, cudaStream_t s) {
    const unsigned blocks = 4u * (unsigned)dev.sm_count;
    const DevCtx ctx = make_ctx(dev);
    if (a.dtype == SATTN_F32) {
        if (a.d == 64) weights_simt_kernel<float, 64><<<blocks, KEYS, 0, s>>>(a, ctx);
        else weights_simt_kernel<float, 128><<<blocks, KEYS, 0, s>>>(a, ctx);
    } else {
        if (a.d == 64) weights_simt_kernel<__nv_bfloat16, 64><<<blocks, KEYS, 0, s>>>(a, ctx);
        else weights_simt_kernel<__nv_bfloat16, 128><<<blocks, KEYS, 0, s>>>(a, ctx);
    }
    return cudaGetLastError();
}

}  // namespace sattn
