// Rotary positions with several axes, queries and keys in one launch.
//
// Column pair i of a head turns by the angle positions[axis[i]][t] * inv_freq[i]:
// (a, b) -> (a cos - b sin, b cos + a sin), or the other way round (the transpose, which
// is also the backward pass). The angle is taken in turns, modulo one, in 64-bit fixed
// point: with F = inv_freq / 2 pi as a fraction of 2^64, position * F mod 2^64 is the
// fraction of a turn, exact for the integer position but for F's own rounding. fp32 would
// lose far positions (at 10^5 it resolves a hundredth of a radian), fp64 runs at 2
// operations a cycle and SM here. The angle's nearest quarter is split off in
// integers, so that what goes to sincospif is at most 1/8 turn and as fine as fp32.
//
// A block takes a few tokens: first the cosines and sines of all their pairs, once for all
// heads, into shared memory, then the heads, two 16-byte vectors an item: the
// vectors that turn into one another (halves), or neighbours; the first ones are on their way
// while the angles are computed.
//
// Bound by memory: 65521 tokens of 32 heads, fp32, d = 64: 159 us for 1.07 GB, 0.99 of the copy
// rate; 14343 tokens of 24 bf16 heads out of rows of 32, d = 128: 35 us for 176 MB, 0.74 (blocks of
// 256 threads 37, of 512 43; eight rows a thread in a block 37). 16 tokens: 4.4 us, latency.
#include "internal.h"

namespace sattn {
namespace {

constexpr int THREADS = 128;
constexpr int MAX_HALF = 128;  // pairs a head
constexpr int MAX_TOKENS = 16;  // tokens a block

// x / n for 0 <= x < 2^31: with s = ceil(log2 n), mul = 2^32 (2^s - n) / n + 1,
// x / n = (high(mul x) + x) >> s.
struct FastDiv {
    uint32_t n, mul, shift;
    __device__ __forceinline__ int div(int x) const {
        return (int)((__umulhi(mul, (uint32_t)x) + (uint32_t)x) >> shift);
    }
};
FastDiv fast_div(uint32_t n) {
    uint32_t s = 0;
    while ((1ull << s) < n) ++s;
    return FastDiv{n, (uint32_t)((((1ull << s) - n) << 32) / n + 1), s};
}

struct Args {
    RopeArgs r;
    int tokens, heads;   // a block
    FastDiv head, items, half;
    int turned, copied;  // items a head that turn; vectors a head behind column rd
};

// f / (2 pi) as a fraction of 2^64: the float's 24-bit integer times 2^64 / (2 pi), shifted
// by its exponent. Off by less than 2^-64 (what is shifted out) + 2^-65 |f| (C's own rounding).
__device__ __forceinline__ uint64_t turns(float f) {
    const uint32_t b = __float_as_uint(f);
    const int e = (int)(b >> 23 & 255);
    const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const uint64_t C = 0x28be60db9391054aull;  // 2^64 / (2 pi)
    const uint64_t lo = m * C, hi = __umul64hi(m, C);
    const int s = 150 - (e ? e : 1);  // f = m 2^-s
    uint64_t r;
    if (s <= 0) r = s > -64 ? lo << -s : 0;
    else if (s < 64) r = hi << (64 - s) | lo >> s;
    else r = s < 128 ? hi >> (s - 64) : 0;
    return b >> 31 ? 0 - r : r;
}

__device__ __forceinline__ float2 cos_sin(float f, int pos) {
    const uint64_t a = (uint64_t)(int64_t)pos * turns(f);
    const uint32_t quarter = (uint32_t)((a + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(a - ((uint64_t)quarter << 62));  // in +-2^61
    float s, c;
    sincospif((float)(int)(rest >> 31) * 2.3283064365386963e-10f, &s, &c);  // 2 rest 2^-64
    const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

template <typename T> struct Vec;  // 16 bytes
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &x, float (&v)[4]) {
        v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &x, float (&v)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                          pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
};

// Two vectors of a head, on their way.
template <typename T> struct Item {
    const T *src;
    T *dst;
    uint4 x, y;
    int tok, c, off;  // token of the block, item of the head, distance of the vectors
    bool two;

    template <bool NEIGHBOURS>
    __device__ __forceinline__ void load(const Args &a, long long t0, int h0, int e, int total) {
        constexpr int N = Vec<T>::N;
        const RopeArgs &r = a.r;
        src = nullptr;
        if (e >= total) return;
        const int th = a.items.div(e);
        c = e - th * (int)a.items.n;
        tok = a.head.div(th);
        const int h = h0 + th - tok * (int)a.head.n;
        const bool key = h >= r.H;
        const size_t t = (size_t)(t0 + tok);
        const T *in = key ? (const T *)r.k + t * r.k_stride + (size_t)(h - r.H) * r.d
                          : (const T *)r.q + t * r.q_stride + (size_t)h * r.d;
        T *out = key ? (T *)r.k_out + t * r.k_out_stride + (size_t)(h - r.H) * r.d
                     : (T *)r.q_out + t * r.q_out_stride + (size_t)h * r.d;
        const bool turn = c < a.turned;
        const int first =
            turn ? (NEIGHBOURS ? 2 * N * c : N * c) : r.rd + 2 * N * (c - a.turned);
        off = turn && !NEIGHBOURS ? r.rd / 2 : N;
        two = turn || 2 * (c - a.turned) + 1 < a.copied;
        dst = out + first;
        if (!turn && in == out) return;  // in place: these columns stay
        src = in + first;
        x = *reinterpret_cast<const uint4 *>(src);
        if (two) y = *reinterpret_cast<const uint4 *>(src + off);
    }
    template <bool NEIGHBOURS>
    __device__ __forceinline__ void turn(const Args &a, const float2 *table) {
        constexpr int N = Vec<T>::N;
        if (!src) return;
        if (c < a.turned) {
            const float2 *cs = table + tok * (a.r.rd / 2) + c * N;
            float p[N], q[N];
            Vec<T>::get(x, p);
            Vec<T>::get(y, q);
            if (NEIGHBOURS) {
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float2 w = cs[i / 2], z = cs[N / 2 + i / 2];
                    const float p0 = p[i], q0 = q[i];
                    p[i] = p0 * w.x - p[i + 1] * w.y;
                    p[i + 1] = p[i + 1] * w.x + p0 * w.y;
                    q[i] = q0 * z.x - q[i + 1] * z.y;
                    q[i + 1] = q[i + 1] * z.x + q0 * z.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float2 w = cs[i];
                    const float p0 = p[i];
                    p[i] = p0 * w.x - q[i] * w.y;
                    q[i] = q[i] * w.x + p0 * w.y;
                }
            }
            x = Vec<T>::put(p);
            y = Vec<T>::put(q);
        }
        *reinterpret_cast<uint4 *>(dst) = x;
        if (two) *reinterpret_cast<uint4 *>(dst + off) = y;
    }
};

template <typename T, bool NEIGHBOURS>
__global__ void __launch_bounds__(THREADS, 10) rope_axes_kernel(const __grid_constant__ Args a,
                                                            const __grid_constant__ DevCtx ctx) {
    extern __shared__ float2 table[];  // [tokens][rd / 2]
    const RopeArgs &r = a.r;
    const int half = r.rd / 2;
    const long long t0 = (long long)blockIdx.x * a.tokens;
    const int nt = (int)min((long long)a.tokens, r.T - t0), h0 = (int)blockIdx.y * a.heads;
    const int total = nt * (int)(a.head.n * a.items.n);
    constexpr int B = 2;  // items in flight a thread
    Item<T> it[B];
    int e = threadIdx.x;
    // the first ones are on their way while the angles are computed
#pragma unroll
    for (int u = 0; u < B; ++u) it[u].template load<NEIGHBOURS>(a, t0, h0, e + u * THREADS, total);
    for (int x = threadIdx.x; x < nt * half; x += THREADS) {
        const int t = a.half.div(x), i = x - t * half;
        const int axis = __ldg(r.axis + i);
        float2 cs = make_float2(1.f, 0.f);
        if (axis < r.axes) {
            const float f = __ldg(r.inv_freq + i);
            cs = cos_sin(f, __ldg(r.positions + (size_t)axis * r.T + t0 + t));
            if (f - f != 0.f) cs = make_float2(NAN, NAN);
        } else if (blockIdx.x == 0) {
            record_error(ctx, DEVERR_INDEX);
        }
        table[x] = make_float2(cs.x, r.inverse ? -cs.y : cs.y);
    }
    __syncthreads();
    for (;;) {
#pragma unroll
        for (int u = 0; u < B; ++u) it[u].template turn<NEIGHBOURS>(a, table);
        e += B * THREADS;
        if (e >= total) break;
#pragma unroll
        for (int u = 0; u < B; ++u)
            it[u].template load<NEIGHBOURS>(a, t0, h0, e + u * THREADS, total);
    }
}

template <typename T> cudaError_t launch(const RopeArgs &r, const DevInfo &dev, cudaStream_t s) {
    constexpr int N = Vec<T>::N;
    const int heads = r.H + (r.k ? r.Hkv : 0);
    Args a;
    a.r = r;
    a.turned = r.rd / (2 * N);
    a.copied = (r.d - r.rd) / N;
    const int items = a.turned + (a.copied + 1) / 2;
    // Blocks of about 512 items (four a thread); with few tokens a token's heads are spread
    // over several (16 tokens, 40 heads of 128: 6.2 us in blocks of 3 tokens).
    const long long per_token = (long long)heads * items;
    a.tokens = (int)max(1ll, min((long long)MAX_TOKENS, 4 * THREADS / per_token));
    while (a.tokens > 1 && (r.T + a.tokens - 1) / a.tokens < 2 * dev.sm_count) a.tokens /= 2;
    const long long blocks = ((long long)r.T + a.tokens - 1) / a.tokens;
    const int want = (int)max(1ll, min(per_token / THREADS, 2 * dev.sm_count / blocks));
    int split = 1;  // of the heads, evenly
    for (int i = 2; i <= want; ++i)
        if (heads % i == 0) split = i;
    a.heads = heads / split;
    a.head = fast_div(a.heads);
    a.items = fast_div(items);
    a.half = fast_div(r.rd / 2);
    const size_t smem = (size_t)a.tokens * (r.rd / 2) * sizeof(float2);  // 16 KB at most
    const dim3 grid((unsigned)blocks, (unsigned)split);
    if (r.interleaved) rope_axes_kernel<T, true><<<grid, THREADS, smem, s>>>(a, make_ctx(dev));
    else rope_axes_kernel<T, false><<<grid, THREADS, smem, s>>>(a, make_ctx(dev));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_axes(const RopeArgs &r, const DevInfo &dev, cudaStream_t s) {
    static_assert(MAX_TOKENS * MAX_HALF * sizeof(float2) <= 48 * 1024, "shared memory of a block");
    return r.dtype == SATTN_BF16 ? launch<__nv_bfloat16>(r, dev, s) : launch<float>(r, dev, s);
}

}  // namespace sattn
