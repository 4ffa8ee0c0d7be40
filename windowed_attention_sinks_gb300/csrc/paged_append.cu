// Append to a paged e4m3 cache, the position rotation applied on the way.
//
// For every new token at position p of its sequence and every KV head: the key
// is rotated by the table's angles of p, and key and value go to row p mod page
// of the page that the page table names for p / page, as e4m3 codes of x / s.
// s is the scale of that page and head, the least power of two with
// amax <= 448 s over everything the page holds. A page's first row sets s; rows
// that join a page later may raise it, and then the codes already there are
// recoded by old / new. With powers of two that is exact (a shift of the
// exponent) until a code falls below the normal range, and x / s is exact too,
// so a value is rounded once: relative error at most 2^-4 of e4m3, as with an
// amax / 448 scale, of which a power of two costs at most one bit of range.
//
// One unit of work is (page touched, key or value, KV head): its amax must be
// known before the first code is written, so NT threads hold the rows as they
// were read (up to HELD items of 16 columns each), take the amax over the group
// and then write, turning the keys a second time rather than keeping them in fp32: what
// counts is how much is in flight, and that goes by the registers. Rows
// beyond HELD are read again (they are in L2 by then). Two
// ways to number the pages that a call touches, from its sizes alone:
//   few tokens a sequence:  unit = token, dropped unless it is the first of
//                           the call in its page; NT = 32;
//   prompts:                sequence b owns the units from
//                           cu[b] / page + 2 b on (a run of n tokens touches
//                           at most n / page + 2 pages).
// (256 single tokens: 7.3 us by tokens, 23 by sequences; prompts 106 and 54.)
// The queries of the same tokens are rotated by further blocks of the launch.
// An item is 16 columns: the two 8-column halves that rotate into one another,
// or 16 neighbours, so all global accesses are 8 or 16 bytes wide.
//
// Bound by bytes in flight. 16 prompts of 33 .. 1777 tokens, bf16, 32 heads on 8, d = 128,
// pages of 64: 54 us for 273 MB, 0.77 of the copy rate; four of 7001 .. 8192, fp32, 16
// heads on 4, d = 64, pages of 16: 71 us, 0.68; 4 single tokens 3.9 us, latency. A group
// loads its unit's rows, waits for them and stores once, with nothing of the next unit in
// flight; three blocks an SM leave 80 registers a thread, of which 28 to 80 bytes spill.
#include "internal.h"
#include "paged.cuh"

namespace sattn {
namespace {

constexpr int THREADS = 256;
// Eight values as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        a = __ldg(reinterpret_cast<const uint4 *>(p));
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
// Items that a thread holds: 128 bytes.
template <typename T> constexpr int HELD = sizeof(T) == 2 ? 4 : 2;
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    Raw8<float> r;
    r.load(p);
    r.get(v);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// First columns of the two halves of item c of a row.
struct Cols {
    int a, b;
    bool turn;
};
__device__ __forceinline__ Cols item_cols(int c, int rd, int interleaved) {
    const bool turn = 16 * c < rd;
    if (turn && !interleaved) return Cols{8 * c, 8 * c + rd / 2, true};
    return Cols{16 * c, 16 * c + 8, turn};
}

// Pairs (a[i], b[i]), or neighbours within a and within b, turned by the angles
// 8c .. 8c + 7 of the row's table entry.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&cs)[8],
                                     const float (&sn)[8], int interleaved) {
    if (!interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * cs[i] - y * sn[i];
            b[i] = y * cs[i] + x * sn[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = a[2 * i], y = a[2 * i + 1];
            a[2 * i] = x * cs[i] - y * sn[i];
            a[2 * i + 1] = y * cs[i] + x * sn[i];
            x = b[2 * i], y = b[2 * i + 1];
            b[2 * i] = x * cs[4 + i] - y * sn[4 + i];
            b[2 * i + 1] = y * cs[4 + i] + x * sn[4 + i];
        }
    }
}

__device__ __forceinline__ float amax16(const float (&a)[8], const float (&b)[8]) {
    float m = 0.f;  // max.f32 drops a NaN operand: a NaN does not set the scale
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max3(m, fabsf(a[i]), fabsf(b[i]));
    return m;
}

__device__ __forceinline__ uint2 code8(const float (&v)[8], float inv) {
    return make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                      e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// The sequence and its checks that an append needs beyond load_seq's.
__device__ __forceinline__ bool append_seq(const PagedAppendArgs &p, int b, PagedSeq &s,
                                           unsigned &err) {
    if (!load_seq(p.cu_seqlens, p.kv_lens, b, p.T, (long long)p.max_pages * p.page, s) ||
        s.len < s.n) {
        err |= DEVERR_SEQLENS;
        return false;
    }
    if (p.rd > 0 && s.len > p.rope_rows) {
        err |= DEVERR_INDEX;
        return false;
    }
    return true;
}

template <typename T, int NT>
__device__ __forceinline__ void append_unit(const PagedAppendArgs &p, long long u, float *red,
                                            unsigned &err) {
    const int tid = threadIdx.x % NT;
    const int h = (int)(u % p.Hkv);
    const bool is_v = u / p.Hkv & 1;
    const long long x = u / p.Hkv >> 1;
    // the pages's sequence and its first new position in the page
    int b;
    PagedSeq s;
    int pos;
    if (p.by_token) {
        b = warp_find(p.B, x, [&](int i) { return (long long)__ldg(p.cu_seqlens + i); });
        if (!append_seq(p, b, s, err)) return;
        const int i = (int)x - s.t0;
        if (i < 0 || i >= s.n) return;  // behind the last sequence
        pos = s.len - s.n + i;
        if (i > 0 && pos % p.page != 0) return;  // not the first in its page
    } else {
        b = warp_find(p.B, x, [&](int i) {
            return (long long)(__ldg(p.cu_seqlens + i) / p.page) + 2ll * i;
        });
        if (!append_seq(p, b, s, err)) return;
        const long long j = x - (s.t0 / p.page + 2ll * b);
        const int p0 = s.len - s.n;
        const long long first = j == 0 ? p0 : ((long long)(p0 / p.page) + j) * p.page;
        if (s.n == 0 || first >= s.len) return;
        pos = (int)first;
    }
    const int row0 = pos % p.page;
    const int rows = min(p.page - row0, s.len - pos);
    const int pid = __ldg(p.page_table + (size_t)b * p.max_pages + pos / p.page);
    const T *src = static_cast<const T *>(is_v ? p.v : p.k) +
                   (size_t)(s.t0 + pos - (s.len - s.n)) * (is_v ? p.v_stride : p.k_stride) +
                   (size_t)h * p.d;
    const size_t stride = is_v ? p.v_stride : p.k_stride;
    const int ic = p.d / 16, items = rows * ic, rd = is_v ? 0 : p.rd;

    using Raw = Raw8<T>;
    auto fetch = [&](int it, Raw &a, Raw &b2) {
        const int r = it / ic, c = it % ic;
        const Cols k = item_cols(c, rd, p.interleaved);
        a.load(src + r * stride + k.a);
        b2.load(src + r * stride + k.b);
    };
    auto values = [&](int it, const Raw &x, const Raw &y, float (&a)[8], float (&bb)[8]) {
        x.get(a);
        y.get(bb);
        const int r = it / ic, c = it % ic;
        if (16 * c < rd) {
            float cs[8], sn[8];
            const float *e = p.cos_sin + (size_t)(pos + r) * p.rd + 8 * c;
            load8(e, cs);
            load8(e + p.rd / 2, sn);
            turn(a, bb, cs, sn, p.interleaved);
        }
    };

    constexpr int N = HELD<T>;
    Raw ra[N], rb[N];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (tid + k * NT < items) fetch(tid + k * NT, ra[k], rb[k]);
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (tid + k * NT < items) {
            float y[8], z[8];
            values(tid + k * NT, ra[k], rb[k], y, z);
            amax = fmaxf(amax, amax16(y, z));
        }
#pragma unroll 1
    for (int it = tid + N * NT; it < items; it += NT) {
        Raw x0, x1;
        float y[8], z[8];
        fetch(it, x0, x1);
        values(it, x0, x1, y, z);
        amax = fmaxf(amax, amax16(y, z));
    }
    if (pid < 0 || pid >= p.num_pages) {  // the same for the whole unit
        err |= DEVERR_INDEX;
        return;
    }
    float *scale = (is_v ? p.v_scale : p.k_scale) + (size_t)pid * p.Hkv + h;
    const float old = row0 > 0 ? *scale : 0.f;
    amax = warp_max(amax);
    if (NT > 32) {
        constexpr int W = NT / 32;
        const int group = threadIdx.x / NT;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(NT) : "memory");
        amax = red[group * W];
#pragma unroll
        for (int w = 1; w < W; ++w) amax = fmaxf(amax, red[group * W + w]);
    } else {
        __syncwarp();  // every lane has read the old scale
    }
    float now = pow2_scale(amax);
    if (row0 > 0) {
        // the held scale as a power of two (it is one already unless the caller
        // filled the page): the least one not below it
        const uint32_t ob = __float_as_uint(old);
        const float held = old > 0.f ? __uint_as_float(min((ob + 0x7fffffu) & 0x7f800000u,
                                                           (uint32_t)(127 + 120) << 23))
                                     : LEAST_SCALE;
        now = fmaxf(now, held);
    }
    const float inv = __frcp_rn(now);  // exact: a power of two in [2^-64, 2^120]
    uint8_t *dst = (is_v ? p.v_cache : p.k_cache) + ((size_t)pid * p.Hkv + h) * p.page * p.d;
    auto put = [&](int it, const float (&y)[8], const float (&z)[8]) {
        const int r = it / ic;
        const Cols k = item_cols(it % ic, rd, p.interleaved);
        uint8_t *at = dst + (size_t)(row0 + r) * p.d;
        *reinterpret_cast<uint2 *>(at + k.a) = code8(y, inv);
        *reinterpret_cast<uint2 *>(at + k.b) = code8(z, inv);
    };
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (tid + k * NT < items) {
            float y[8], z[8];
            values(tid + k * NT, ra[k], rb[k], y, z);
            put(tid + k * NT, y, z);
        }
#pragma unroll 1
    for (int it = tid + N * NT; it < items; it += NT) {
        Raw x0, x1;
        float y[8], z[8];
        fetch(it, x0, x1);
        values(it, x0, x1, y, z);
        put(it, y, z);
    }
    if (row0 > 0 && now != old) {  // the page's other rows move to the new scale
        const float ratio = old * inv;
        const int from = row0 * p.d / 8, count = rows * p.d / 8;
        for (int k = tid; k < p.page * p.d / 8 - count; k += NT) {
            const int i = k < from ? k : k + count;
            uint2 w = reinterpret_cast<uint2 *>(dst)[i];
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = e4m3x2_to_f32((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
                v[2 * e] = f.x, v[2 * e + 1] = f.y;
            }
            reinterpret_cast<uint2 *>(dst)[i] = code8(v, ratio);
        }
    }
    if (tid == 0) *scale = now;
}

// Threads that rotate the queries of a token: 64, or 32 where so few items make
// HELD for each of those.
template <typename T> __host__ __device__ constexpr int query_threads(int H, int d) {
    return H * (d / 16) <= 32 * HELD<T> ? 32 : 64;
}

// Rotated queries of a token; a thread keeps its columns' angles for its heads,
// and loads up to HELD of them before it needs to know the token's position.
template <typename T>
__device__ __forceinline__ void rotate_queries(const PagedAppendArgs &p, long long t, int threads,
                                               unsigned &err) {
    if (t >= p.T) return;
    constexpr int N = HELD<T>;
    const int ic = p.d / 16, c = threadIdx.x % ic, lanes = threads / ic, h0 = threadIdx.x % threads / ic;
    const Cols k = item_cols(c, p.rd, p.interleaved);
    const T *src = static_cast<const T *>(p.q) + (size_t)t * p.q_stride;
    T *dst = static_cast<T *>(p.q_out) + (size_t)t * p.H * p.d;
    Raw8<T> a[N], b[N];
    auto fetch = [&](int h) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (h + i * lanes < p.H) {
                a[i].load(src + (size_t)(h + i * lanes) * p.d + k.a);
                b[i].load(src + (size_t)(h + i * lanes) * p.d + k.b);
            }
    };
    fetch(h0);
    const int bs = warp_find(p.B, t, [&](int i) { return (long long)__ldg(p.cu_seqlens + i); });
    PagedSeq s;
    if (!append_seq(p, bs, s, err)) return;
    const int i0 = (int)t - s.t0;
    if (i0 < 0 || i0 >= s.n) return;
    const int pos = s.len - s.n + i0;
    float cs[8], sn[8];
    if (k.turn) {
        const float *e = p.cos_sin + (size_t)pos * p.rd + 8 * c;
        load8(e, cs);
        load8(e + p.rd / 2, sn);
    }
#pragma unroll 1
    for (int h = h0; h < p.H; h += N * lanes) {
        if (h > h0) fetch(h);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (h + i * lanes < p.H) {
                float x[8], y[8];
                a[i].get(x);
                b[i].get(y);
                if (k.turn) turn(x, y, cs, sn, p.interleaved);
                store8(dst + (size_t)(h + i * lanes) * p.d + k.a, x);
                store8(dst + (size_t)(h + i * lanes) * p.d + k.b, y);
            }
    }
}

template <typename T, int NT>
__global__ void __launch_bounds__(THREADS, 3) append_kernel(const PagedAppendArgs p, const DevCtx ctx) {
    __shared__ float red[THREADS / 32];
    unsigned err = 0;
    if (blockIdx.x < p.unit_blocks) {
        const long long u = (long long)blockIdx.x * (THREADS / NT) + threadIdx.x / NT;
        if (u < p.units) append_unit<T, NT>(p, u, red, err);
    } else {
        const int n = query_threads<T>(p.H, p.d);
        rotate_queries<T>(
            p, (long long)(blockIdx.x - p.unit_blocks) * (THREADS / n) + threadIdx.x / n, n, err);
    }
    if (err && (threadIdx.x & 31) == 0) record_error(ctx, err);
}

template <typename T, int NT>
cudaError_t launch(PagedAppendArgs p, const DevInfo &dev, cudaStream_t s) {
    const long long ub = (p.units + THREADS / NT - 1) / (THREADS / NT);
    const int per = p.q ? THREADS / query_threads<T>(p.H, p.d) : 1;
    const long long qb = p.q ? ((long long)p.T + per - 1) / per : 0;
    if (ub + qb > INT_MAX) return cudaErrorInvalidValue;
    p.unit_blocks = (unsigned)ub;
    append_kernel<T, NT><<<(unsigned)(ub + qb), THREADS, 0, s>>>(p, make_ctx(dev));
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(PagedAppendArgs p, const DevInfo &dev, cudaStream_t s) {
    const long long slots = p.T / p.page + 2ll * p.B;
    p.by_token = p.T <= slots;
    p.units = (p.by_token ? p.T : slots) * 2 * p.Hkv;
    // whole pages: as many threads as hold one in registers. (Groups of 32, 64, 128, 256
    // threads: the bf16 prompts above 58, 53, 54, 63 us, where this gives 128; the fp32
    // ones 72, 79, 102, 147, where it gives 32.)
    const int want = p.by_token ? 32 : p.page * p.d / (16 * HELD<T>);
    if (want <= 32) return launch<T, 32>(p, dev, s);
    if (want <= 64) return launch<T, 64>(p, dev, s);
    if (want <= 128) return launch<T, 128>(p, dev, s);
    return launch<T, 256>(p, dev, s);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs &a, const DevInfo &dev, cudaStream_t s) {
    return a.dtype == SATTN_BF16 ? pick<__nv_bfloat16>(a, dev, s) : pick<float>(a, dev, s);
}

}  // namespace sattn
