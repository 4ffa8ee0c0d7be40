// Attention of a few tokens a sequence over the paged e4m3 cache (tcgen05).
//
// o_r = sum_j softmax_j(scale <q_r, k_j>) v_j over a unit's R query rows (the
// heads of a KV group times the call's tokens), 128 keys a tile. With so few
// rows a key is used once or twice per byte, so the bound is reading the codes
// from HBM, and everything is arranged around one pass over them:
//
//  * The codes go into the tensor core as they are; nothing is widened in
//    shared memory. Both products are taken with the keys (then the columns of V) as the
//    128 rows of the MMA and the query rows as its N columns:
//      S^T [128 keys, 2R]   = K [128, D]   Q^T,
//      O^T [D, 4R]         += V^T [D, 128] P^T   (V read column-major).
//  * An e4m3 operand has 4 significant bits, so Q is split: x = hi +
//    lo / 16 with hi = e4m3(x) and lo = e4m3(16 (x - hi)), side by side as 2R
//    columns, joined again in fp32. hi + lo / 16 has 8 significant bits, a
//    bf16's, for |x| from 2^-6 to 448, and an absolute error of at most 2^-14
//    below that. Each row of Q is scaled by a power of two so that its largest value is
//    in [128, 256): bf16 queries go in exactly down to 2^-14 of the row's largest.
//  * P needs range above all: a long tail of keys far below the largest weighs as much
//    as that, and what P V loses of each, the row sum counts. So P goes in as
//    e5m2 (kind::f8f6f4 takes its operands' types apart), in 4R columns: P = 2^(10 + e - m)
//    <= 2^15, with e the exponent below, in f16 and cut into t0 + t1 / 8 + t2 / 64 + t3 / 512.
//    An e5m2 is an f16's upper byte, so each term is the next byte of what the ones
//    before leave: 3 + 3 + 3 + 2 bits, all that f16 has, and no conversion. With 32 rows three
//    terms, of P rounded to 9 bits. Those bits hold down to 2^-14, which is 2^-24 of the
//    largest weight; below that P is off by at most 2^-23, 2^-33 of it. (Two e4m3 terms as for
//    Q lose all below 2^-18 of the largest: 32768 equal keys 13 nats below another one's
//    gave half of their share. A second pair of them for the rest of small P is right too,
//    but its conversions take drafted tokens from 102 to 200 us; these terms to 104.)
//  The extra columns are free: the MMA is a small part of the time a tile takes to arrive.
//  * A thread holds one key, so the page's scales are scalars to it: the key's multiplies S, the
//    value's goes into the exponent, e = scale log2(e) s + log2(v_scale), and
//    V's codes need no scaling. The row sum divides it out again.
//  * The running maximum m (of e) is moved only where a tile exceeds it by more
//    than 2^4, so a tile costs one block vote instead of a reduction over its
//    128 keys; O is rescaled in TMEM when it moves.
//
// One persistent CTA per SM (kernels that allocate TMEM run one) over an equal
// piece of the tiles (paged_plan.cuh):
//   warp 0      the units; TMA: K and V tiles, one copy a page, two rings of
//               STAGES tiles; the pages' scales
//   warps 1, 2  MMA issuers: S, and P V. (Every wait of such a thread costs it 100 to
//               200 cycles even if it is met; one thread for both took 1900 cycles a
//               tile, more than the tile takes to arrive.)
//   warp 3      Q of the next units, split and swizzled; the rows' addresses
//   warps 4-11  softmax: two groups of four, each with its own m, l, P and O^T.
//               They take the tiles of a unit in turn, so that one's exponentials
//               run beside the other's loads and votes, and are joined at its
//               end; a unit of at most SOLO tiles is one group's alone, and the
//               groups take such units in turn.
//
// Measured (32 heads on 8, d = 128, replayed graphs): 64 requests of 8001 .. 32768
// positions 411 us, the copy rate; 32 of 301 .. 8192 53.6 us, 0.73 of it; one of 1000 11.4 us,
// all latency; 3 to 5 drafted tokens for 32 of 1000 .. 16000 109 us, 0.65 (at a unit's
// end the ring of tiles is full and HBM waits). 128 requests with a window of 127 (64
// heads on 8, d = 64): 36.8 us, latency of units of two tiles. Of these, sums apart for far
// value scales cost 2 us of the last and 3 of the drafted tokens, and the counters' launch 1
// of each. (When first built, one thread for both products took 486 and 64 us on the
// first two, 410 and 57 with two.)
#include <limits.h>
#include <math.h>
#include <stdio.h>

#include "paged_mma.cuh"
#include "paged_plan.cuh"

namespace sattn {
namespace {

constexpr int NTHREADS = 384;
constexpr int SRING = 16;
constexpr int UNITS = 8;  // units handed on ahead
// Tiles of a unit that one group takes alone, at least 1 (a group needs a tile): with 1, 2
// and 4 the windowed requests above take 37.5, 36.9 and 37.0 us.
constexpr int SOLO = 2;
// P = 2^(BASE + e - m). One more would halve the floor, and m moves sooner: with 9, 10 and 11 the
// drafted tokens below take 103, 104 and 105 us, with four times their logits 116, 119 and 122.
constexpr float BASE = 10.f;
constexpr float LIMIT = 15.f;  // m moves when BASE + e - m exceeds this

struct DecodeParams {
    PlanArgs plan;
    const __nv_bfloat16 *q;
    int64_t q_stride;
    const uint8_t *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *page_table;
    int H, num_pages, page, page_shift, max_pages;
    int rows_total;  // first row behind the pool: a copy from there reads zeros
    float scale_l2;
    const float *sinks;
    int sink_mode;
    __nv_bfloat16 *o;
    float *lse;
    uint8_t *ws;
};

template <int D, int R> struct Cfg {
    static constexpr int N = 2 * R;  // columns of S: Q's hi and lo
    // P's terms: a fourth costs the 32 rows of drafted tokens 11 us of 110, fewer rows nothing.
    // Columns of O, and the bytes of a key's row of P (a power of two for the swizzle).
    static constexpr int TERMS = R <= 16 ? 4 : 3, NO = TERMS * R, PW = 4 * R;
    static constexpr uint32_t TILE_BYTES = TILE * D;
    // what shared memory holds beside Q and P: 160 KB of tiles, 192 KB with fewer rows
    static constexpr int STAGES = (R <= 16 ? 6 : 5) * (128 / D);
    static constexpr int SBUF = 4;  // S buffers
    // A unit's own cost, in tiles. With 0, 2, 4 and 6: 32 requests 65, 56, 54, 54 us, drafted
    // tokens 129, 120, 111, 106 us (their ends join and store four times the rows).
    static constexpr int EXTRA = R <= 16 ? 4 : 6;
    static constexpr int QB = R <= 8 ? 4 : 2;  // units whose Q is at hand
    static constexpr uint32_t O_COL = SBUF * N;
    static constexpr uint32_t USED = O_COL + 2 * NO;
    static constexpr uint32_t COLS = USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
};

template <int D, int R> struct alignas(1024) Smem {
    using C = Cfg<D, R>;
    uint8_t k[C::STAGES][C::TILE_BYTES];
    uint8_t v[C::STAGES][C::TILE_BYTES];
    uint8_t q[C::QB][C::N * D];
    uint8_t p[2][C::PW * TILE];
    float4 sc[SRING][8];        // page's k scale, log2 v scale, 1 / v scale, v scale > 0
    float wmax[2][4][R];        // column maxima of the warps
    float alpha[2][R];          // what a move of m multiplies l and O by
    // of a unit (by its Q buffer):
    alignas(16) float mx[C::QB][2][R];  // the groups' running maxima m
    // sums apart, where a group's last such unit is this one: their maxima and sums, of
    // each warp, and the m that the group's other sums are in terms of
    int apart[2];
    float fn[2][4][R], fl[2][4][R], fm[2][R];
    float lx[C::QB][2][4][R];   // the warps' row sums
    float wt[C::QB][2][R];      // what a row of each group's O^T is multiplied by
    float half[C::QB][R];       // and, where row sums are apart, before that
    long long orow[C::QB][R];   // output row of each query row, -1 past the last
    int rpos[C::QB][R];         // its position
    float rsink[C::QB][R];      // its sink (log2 units)
    alignas(16) float qf[C::QB][R];  // its scale log2(e) / the power of two in its Q
    PlanStart plan;
    UnitRing<R, UNITS> units;
    uint64_t k_full[C::STAGES], k_empty[C::STAGES], v_full[C::STAGES], v_empty[C::STAGES];
    uint64_t sc_full[SRING], sc_empty[SRING];
    uint64_t q_full[C::QB], q_empty[C::QB];
    uint64_t s_full[C::SBUF], s_empty[C::SBUF], p_full[2], pv_done[2], o_empty[2], both, drain[2];
    uint32_t tmem_base;
    int abort, last[3];  // last: of a group alone, of both
};

// ---------------------------------------------------------------- PTX used here alone

__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
}
__device__ __forceinline__ void tmem_ld4(uint32_t a, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ float redux_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
// Barrier of `THREADS` threads that also ORs a predicate.
template <int THREADS> __device__ __forceinline__ bool sync_any(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "n"(THREADS)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---------------------------------------------------------------- roles

template <int D, int R>
__device__ void load_tiles(const DecodeParams &p, const CUtensorMap *tk, const CUtensorMap *tv,
                           Smem<D, R> &sm, const DevCtx &ctx) {
    using C = Cfg<D, R>;
    const int lane = threadIdx.x & 31;
    const int per_tile = TILE >> p.page_shift, chunk = 32 >> (7 - p.page_shift);  // tiles a chunk
    const uint32_t page_bytes = (uint32_t)p.page * D;
    int t = 0;
    bool ok = true;
    unsigned bad = 0;
    if (lane == 0) {
        prefetch_tmap(tk);
        prefetch_tmap(tv);
    }
    UnitIter<R> it(p.plan, sm.plan);
    int index = 0;
#pragma unroll 1
    for (; it.live && ok; it.next(p.plan, sm.plan)) {
        const Unit<R> &u = it.u;
        if (u.begin == u.end) continue;
        if (lane == 0) ok = sm.units.put(index, u, ctx, &sm.abort);
        ++index;
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        bool far = false;
        for (int c = u.begin; c < u.end && ok; c += chunk) {
            // a page a lane
            const int j = (u.t_first + c) * per_tile + lane;
            const int pid =
                c + lane / per_tile < u.end
                    ? page_of(p.page_table, p.max_pages, p.num_pages, p.page_shift, u, j)
                    : -1;
            bad |= pid == -2;
            const int row = pid < 0 ? p.rows_total : (pid * p.plan.Hkv + u.h) * p.page;
            float4 s = page_scales(p.k_scale, p.v_scale, pid, p.plan.Hkv, u.h);
            const int nt = min(chunk, u.end - c);
#pragma unroll 1
            for (int i = 0; i < nt; ++i, ++t) {
                const int st = t % C::STAGES, use = t / C::STAGES;
                // lane i * per_tile + k holds the page of the tile's slot k
                const int k = lane - i * per_tile;
                const bool here = k >= 0 && k < per_tile;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t full = smem_u32(kv ? &sm.v_full[st] : &sm.k_full[st]);
                    const uint32_t empty = smem_u32(kv ? &sm.v_empty[st] : &sm.k_empty[st]);
                    const uint32_t dst = smem_u32(kv ? sm.v[st] : sm.k[st]);
                    bool go = true;
                    if (lane == 0) {
                        if (use >= 1) go = bar_wait(empty, (use - 1) & 1, ctx, &sm.abort);
                        if (go) mbar_arrive_expect_tx(full, C::TILE_BYTES);
                    }
                    ok = __shfl_sync(0xffffffffu, go ? 1 : 0, 0) != 0;
                    if (!ok) break;
                    if (here)
                        tma_load_2d(dst + (uint32_t)k * page_bytes, kv ? tv : tk, full, 0, row);
                }
                if (!ok) break;
                const int ss = t % SRING;
                if (t >= SRING)
                    ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&sm.sc_empty[ss]),
                                                           (t / SRING - 1) & 1, ctx, &sm.abort));
                if (!ok) break;
                if (i == 0) {  // (behind the tile's copies: they are what takes long)
                    far = far || __any_sync(0xffffffffu, pid >= 0 && far_log2(s.y));
                    if (far) {
                        s.z = -1.f;
                        if (lane == 0) sm.units.u[(index - 1) % UNITS].far = 1;
                    }
                }
                if (here) sm.sc[ss][k] = s;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.sc_full[ss]));
            }
        }
    }
    if (lane == 0 && ok) {
        Unit<R> last{};
        sm.units.put(index, last, ctx, &sm.abort);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(ctx, DEVERR_INDEX);
    // copies in flight land before the CTA leaves (at once on the normal path)
    if (lane == 0) {
        int zero = 0;
#pragma unroll 1
        for (int i = 1; i <= C::STAGES && i <= t; ++i) {
            bar_wait(smem_u32(&sm.k_full[(t - i) % C::STAGES]), ((t - i) / C::STAGES) & 1, ctx,
                      &zero);
            bar_wait(smem_u32(&sm.v_full[(t - i) % C::STAGES]), ((t - i) / C::STAGES) & 1, ctx,
                      &zero);
        }
    }
}

// Q of a unit: each row scaled by a power of two, split into hi and 16 lo, K-major rows
// hi 0 .. R-1, lo R .. 2R-1. A lane holds 8 columns, CH lanes a row.
template <int D, int R>
__device__ void load_queries(const DecodeParams &p, Smem<D, R> &sm, const DevCtx &ctx) {
    using C = Cfg<D, R>;
    constexpr int CH = D / 8, PER = R * CH / 32;  // items a lane
    const int lane = threadIdx.x & 31;
    const int G = p.plan.G;
    bool ok = true;
    for (int n = 0;; ++n) {
        if (!__all_sync(0xffffffffu, sm.units.wait(n, ctx, &sm.abort))) break;
        const Unit<R> u = sm.units.u[n % UNITS];
        __syncwarp();
        if (lane == 0) sm.units.release(n);
        if (u.begin == u.end) break;
        const int w = n % C::QB;
        static_assert(R <= 32, "a row a lane");
        const int row0 = u.row0 + lane, tok0 = p.plan.token(row0), head0 = u.h * G + row0 - tok0 * G;
        const bool in = lane < R && lane < u.nrows;
        const float sink = in && p.sinks ? sink_log2(__ldg(p.sinks + head0)) : 0.f;
        constexpr int B = PER < 4 ? PER : 4;  // items in flight
#pragma unroll 1
        for (int i0 = 0; i0 < PER; i0 += B) {
            uint4 x[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int r = ((i0 + i) * 32 + lane) / CH, c = ((i0 + i) * 32 + lane) % CH;
                const int row = u.row0 + r, tok = p.plan.token(row);
                x[i] = make_uint4(0, 0, 0, 0);
                if (r < u.nrows)
                    x[i] = __ldg(reinterpret_cast<const uint4 *>(
                        p.q + (size_t)(u.s.t0 + tok) * p.q_stride +
                        (size_t)(u.h * G + row - tok * G) * D + 8 * c));
            }
            if (i0 == 0 && n >= C::QB)
                ok = bar_wait(smem_u32(&sm.q_empty[w]), (n / C::QB - 1) & 1, ctx, &sm.abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int r = ((i0 + i) * 32 + lane) / CH, c = ((i0 + i) * 32 + lane) % CH;
                const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t top = 0;  // the row's largest finite |q|, as bf16 bits
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t a = v[e] & 0x7fff7fffu;  // inf and NaN set no scale
                    top = __vmaxu2(top, a & __vcmpltu2(a, 0x7f807f80u));
                }
#pragma unroll
                for (int o = 1; o < CH; o <<= 1)
                    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = max(top >> 16, top & 0xffffu);
                // 2^k with the largest |q| 2^k in [128, 256), k within fp32's normal range
                const int k = top ? max(-120, min(7 - ((int)(top >> 7) - 127), 120)) : 0;
                const float up = __uint_as_float((uint32_t)(127 + k) << 23);
                uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // by way of f16, which holds a scaled bf16 down to 2^-24; inf and NaN
                    // become NaN and spoil their own row
                    const uint32_t ab = pack_f16x2(__uint_as_float(v[e] << 16) * up,
                                                   __uint_as_float(v[e] & 0xffff0000u) * up) |
                                        (__vcmpgeu2(v[e] & 0x7fff7fffu, 0x7f807f80u) & 0x7fff7fffu);
                    const uint32_t h = e4m3x2_of_f16x2(ab);
                    hi[e >> 1] |= h << (16 * (e & 1));
                    lo[e >> 1] |= e4m3x2_of_f16x2(times_difference<16>(ab, e4m3x2_to_f16x2(h)))
                                  << (16 * (e & 1));
                }
                // 8 bytes: half of the 16-byte unit c / 2
                *reinterpret_cast<uint2 *>(sm.q[w] + sw_offset<D>(r, c >> 1) + 8 * (c & 1)) =
                    make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(sm.q[w] + sw_offset<D>(R + r, c >> 1) + 8 * (c & 1)) =
                    make_uint2(lo[0], lo[1]);
                if (c == 0)
                    sm.qf[w][r] = p.scale_l2 * __uint_as_float((uint32_t)(127 - k) << 23);
            }
        }
        if (!ok) break;
        if (lane < R) {
            sm.orow[w][lane] = in ? (long long)(u.s.t0 + tok0) * p.H + head0 : -1;
            sm.rpos[w][lane] = u.s.len - u.s.n + tok0;
            sm.rsink[w][lane] = sink;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[w]));
    }
}

template <int D, int R>
__device__ void issue_s(Smem<D, R> &sm, uint32_t tmem, const DevCtx &ctx) {
    using C = Cfg<D, R>;
    constexpr uint32_t IDESC = idesc_e4m3_f32(128, C::N, 0, 0);
    volatile int *abort = &sm.abort;
    if (ctx.stall) bar_wait(smem_u32(&sm.drain[0]), 0, ctx, abort);  // test hook: runs out
    const uint64_t dk = desc_rows<D>(smem_u32(sm.k[0])), dq = desc_rows<D>(smem_u32(sm.q[0]));
    auto wait = [&](uint64_t &bar, int phase) {
        return bar_wait(smem_u32(&bar), phase & 1, ctx, abort);
    };
    int t = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
        if (!(ok = sm.units.wait(i, ctx, abort))) break;
        const int w = i % C::QB, n = sm.units.u[i % UNITS].end - sm.units.u[i % UNITS].begin;
        sm.units.release(i);
        if (n == 0) break;
        ok = wait(sm.q_full[w], i / C::QB);
        const uint64_t b = dq + (uint64_t)(w * (C::N * D >> 4));
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j, ++t) {
            const int st = t % C::STAGES, sb = t % C::SBUF;
            ok = wait(sm.k_full[st], t / C::STAGES) &&
                 (t < C::SBUF || wait(sm.s_empty[sb], t / C::SBUF - 1));
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = dk + (uint64_t)(st * (C::TILE_BYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
                mma_f8(tmem + (uint32_t)sb * C::N, a + (uint64_t)(kk * 2), b + (uint64_t)(kk * 2),
                       IDESC, kk > 0);
            tc_commit(smem_u32(&sm.s_full[sb]));
            tc_commit(smem_u32(&sm.k_empty[st]));
            if (j == n - 1) tc_commit(smem_u32(&sm.q_empty[w]));
        }
    }
    tc_commit(smem_u32(&sm.drain[0]));  // every MMA is done before TMEM goes
    int zero = 0;
    bar_wait(smem_u32(&sm.drain[0]), 0, ctx, &zero);
}

// The group that takes tile t, the j-th of unit i with n tiles.
__device__ __forceinline__ int group_of(int i, int n, int t) { return (n <= SOLO ? i : t) & 1; }

template <int D, int R>
__device__ void issue_pv(Smem<D, R> &sm, uint32_t tmem, const DevCtx &ctx) {
    using C = Cfg<D, R>;
    constexpr uint32_t IDESC = idesc_e4m3_f32(D, C::NO, 1, 1) | B_E5M2;
    volatile int *abort = &sm.abort;
    const uint64_t dv = desc_rows<D>(smem_u32(sm.v[0])), dp = desc_rows<C::PW>(smem_u32(sm.p[0]));
    auto wait = [&](uint64_t &bar, int phase) {
        return bar_wait(smem_u32(&bar), phase & 1, ctx, abort);
    };
    int t = 0, done0 = 0, done1 = 0, units0 = 0, units1 = 0;  // of group 0 and 1
    bool ok = true;
    for (int i = 0; ok; ++i) {
        if (!(ok = sm.units.wait(i, ctx, abort))) break;
        const int n = sm.units.u[i % UNITS].end - sm.units.u[i % UNITS].begin;
        sm.units.release(i);
        if (n == 0) break;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j, ++t) {
            const int st = t % C::STAGES, g = group_of(i, n, t);
            const bool first = n <= SOLO ? j == 0 : j < 2;  // of the group in this unit
            ok = wait(sm.v_full[st], t / C::STAGES);
            // the first P V overwrites the O that an earlier unit's end reads
            const int units = g ? units1 : units0, done = g ? done1 : done0;
            if (first && units >= 1) ok = ok && wait(sm.o_empty[g], units - 1);
            ok = ok && wait(sm.p_full[g], done);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = dv + (uint64_t)(st * (C::TILE_BYTES >> 4));
            const uint64_t b = dp + (uint64_t)(g * (C::PW * TILE >> 4));
            const uint32_t o = tmem + C::O_COL + (uint32_t)g * C::NO;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 keys: 32 rows of V and of P
                mma_f8(o, a + (uint64_t)(kk * (32 * D >> 4)), b + (uint64_t)(kk * (32 * C::PW >> 4)),
                       IDESC, kk > 0 || !first);
            tc_commit(smem_u32(&sm.pv_done[g]));
            tc_commit(smem_u32(&sm.v_empty[st]));
            if (g) ++done1, units1 += first;
            else ++done0, units0 += first;
        }
    }
    tc_commit(smem_u32(&sm.drain[1]));
    int zero = 0;
    bar_wait(smem_u32(&sm.drain[1]), 0, ctx, &zero);
}

// Sums of each l[r] over the warp, to out[0 .. R-1]. Lanes halve the rows they
// hold while they halve the lanes, so that R rows take about R shuffles instead of 5 R.
template <int R> __device__ __forceinline__ void column_sums(float (&l)[R], float *out, int lane) {
    int row = 0;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        const int o = 16 >> k, n = R >> (k + 1);  // rows left after this step
        if (n >= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int r = 0; r < n; ++r) {
                const float send = up ? l[r] : l[r + n], keep = up ? l[r + n] : l[r];
                l[r] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
            row += up ? n : 0;
        } else {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        }
    }
    // lanes that differ in the bits below R's share hold the same row
    out[row] = l[0];
}

// Joins the parts of a cut unit: w_c = z_c 2^(m_c - m), lse = m + log2 sum_c w_c (+ the
// null logit), o = sum_c w_c o_c / sum_c w_c, in the order of the pieces. A warp takes RG
// rows at a time, for as many loads in flight; lane c holds part c's sums, the
// columns are spread over the lanes.
template <int D, int R>
__device__ void join_parts(const DecodeParams &p, int c0, int parts, const long long *orow,
                           const float *rsink, int warp, int warps, int lane) {
    const float2 *sums = part_sums(p.ws);
    const float *prow = reinterpret_cast<const float *>(p.ws + plan_rows_offset(R));
    constexpr int E = D / 32, RG = R / 8;
    // part i of the unit: the last of piece c0, then the first of c0 + 1, c0 + 2, ...
    auto slot = [&](int i) { return (size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0); };
#pragma unroll 1
    for (int r0 = warp * RG; r0 < R; r0 += warps * RG) {
        if (orow[r0] < 0) break;  // (rows past the unit's last are the last ones)
        float m[RG], z[RG], acc[RG][E] = {}, first[RG];
#pragma unroll
        for (int g = 0; g < RG; ++g) m[g] = NOTHING;
#pragma unroll 1
        for (int i = lane; i < parts; i += 32)
#pragma unroll
            for (int g = 0; g < RG; ++g)
                m[g] = fmaxf(m[g], __ldcg(sums + slot(i) * R + r0 + g).x);
#pragma unroll
        for (int g = 0; g < RG; ++g) m[g] = warp_max(m[g]);
        auto weight = [&](int i, int g) {
            if (i >= parts) return 0.f;
            const float2 s = __ldcg(sums + slot(i) * R + r0 + g);
            return s.y * ex2(s.x - m[g]);
        };
#pragma unroll
        for (int g = 0; g < RG; ++g) first[g] = weight(lane, g);
#pragma unroll
        for (int g = 0; g < RG; ++g) z[g] = warp_sum(first[g]);
#pragma unroll 1
        for (int i0 = 32; i0 < parts; i0 += 32)
#pragma unroll
            for (int g = 0; g < RG; ++g) z[g] += warp_sum(weight(i0 + lane, g));
        float inv[RG], lse2[RG];
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            lse2[g] = z[g] == 0.f ? -INFINITY : m[g] + __log2f(z[g]);
            inv[g] = z[g] == 0.f ? 0.f : __fdividef(1.f, z[g]);
            if (p.sink_mode == 2) with_null_sink(rsink[r0 + g], lse2[g], inv[g]);
        }
        // (the weights over their sum: values near fp32's largest do not overflow)
#pragma unroll 1
        for (int i0 = 0; i0 < parts; i0 += 32) {
            float wt[RG];
#pragma unroll
            for (int g = 0; g < RG; ++g)
                wt[g] = (i0 == 0 ? first[g] : weight(i0 + lane, g)) * inv[g];
            const int cnt = min(32, parts - i0);
#pragma unroll (8 / RG)
            for (int i = 0; i < cnt; ++i) {
#pragma unroll
                for (int g = 0; g < RG; ++g) {
                    const float wi = __shfl_sync(0xffffffffu, wt[g], i);
                    const float *at = prow + (slot(i0 + i) * R + r0 + g) * D + lane * E;
                    if constexpr (E == 4) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(at));
                        acc[g][0] = fmaf(wi, v.x, acc[g][0]), acc[g][1] = fmaf(wi, v.y, acc[g][1]);
                        acc[g][2] = fmaf(wi, v.z, acc[g][2]), acc[g][3] = fmaf(wi, v.w, acc[g][3]);
                    } else {
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(at));
                        acc[g][0] = fmaf(wi, v.x, acc[g][0]), acc[g][1] = fmaf(wi, v.y, acc[g][1]);
                    }
                }
            }
        }
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            const long long row = orow[r0 + g];
            if (row < 0) continue;
            __nv_bfloat16 *dst = p.o + row * D + lane * E;
            if constexpr (E == 4)
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(pack_bf16x2(acc[g][0], acc[g][1]),
                               pack_bf16x2(acc[g][2], acc[g][3]));
            else
                *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[g][0], acc[g][1]);
            if (p.lse && lane == 0) p.lse[row] = lse2[g] * LN2;
        }
    }
}

// A tile's share of a unit's row sums from the logits alone, a row at a time, for a warp
// whose keys' S is at `at`. (Not inlined: see page_scales.)
template <int D, int R>
__device__ __noinline__ void sum_apart(Smem<D, R> &sm, uint32_t at, float k_scale, bool hidden,
                                       int kpos, int hi, int causal, int wl, int key0, int g, int w,
                                       int start) {
    const int lane = threadIdx.x & 31, quarter = threadIdx.x >> 5 & 3;
    float *fn = sm.fn[g][quarter], *fl = sm.fl[g][quarter];
    if (start) {  // the unit's number and 1
        if (quarter == 0 && lane < R) sm.fm[g][lane] = sm.mx[w][g][lane];
        if (lane < R) fn[lane] = NOTHING, fl[lane] = 0.f;
        if (quarter == 0 && lane == 0) sm.apart[g] = start;
        __syncwarp();
    }
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
        const float high = tmem_ld1(at + r), low = tmem_ld1(at + R + r);
        float y = fmaf(low, 0.0625f, high) * (k_scale * sm.qf[w][r]);
        if (key0 && kpos == 0) y += sm.rsink[w][r];
        const int pos = sm.rpos[w][r];
        if (hidden || kpos > (causal ? pos : hi) || (wl >= 0 && kpos < pos - wl)) y = -INFINITY;
        const float n = fn[r], nn = fmaxf(n, redux_max(y));
        const float sum = warp_sum(ex2(y - nn + BASE));
        __syncwarp();
        if (lane == 0) {
            fl[r] = fmaf(fl[r], ex2(n - nn), sum);
            fn[r] = nn;
        }
    }
    __syncwarp();
}

// Notes NaN codes of a value that is cleared for its scale of 0: NaN times 0 is NaN.
template <int D, int R> __device__ __noinline__ void note_nan(const uint4 *v, bool zero,
                                                                    Unit<R> &u) {
    bool nan = false;
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
        uint4 y = v[c];
        nan = without_nan(y) || nan;
    }
    if (nan && zero) u.nan_values = u.nan_zero = 1;
}

// A row's denominator z and what it is in terms of, with such sums beside its groups'.
template <int D, int R>
__device__ __noinline__ float2 join_apart(const Smem<D, R> &sm, int w, int row, int groups,
                                          int stamp) {
    float nn = NOTHING, z = 0.f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass)
#pragma unroll 1
        for (int s = 0; s < 8; ++s) {
            const int g = s >> 2, q = s & 3;
            if (!(groups >> g & 1)) continue;
            const bool apart = sm.apart[g] == stamp;
            const float n = apart ? sm.fm[g][row] : sm.mx[w][g][row];
            const float fn = apart ? sm.fn[g][q][row] : NOTHING;
            if (pass == 0) {
                nn = fmaxf(nn, fmaxf(n, fn));
            } else {
                z = fmaf(ex2(n - nn), sm.lx[w][g][q][row], z);
                if (apart) z = fmaf(ex2(fn - nn), sm.fl[g][q][row], z);
            }
        }
    return make_float2(nn, z);
}

// Rows r0 .. r1 - 1 of the groups' O^T times half.
template <int D, int R>
__device__ __noinline__ void scale_rows(const Smem<D, R> &sm, uint32_t o_tmem, int w, int r0,
                                        int r1, int groups) {
#pragma unroll 1
    for (int r = r0; r < r1; ++r)
#pragma unroll 1
        for (int k = 0; k < 2 * Cfg<D, R>::TERMS; ++k) {  // (the groups' columns lie side by side)
            const uint32_t at = o_tmem + (uint32_t)(k * R + r);
            if (groups >> k / Cfg<D, R>::TERMS & 1) tmem_st1(at, tmem_ld1(at) * sm.half[w][r]);
        }
}

template <int D, int R>
__device__ void softmax(const DecodeParams &p, Smem<D, R> &sm, uint32_t tmem, const DevCtx &ctx) {
    using C = Cfg<D, R>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = (warp - 4) >> 2, quarter = warp & 3;
    const int key = quarter * 32 + lane;  // key of the tile = TMEM lane
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + C::O_COL + lanes;
    volatile int *abort = &sm.abort;
    const int bar_g = 1 + g;
    // Once a wait has given up (ok), the warp goes through the rest of its unit
    // without waiting and without writing to global memory: every warp of the group
    // reaches every named barrier, so none is left waiting there. Between the groups
    // there are bounded waits alone.
    bool ok = true;
    auto wait = [&](uint64_t &bar, int phase) {
        ok = ok && bar_wait(smem_u32(&bar), phase & 1, ctx, abort);
        ok = __all_sync(0xffffffffu, ok);
    };
    int t0 = 0, done = 0, meets = 0;  // tiles before the unit; the group's; meetings of both
    for (int i = 0;; ++i) {
        const int w = i % C::QB;
        ok = ok && sm.units.wait(i, ctx, abort);
        if (sync_any<128>(bar_g, !ok)) break;  // the group's four warps go on, or none
        const Unit<R> &u = sm.units.u[i % UNITS];
        const int n = u.end - u.begin;
        if (n == 0) break;
        const bool solo = n <= SOLO;
        if (solo && (i & 1) != g) {
            t0 += n;
            __syncwarp();
            if (lane == 0) sm.units.release(i);
            continue;
        }
        wait(sm.q_full[w], i / C::QB);
        if (key < R) sm.mx[w][g][key] = NOTHING;
        named_sync(bar_g, 128);
        // the group's threads meet, or both groups'
        auto meet = [&]() {
            if (solo) {
                named_sync(bar_g, 128);
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.both));
                wait(sm.both, meets++);
            }
        };
        const float4 *qf4 = reinterpret_cast<const float4 *>(sm.qf[w]);
        // m is the group's and lies in shared memory: 32 rows of it would not fit
        // beside the scores and sums in registers
        const float4 *m4 = reinterpret_cast<const float4 *>(sm.mx[w][g]);
        float l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = 0.f;
        bool apart = false;  // the row sums have a maximum of their own
        const int step = solo ? 1 : 2, j0 = solo ? 0 : (g ^ t0) & 1;
#pragma unroll 1
        for (int j = j0; j < n; j += step, ++done) {
            const int t = t0 + j, sb = t % C::SBUF, ss = t % SRING;
            const int kpos = (u.t_first + u.begin + j) * TILE + key;
            const int base = kpos - key;
            wait(sm.sc_full[ss], t / SRING);
            const float4 sc = sm.sc[ss][key >> p.page_shift];
            wait(sm.s_full[sb], t / C::SBUF);
            tc_fence_after();
            if (__builtin_expect(sc.z < 0.f, 0)) {
                sum_apart<D, R>(sm, tmem + (uint32_t)sb * C::N + lanes, sc.x, sc.y == -INFINITY,
                                kpos, u.hi, p.plan.causal, p.plan.wl, p.sink_mode == 1, g, w,
                                apart ? 0 : i + 1);
                apart = true;
            }
            float x[R];  // e of this key for every row
            {
                constexpr int CH = R < 16 ? R : 16;
#pragma unroll
                for (int c = 0; c < R; c += CH) {
                    uint32_t hi[CH], lo[CH];
                    if constexpr (CH == 8) {
                        tmem_ld8(tmem + (uint32_t)sb * C::N + lanes + c, hi);
                        tmem_ld8(tmem + (uint32_t)sb * C::N + lanes + R + c, lo);
                    } else {
                        tmem_ld16(tmem + (uint32_t)sb * C::N + lanes + c, hi);
                        tmem_ld16(tmem + (uint32_t)sb * C::N + lanes + R + c, lo);
                    }
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < CH; ++e) {
                        const float4 f = qf4[(c + e) / 4];
                        x[c + e] = fmaf(fmaf(__uint_as_float(lo[e]), 0.0625f,
                                             __uint_as_float(hi[e])),
                                        sc.x * (e % 4 == 0 ? f.x : e % 4 == 1 ? f.y
                                                : e % 4 == 2 ? f.z : f.w),
                                        sc.y);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm.s_empty[sb]));
                mbar_arrive(smem_u32(&sm.sc_empty[ss]));
            }
            if (p.sink_mode == 1 && kpos == 0) {
#pragma unroll
                for (int r = 0; r < R; ++r) x[r] += sm.rsink[w][r];
            }
            if (base < u.ilo || base + TILE - 1 > u.ihi) {  // some row does not see some key
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int pos = sm.rpos[w][r];
                    const bool in = kpos <= (p.plan.causal ? pos : u.hi) &&
                                    (p.plan.wl < 0 || kpos >= pos - p.plan.wl);
                    uint32_t b = __float_as_uint(x[r]);
                    hide_unless(b, in);
                    x[r] = __uint_as_float(b);
                }
            }
            // values that no row sees may hold anything, NaN codes too, and the MMA
            // multiplies them by 0: they are cleared, and so are those of a zero scale
            const bool some = kpos < u.ilo || kpos > u.ihi;  // not every row sees the key
            if (__any_sync(0xffffffffu, some || sc.w == 0.f)) {
                const bool clear = kpos < u.lo || kpos > u.hi || sc.w == 0.f;
                const int st = t % C::STAGES;
                wait(sm.v_full[st], t / C::STAGES);
                const bool zero = sc.w == 0.f && kpos >= u.lo && kpos <= u.hi;
                if (__builtin_expect(__any_sync(0xffffffffu, zero), 0))
                    note_nan<D>(reinterpret_cast<const uint4 *>(sm.v[st] + key * D), zero,
                                sm.units.u[i % UNITS]);
                if (some || clear) {
                    uint4 *v = reinterpret_cast<uint4 *>(sm.v[st] + key * D);
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint4 y = v[c];
                        if (clear) {
                            v[c] = make_uint4(0, 0, 0, 0);
                        } else if (without_nan(y)) {
                            v[c] = y;
                            sm.units.u[i % UNITS].nan_values = 1;
                        }
                    }
                }
            }
            const float sum_scale = apart ? 0.f : sc.z;
            float top = -INFINITY;
#pragma unroll
            for (int r = 0; r < R; r += 4) {
                const float4 m = m4[r / 4];
                top = max3(max3(top, x[r] - m.x, x[r + 1] - m.y), x[r + 2] - m.z, x[r + 3] - m.w);
            }
            const bool move = sync_any<128>(bar_g, top > LIMIT - BASE);
            if (move) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float c = redux_max(x[r]);
                    if (lane == 0) sm.wmax[g][quarter][r] = c;
                }
                named_sync(bar_g, 128);
                if (key < R) {
                    const float c = fmaxf(fmaxf(sm.wmax[g][0][key], sm.wmax[g][1][key]),
                                          fmaxf(sm.wmax[g][2][key], sm.wmax[g][3][key]));
                    const float m = sm.mx[w][g][key], mn = fmaxf(m, c);
                    sm.alpha[g][key] = ex2(m - mn);
                    sm.mx[w][g][key] = mn;
                }
                named_sync(bar_g, 128);
                if (!apart) {
#pragma unroll
                    for (int r = 0; r < R; ++r) l[r] *= sm.alpha[g][r];
                }
                if (j > j0) {
                    wait(sm.pv_done[g], done - 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < C::NO; c += 8) {
                        uint32_t v[8];
                        tmem_ld8(o_tmem + (uint32_t)(g * C::NO + c), v);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = __float_as_uint(__uint_as_float(v[e]) * sm.alpha[g][(c + e) % R]);
                        tmem_st8(o_tmem + (uint32_t)(g * C::NO + c), v);
                    }
                    tc_wait_st();
                }
            }
            // P overwrites the group's last one, which its P V has read by now as a rule
            if (done >= 1) wait(sm.pv_done[g], done - 1);
            // the key's row of P: R codes of each term, 16 bytes a store
#pragma unroll
            for (int c = 0; c < R; c += 16) {
                constexpr int CH = R < 16 ? R : 16;
                uint32_t t[C::TERMS][4];
#pragma unroll
                for (int e = 0; e < CH; e += 4) {
                    const float4 m = m4[(c + e) / 4];
                    const float mm[4] = {m.x, m.y, m.z, m.w};
                    uint32_t y[2][C::TERMS];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = c + e + 2 * h;
                        const float a = ex2(x[r] - mm[2 * h] + BASE);
                        const float b = ex2(x[r + 1] - mm[2 * h + 1] + BASE);
                        l[r] = fmaf(a, sum_scale, l[r]);
                        l[r + 1] = fmaf(b, sum_scale, l[r + 1]);
                        e5m2_terms(pack_f16x2(a, b), y[h]);
                    }
#pragma unroll
                    for (int k = 0; k < C::TERMS; ++k)  // the upper bytes
                        t[k][e >> 2] = __byte_perm(y[0][k], y[1][k], 0x7531);
                }
                if constexpr (R == 8) {
                    *reinterpret_cast<uint4 *>(sm.p[g] + sw_offset<C::PW>(key, 0)) =
                        make_uint4(t[0][0], t[0][1], t[1][0], t[1][1]);
                    *reinterpret_cast<uint4 *>(sm.p[g] + sw_offset<C::PW>(key, 1)) =
                        make_uint4(t[2][0], t[2][1], t[3][0], t[3][1]);
                } else {
#pragma unroll
                    for (int k = 0; k < C::TERMS; ++k)
                        *reinterpret_cast<uint4 *>(
                            sm.p[g] + sw_offset<C::PW>(key, (k * R + c) / 16)) =
                            make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[g]));
        }
        // ---- the unit's end: the groups' maxima, row sums and O^T, joined
        column_sums<R>(l, sm.lx[w][g][quarter], lane);
        wait(sm.pv_done[g], done - 1);
        tc_fence_before();
        meet();
        tc_fence_after();
        const bool has[2] = {!solo || g == 0, !solo || g == 1};
        const bool scaled = u.far;
        const bool part = u.begin > 0 || u.end < u.ntiles;
        const size_t slot = (size_t)blockIdx.x * 2 + (u.begin > 0 ? 0 : 1);
        // a thread a row: what each group's O^T is multiplied by, and the denominator
        const int me = solo ? key : threadIdx.x - 128;
        if (me < R) {
            const float m0 = has[0] ? sm.mx[w][0][me] : NOTHING;
            const float m1 = has[1] ? sm.mx[w][1][me] : NOTHING, mm = fmaxf(m0, m1);
            const float w0 = has[0] ? ex2(m0 - mm) : 0.f, w1 = has[1] ? ex2(m1 - mm) : 0.f;
            float z = 0.f, nn = mm, half = 1.f;
            if (__builtin_expect(scaled, 0)) {
                const float2 nz = join_apart<D, R>(
                    sm, w, me, (has[0] ? 1 : 0) | (has[1] ? 2 : 0), i + 1);
                nn = nz.x, z = nz.y;
                // 2^(m - n) is a value scale's size: in two steps, as it may leave fp32's range
                sm.half[w][me] = half = ex2(0.5f * (mm - nn));
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (has[0]) z = fmaf(w0, sm.lx[w][0][q][me], z);
                    if (has[1]) z = fmaf(w1, sm.lx[w][1][q][me], z);
                }
            }
            float inv = z == 0.f ? 0.f : __fdividef(1.f, z);
            if (part) {
                if (ok)
                    part_sums(p.ws)[slot * R + me] = make_float2(nn, z * (1.f / (1 << (int)BASE)));
            } else {
                float lse2 = z == 0.f ? -INFINITY : nn - BASE + __log2f(z);
                if (p.sink_mode == 2) with_null_sink(sm.rsink[w][me], lse2, inv);
                const long long row = sm.orow[w][me];
                if (ok && p.lse && row >= 0) p.lse[row] = lse2 * LN2;
            }
            sm.wt[w][0][me] = w0 * inv * half;
            sm.wt[w][1][me] = w1 * inv * half;
        }
        meet();
        const bool writes = (D == 128 || lane < 16) && ok;  // 64 rows of O^T: 16 lanes of every 32
        const int col = D == 128 ? key : quarter * 16 + lane;
        float *prow = reinterpret_cast<float *>(p.ws + plan_rows_offset(R)) + slot * R * D + col;
        const int rows0 = solo ? 0 : g * (R / 2), rows1 = solo ? R : rows0 + R / 2;
        constexpr int STEP = R / 2 < 8 ? R / 2 : 8;  // rows at a time
        if (__builtin_expect(scaled, 0))
            scale_rows<D, R>(sm, o_tmem, w, rows0, rows1, (has[0] ? 1 : 0) | (has[1] ? 2 : 0));
        uint32_t nan_rows = 0;  // rows whose column is NaN
        if (u.nan_values && writes)
            each_partial_key<D>(p, u, u.lo, u.hi, [&](int k, const uint8_t *codes) {
                if ((__ldg(codes + col) & 0x7f) != 0x7f) return;
#pragma unroll 1
                for (int r = 0; r < R; ++r) {
                    const int pos = sm.rpos[w][r];
                    if (k <= (p.plan.causal ? pos : u.hi) && (p.plan.wl < 0 || k >= pos - p.plan.wl))
                        nan_rows |= 1u << r;
                }
            });
#pragma unroll 1
        for (int r0 = rows0; r0 < rows1; r0 += STEP) {
            constexpr int M = C::TERMS;
            uint32_t v[2 * M][STEP];  // the terms of group 0, of group 1
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (!has[s]) continue;
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    const uint32_t at = o_tmem + (uint32_t)(s * C::NO + k * R + r0);
                    if constexpr (STEP == 8) tmem_ld8(at, v[M * s + k]);
                    else tmem_ld4(at, v[M * s + k]);
                }
            }
            tc_wait_ld();
            float acc[STEP];
#pragma unroll
            for (int e = 0; e < STEP; ++e) {
                acc[e] = 0.f;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!has[s]) continue;
                    float o = __uint_as_float(v[M * s + M - 1][e]);
#pragma unroll
                    for (int k = M - 2; k >= 0; --k)
                        o = fmaf(o, 0.125f, __uint_as_float(v[M * s + k][e]));
                    acc[e] = fmaf(sm.wt[w][s][r0 + e], o, acc[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < STEP; ++e) {
                const int r = r0 + e;
                if (!writes) continue;
                if (nan_rows >> r & 1) acc[e] = NAN;
                if (part) {
                    prow[(size_t)r * D] = acc[e];
                } else if (sm.orow[w][r] >= 0) {
                    p.o[sm.orow[w][r] * D + col] = __float2bfloat16_rn(acc[e]);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        // both groups have read both O^T, or the one group its own: eight arrivals each
        if (lane == 0) {
            for (int s = 0; s < 2; ++s)
                if (has[s]) mbar_arrive_n(smem_u32(&sm.o_empty[s]), solo ? 2 : 1);
        }
        if (part) {  // the last of the unit's pieces to get here joins them
            __threadfence();
            meet();
            if (me == 0) {
                asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zero
                sm.last[solo ? g : 2] = atomicAdd(join_counters(p.ws) + u.c0, 1u) ==
                                            (unsigned)u.parts - 1 && !*abort;
            }
            meet();
            // (a group alone, or group 0 for both, has asked)
            if (ok && sm.last[solo ? g : 2]) {
                __threadfence();
                join_parts<D, R>(p, u.c0, u.parts, sm.orow[w], sm.rsink[w],
                                 solo ? warp & 3 : warp - 4, solo ? 4 : 8, lane);
            }
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive_n(smem_u32(&sm.q_empty[w]), solo ? 2 : 1);
            sm.units.release(i);
        }
        t0 += n;
    }
}

template <int D, int R>
__global__ void __launch_bounds__(NTHREADS, 1)
decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
              const DecodeParams p, const DevCtx ctx) {
    using C = Cfg<D, R>;
    extern __shared__ __align__(1024) uint8_t dsmem[];
    Smem<D, R> &sm = *reinterpret_cast<Smem<D, R> *>(dsmem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(dsmem) & 1023u) {  // the swizzle is anchored to 1024-byte boundaries
        if (threadIdx.x == 0) record_error(ctx, DEVERR_LAYOUT);
        return;
    }
    if (warp == 2) {  // a lane a barrier: one thread would take longer than the plan
        static_assert(C::STAGES <= 32 && SRING <= 32 && UNITS <= 32, "a lane a barrier");
        if (lane < C::STAGES) {
            mbar_init(smem_u32(&sm.k_full[lane]), 1);
            mbar_init(smem_u32(&sm.k_empty[lane]), 1);
            mbar_init(smem_u32(&sm.v_full[lane]), 1);
            mbar_init(smem_u32(&sm.v_empty[lane]), 1);
        }
        if (lane < SRING) {
            mbar_init(smem_u32(&sm.sc_full[lane]), 1);
            mbar_init(smem_u32(&sm.sc_empty[lane]), 4);
        }
        if (lane < C::QB) {
            mbar_init(smem_u32(&sm.q_full[lane]), 1);
            mbar_init(smem_u32(&sm.q_empty[lane]), 1 + 8);  // the MMAs and the softmax warps
        }
        if (lane < 2) {
            mbar_init(smem_u32(&sm.p_full[lane]), 4);
            mbar_init(smem_u32(&sm.pv_done[lane]), 1);
            mbar_init(smem_u32(&sm.o_empty[lane]), 8);
            mbar_init(smem_u32(&sm.drain[lane]), 1);
        }
        if (lane < C::SBUF) {
            mbar_init(smem_u32(&sm.s_full[lane]), 1);
            mbar_init(smem_u32(&sm.s_empty[lane]), 4);
        }
        if (lane == 0) {
            mbar_init(smem_u32(&sm.both), 8);
            sm.abort = 0;
            sm.apart[0] = sm.apart[1] = 0;
        }
        sm.units.init(2 + 1 + 8, lane);  // MMA issuers, queries, softmax
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sm.tmem_base), C::COLS);
        tmem_relinquish();
    }
    plan_start<R>(p.plan, sm.plan, ctx);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    if (warp == 0) {
        load_tiles<D, R>(p, &tk, &tv, sm, ctx);
    } else if (warp < 3) {
        if (lane == 0) {
            if (warp == 1) issue_s<D, R>(sm, tmem, ctx);
            else issue_pv<D, R>(sm, tmem, ctx);
        }
        __syncwarp();
    } else if (warp == 3) {
        load_queries<D, R>(p, sm, ctx);
    } else {
        softmax<D, R>(p, sm, tmem, ctx);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        // (no CTA ends before the counters are zero: they are the next call's then)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (sm.abort == TIMED_OUT) record_error(ctx, DEVERR_TIMEOUT);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

// Zeroes a call's join counters, which lie in its workspace so that no call meets another
// one's: the decode kernel, its programmatic dependent, starts beside it and waits for it
// before a piece arrives. (One request of 1000 positions: 11.4 us; with a memset in front
// 14.5, with counters built into the library, which calls had to share, 10.7.)
__global__ void __launch_bounds__(MAX_PIECES) zero_counters(uint8_t *ws) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    join_counters(ws)[threadIdx.x] = 0;
}

template <int D, int R>
cudaError_t launch(const PagedArgs &a, const DevInfo &dev, cudaStream_t s) {
    const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap tk, tv;
    if (!map_cache(&tk, a.k_cache, a, sw) || !map_cache(&tv, a.v_cache, a, sw))
        return cudaErrorInvalidValue;
    const size_t smem = sizeof(Smem<D, R>);
    static_assert(sizeof(Smem<D, R>) <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = ensure_smem_attr((const void *)decode_kernel<D, R>, smem, dev);
    if (e != cudaSuccess) return e;
    const int grid = dev.sm_count < MAX_PIECES ? dev.sm_count : MAX_PIECES;
    const bool split = a.workspace && a.workspace_bytes >= plan_workspace(R, D);
    DecodeParams p{plan_args(a, split, Cfg<D, R>::EXTRA), static_cast<const __nv_bfloat16 *>(a.q), a.q_stride,
                   a.v_cache, a.k_scale, a.v_scale, a.page_table, a.H, a.num_pages, a.page, page_shift(a.page),
                   a.max_pages, a.num_pages * a.Hkv * a.page, a.scale * LOG2E, a.sinks, a.sink_mode,
                   static_cast<__nv_bfloat16 *>(a.o), a.lse, static_cast<uint8_t *>(a.workspace)};
    if (verbose())
        fprintf(stderr, "sattn: paged decode_kernel<%d, %d> grid=%d smem=%zu split=%d\n", D, R, grid,
                smem, (int)split);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    if (split) {
        zero_counters<<<1, MAX_PIECES, 0, s>>>(p.ws);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, decode_kernel<D, R>, tk, tv, p, make_ctx(dev));
}

}  // namespace

// Rows a unit for that many tokens a sequence: enough for a whole KV group's
// where 32 are, so that its keys are read once.
static int decode_rows(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

size_t paged_decode_workspace(int max_q_len, int G, int d) {
    return plan_workspace(decode_rows((long long)max_q_len * G), d);
}

cudaError_t launch_paged_decode(const PagedArgs &a, const DevInfo &dev, cudaStream_t s) {
    const int r = decode_rows((long long)a.max_q_len * (a.H / a.Hkv));
    if (a.d == 64) {
        if (r == 8) return launch<64, 8>(a, dev, s);
        return r == 16 ? launch<64, 16>(a, dev, s) : launch<64, 32>(a, dev, s);
    }
    if (r == 8) return launch<128, 8>(a, dev, s);
    return r == 16 ? launch<128, 16>(a, dev, s) : launch<128, 32>(a, dev, s);
}

}  // namespace sattn
