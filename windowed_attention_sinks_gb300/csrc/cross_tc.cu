// Cross attention to encoder states on the tensor cores (tcgen05), bf16.
//
// Query rows are tokens times the heads of a KV group, token-major, fetched as boxes of G heads and
// floor(128 / G) tokens, so that any group size fills the 128 rows of an MMA. The states
// come as tiles of 128 keys, K and V in turn through one ring of shared memory.
//   S = Q K^T   [128 x 128] into TMEM
//   P = 2^(S scale log2(e) - m), bf16, 64 keys at a time over the columns of S that
//       have been read; l += its sum, unrounded
//   O += P V    P from TMEM, 64 keys at a time: while the second half of P is computed the
//       product with the first runs
// m is the maximum of a row's first 64 keys and stays unless 64 keys' P sum up to more than
// 2^15: P is computed on trust in one pass over S that looks for no maximum, and where the
// sum says that this was wrong m moves, O is rescaled and the pass is repeated.
// V rows behind the sequence's last state are zeroed in shared memory (the MMA multiplies them
// by P = 0, and they may be NaN).
//
// One persistent CTA per SM over an equal piece of the line of units (states_plan.cuh), two
// halves that work in turn, so that one's softmax runs beside the other's products:
//   many rows   a unit is 256 rows; both halves use every tile
//   FEW         a unit is 64 rows at most; the halves take every other tile and are
//               joined through shared memory at the unit's end. Twice as many tiles are in
//               work at a time: what bounds is the memory, and a tile's chain of products
//               and exponentials is longer than its load.
// Roles: warp 0 units and TMA; 1, 3 S of the halves; 4, 5 P V; 2 the last V tile's rows;
// 8-11, 12-15 softmax and epilogue, a thread a row.
#include <math.h>
#include <stdio.h>

#include "paged_plan.cuh"
#include "states_plan.cuh"

namespace sattn {
namespace {

constexpr int NTHREADS = 512;
constexpr int SOFTMAX = 8;   // first softmax warp
constexpr int UNITS = 4;     // units handed on ahead
constexpr int CHUNK = 64;    // keys whose P is handed on at a time
constexpr int FEW_ROWS = 64;
constexpr float SUM_LIMIT = 32768.f;  // m moves when 64 keys' P sum up to more
constexpr float FAR = 1 << 20;  // m up to which x - m may be taken in one rounding
constexpr uint32_t TMEM_COLS = 512, HALF_COLS = 256, O_COL = 128;

struct CrossParams {
    LineArgs line;
    int H, G, tokens;  // tokens: of a half's rows
    int rows;          // tokens * G
    int warps;         // softmax warps of a half that have rows
    float scale_l2;
    const float *sinks;
    int sink_mode;
    __nv_bfloat16 *o;
    float *lse;
    uint8_t *ws;
    uint32_t g_mul, g_shift;

    // row / G for 0 <= row < 2^31 (as PlanArgs::token)
    __device__ __forceinline__ int token(int row) const {
        return (int)((__umulhi(g_mul, (uint32_t)row) + (uint32_t)row) >> g_shift);
    }
};

template <int D> struct alignas(1024) Smem {
    static constexpr int NH = D / 64;                     // 64-column parts of a row
    static constexpr uint32_t PART = 128 * 128;           // 128 rows of 64 bf16
    static constexpr uint32_t TILE_BYTES = NH * PART;
    static constexpr int R = D == 128 ? 5 : 12;           // ring of K and V tiles
    uint8_t q[2][TILE_BYTES];  // (FEW: q[1] takes half 1's O at a unit's end)
    uint8_t kv[R][TILE_BYTES];
    LineStart line;
    LineRing<UNITS> units;
    float2 ml[FEW_ROWS];  // FEW: half 1's m and l
    uint64_t full[R], empty[R], raw[R];
    uint64_t q_full, q_empty, mg_full, mg_empty;
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], o_empty[2], drain[4];
    uint32_t tmem_base;
    int issued;  // loads into the ring so far
    int abort;
};

// The last tile of a sequence: its keys, if they do not fill it (0 for a sequence without
// states), and whether the unit's piece has it.
__device__ __forceinline__ bool ragged(const LineUnit &u) {
    return u.end == u.steps && u.steps * STATE_KEYS != u.s.len;
}
// 64-key chunks of step j that have keys (one for an empty sequence).
__device__ __forceinline__ int chunks(const LineUnit &u, int j) {
    return j * STATE_KEYS + CHUNK < u.s.len ? 2 : 1;
}

template <int D, bool FEW>
__device__ void load_tiles(const CrossParams &p, const CUtensorMap *tq,
                                           const CUtensorMap *tk, const CUtensorMap *tv,
                                           Smem<D> &sm, const DevCtx &ctx) {
    using S = Smem<D>;
    if ((threadIdx.x & 31) != 0) return;
    volatile int *abort = &sm.abort;
    prefetch_tmap(tq);
    prefetch_tmap(tk);
    prefetch_tmap(tv);
    LineIter<false> it(p.line, sm.line);
    if (p.line.split) {
        PlanNote n{};
        if (it.live) {
            const LineUnit &u = it.u;
            n.cont = u.begin > 0;
            n.through = u.begin > 0 && u.end < u.steps;
            n.t0 = u.s.t0;
            n.h = u.h;
            n.row0 = u.u * p.line.tokens * p.G;
            n.nrows = min(p.line.tokens, u.s.n - u.u * p.line.tokens) * p.G;
        }
        reinterpret_cast<PlanNote *>(p.ws)[blockIdx.x] = n;
    }
    int t = 0, index = 0, queries = 0;  // loads into the ring; units; loads of Q
    uint32_t raws = 0, on_raw = 0;      // bit i: raw[i]'s phase; slot i's last load counts there
    bool ok = true;
#pragma unroll 1
    for (; it.live && ok; it.next(p.line, sm.line)) {
        const LineUnit &u = it.u;
        if (u.begin == u.end) continue;
        ok = sm.units.put(index, u, ctx, abort);
        const bool tail = ragged(u);
#pragma unroll 1
        for (int j = u.begin; j < u.end && ok; ++j) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++t) {
                const int st = t % S::R, use = t / S::R;
                if (use >= 1) ok = ok && bar_wait(smem_u32(&sm.empty[st]), (use - 1) & 1, ctx, abort);
                if (!ok) break;
                uint32_t bar = smem_u32(&sm.full[st]);
                on_raw &= ~(1u << st);
                if (kv && tail && j == u.end - 1) {
                    bar = smem_u32(&sm.raw[st]);
                    raws ^= 1u << st;
                    on_raw |= 1u << st;
                }
                mbar_arrive_expect_tx(bar, S::TILE_BYTES);
#pragma unroll
                for (int c = 0; c < S::NH; ++c)
                    tma_load_3d(smem_u32(sm.kv[st]) + c * S::PART, kv ? tv : tk, bar, 64 * c, u.h,
                                u.s.s0 + j * STATE_KEYS);
                count_set(smem_u32(&sm.issued), t + 1);
            }
            if (j == u.begin && ok) {  // behind the first tile, which need not wait for it
                if (index >= 1) ok = bar_wait(smem_u32(&sm.q_empty), (index - 1) & 1, ctx, abort);
                if (!ok) break;
                const uint32_t bar = smem_u32(&sm.q_full);
                const int tok = u.s.t0 + u.u * p.line.tokens;
                const bool two = !FEW && u.s.n - u.u * p.line.tokens > p.tokens;
                mbar_arrive_expect_tx(bar, (two ? 2 : 1) * S::NH * p.rows * 128);
#pragma unroll
                for (int half = 0; half < (FEW ? 1 : 2); ++half)
                    if (half == 0 || two)
#pragma unroll
                        for (int c = 0; c < S::NH; ++c)
                            tma_load_3d(smem_u32(sm.q[half]) + c * S::PART, tq, bar, 64 * c,
                                        u.h * p.G, tok + half * p.tokens);
                ++queries;
            }
        }
        ++index;
    }
    if (ok) {
        LineUnit last{};
        sm.units.put(index, last, ctx, abort);
    }
    // copies in flight land before the CTA leaves
    int zero = 0;
#pragma unroll 1
    for (int st = 0; st < S::R; ++st) {
        bar_wait(smem_u32(&sm.raw[st]), (raws >> st & 1) ^ 1, ctx, &zero);
        const int use = (t - 1 - st) / S::R;  // the slot's last load
        if (st < t && !(on_raw >> st & 1))
            bar_wait(smem_u32(&sm.full[st]), use & 1, ctx, &zero);
    }
    if (queries > 0) bar_wait(smem_u32(&sm.q_full), (queries - 1) & 1, ctx, &zero);
}

// Zeroes the rows of a sequence's last V tile behind its last state. A warp.
template <int D> __device__ void clear_tails(Smem<D> &sm, const DevCtx &ctx) {
    using S = Smem<D>;
    const int lane = threadIdx.x & 31;
    volatile int *abort = &sm.abort;
    int t = 0;
    uint32_t raws = 0;
    for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, sm.units.wait(i, ctx, abort))) return;
        const LineUnit &u = sm.units.u[i % UNITS];
        const int n = u.end - u.begin;
        if (n == 0) return;
        t += 2 * n;
        if (ragged(u)) {
            const int st = (t - 1) % S::R;
            const int r0 = u.s.len - (u.steps - 1) * STATE_KEYS;
            const int r1 = chunks(u, u.steps - 1) * CHUNK;
            if (!__all_sync(0xffffffffu,
                            bar_wait(smem_u32(&sm.raw[st]), raws >> st & 1, ctx, abort)))
                return;
            raws ^= 1u << st;
            for (int c = 0; c < S::NH; ++c)
                for (int e = r0 * 8 + lane; e < r1 * 8; e += 32)
                    *reinterpret_cast<uint4 *>(sm.kv[st] + c * S::PART + e * 16) =
                        make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.full[st]));
        }
        __syncwarp();
        if (lane == 0) sm.units.release(i);
    }
}

// Load number t into the ring has landed. A role that does not look at every load cannot tell
// by a parity whether a slot holds its load or the one before the last, so it first waits until
// its load has been issued: by then the slot's load before has landed and been used.
template <int D>
__device__ __forceinline__ bool landed(Smem<D> &sm, int t, const DevCtx &ctx, volatile int *abort) {
    const int st = t % Smem<D>::R, use = t / Smem<D>::R;
    return count_wait(smem_u32(&sm.issued), t + 1, ctx, abort) &&
           bar_wait(smem_u32(&sm.full[st]), use & 1, ctx, abort);
}

// S of one half, a tile at a time, when P V of the half's tile before has read its P. A warp.
template <int D, bool FEW>
__device__ void issue_s(const CrossParams &p, Smem<D> &sm, uint32_t tmem, int half,
                        const DevCtx &ctx) {
    using S = Smem<D>;
    constexpr uint32_t IDESC = idesc_bf16_f32(128, CHUNK, 0, 0);
    volatile int *abort = &sm.abort;
    if (ctx.stall) bar_wait(smem_u32(&sm.drain[half]), 0, ctx, abort);  // test hook: runs out
    const uint64_t dq = desc_rows<128>(smem_u32(sm.q[FEW ? 0 : half]));
    const uint64_t dk = desc_rows<128>(smem_u32(sm.kv[0]));
    const uint32_t cols = tmem + (uint32_t)half * HALF_COLS;
    auto wait = [&](uint64_t &bar, int phase) {
        return bar_wait(smem_u32(&bar), phase & 1, ctx, abort);
    };
    int x = 0, t0 = 0;  // this half's steps; loads before the unit
    bool ok = true;
    for (int i = 0; ok; ++i) {
        if (!(ok = __all_sync(0xffffffffu, sm.units.wait(i, ctx, abort)))) break;
        const LineUnit u = sm.units.u[i % UNITS];
        const int n = u.end - u.begin;
        const bool none = !FEW && half && u.s.n - u.u * p.line.tokens <= p.tokens;
        __syncwarp();
        if (elect_one()) sm.units.release(i);
        if (n == 0) break;
        if (none) {  // no rows in this half: its share in freeing the ring
            for (int j = 0; j < n && ok; ++j) {
                const int t = t0 + 2 * j;
                ok = __all_sync(0xffffffffu, landed(sm, t, ctx, abort));
                if (elect_one()) mbar_arrive(smem_u32(&sm.empty[t % S::R]));
            }
        }
        // (also where it is not used: no phase is passed over)
        ok = __all_sync(0xffffffffu, ok && wait(sm.q_full, i));
        if (none || (FEW && half >= n))
            if (elect_one()) mbar_arrive(smem_u32(&sm.q_empty));
        const int step = FEW ? 2 : 1;
#pragma unroll 1
        for (int j = FEW ? half : 0; j < n && ok && !none; j += step) {
            const int t = t0 + 2 * j, st = t % S::R, nch = chunks(u, u.begin + j);
            ok = landed(sm, t, ctx, abort);
#pragma unroll 1
            for (int c = 0; c < nch; ++c, ++x) {
                const int b = x & 1;
                if (x >= 2) ok = ok && wait(sm.pv_done[half][b], (x >> 1) - 1);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                const uint64_t kd =
                    dk + (uint64_t)(st * (S::TILE_BYTES >> 4) + c * (CHUNK * 128 >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t at = (uint64_t)((kk >> 2) * (S::PART >> 4) + 2 * (kk & 3));
                        tc_mma_f16(cols + (uint32_t)(b * CHUNK), dq + at, kd + at, IDESC, kk > 0);
                    }
                    tc_commit(smem_u32(&sm.s_full[half][b]));
                    if (c == nch - 1) {
                        tc_commit(smem_u32(&sm.empty[st]));
                        if (j + step >= n) tc_commit(smem_u32(&sm.q_empty));
                    }
                }
            }
        }
        t0 += 2 * n;
    }
    __syncwarp();
    if (elect_one()) tc_commit(smem_u32(&sm.drain[half]));  // every MMA is done before TMEM goes
    int zero = 0;
    bar_wait(smem_u32(&sm.drain[half]), 0, ctx, &zero);
}

// P V of one half, 64 keys at a time. A warp.
template <int D, bool FEW>
__device__ void issue_pv(const CrossParams &p, Smem<D> &sm, uint32_t tmem, int half,
                         const DevCtx &ctx) {
    using S = Smem<D>;
    constexpr uint32_t IDESC = idesc_bf16_f32(128, D, 0, 1);
    volatile int *abort = &sm.abort;
    const uint64_t dv = smem_desc_sw128(smem_u32(sm.kv[0]), S::PART, 1024u);
    const uint32_t cols = tmem + (uint32_t)half * HALF_COLS;
    auto wait = [&](uint64_t &bar, int phase) {
        return bar_wait(smem_u32(&bar), phase & 1, ctx, abort);
    };
    int x = 0, t0 = 1, ec = 0;  // this half's steps; V loads before the unit; units
    bool ok = true;
    for (int i = 0; ok; ++i) {
        if (!(ok = __all_sync(0xffffffffu, sm.units.wait(i, ctx, abort)))) break;
        const LineUnit u = sm.units.u[i % UNITS];
        const int n = u.end - u.begin;
        const bool none = !FEW && half && u.s.n - u.u * p.line.tokens <= p.tokens;
        __syncwarp();
        if (elect_one()) sm.units.release(i);
        if (n == 0) break;
        if (none) {
            for (int j = 0; j < n && ok; ++j) {
                const int t = t0 + 2 * j;
                ok = __all_sync(0xffffffffu, landed(sm, t, ctx, abort));
                if (elect_one()) mbar_arrive(smem_u32(&sm.empty[t % S::R]));
            }
        }
        const int first = FEW ? half : 0;
#pragma unroll 1
        for (int j = first; j < n && ok && !none; j += FEW ? 2 : 1) {
            const int t = t0 + 2 * j, st = t % S::R, nch = chunks(u, u.begin + j);
            ok = landed(sm, t, ctx, abort);
            // the first P V overwrites the O that the last unit's epilogue reads
            if (j == first && ec >= 1) ok = ok && wait(sm.o_empty[half], ec - 1);
#pragma unroll 1
            for (int c = 0; c < nch; ++c, ++x) {
                const int b = x & 1;
                ok = ok && wait(sm.p_full[half][b], x >> 1);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                const uint64_t vd =
                    dv + (uint64_t)(st * (S::TILE_BYTES >> 4) + c * (CHUNK * 128 >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < CHUNK / 16; ++kk)
                        tc_mma_f16_ts(cols + O_COL, cols + (uint32_t)(b * CHUNK + 8 * kk),
                                      vd + (uint64_t)(kk * (2048u >> 4)), IDESC,
                                      c > 0 || kk > 0 || j > first);
                    tc_commit(smem_u32(&sm.pv_done[half][b]));
                    if (c == nch - 1) tc_commit(smem_u32(&sm.empty[st]));
                }
            }
        }
        if (ok && !none && first < n) {
            if (elect_one()) tc_commit(smem_u32(&sm.o_full[half]));
            ++ec;
        }
        t0 += 2 * n;
    }
    __syncwarp();
    if (elect_one()) tc_commit(smem_u32(&sm.drain[2 + half]));
    int zero = 0;
    bar_wait(smem_u32(&sm.drain[2 + half]), 0, ctx, &zero);
}

// 16-byte piece c of row r of the O that half 1 leaves for half 0 (no two rows of a warp in one bank).
template <int D> __device__ __forceinline__ float4 *merge_at(Smem<D> &sm, int r, int c) {
    constexpr int N = D / 4;
    return reinterpret_cast<float4 *>(sm.q[1]) + r * N + (c ^ (r & (N - 1)));
}

template <int D, bool FEW>
__device__ void softmax(const CrossParams &p, Smem<D> &sm, uint32_t tmem_base,
                                        const DevCtx &ctx) {
    constexpr int ROWS = FEW ? FEW_ROWS : 256;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = (warp - SOFTMAX) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the half
    const uint32_t tmem = tmem_base + (uint32_t)half * HALF_COLS + ((uint32_t)(quarter * 32) << 16);
    volatile int *abort = &sm.abort;
    if (quarter >= p.warps) return;  // no rows
    auto wait = [&](uint64_t &bar, int phase) {
        return __all_sync(0xffffffffu, bar_wait(smem_u32(&bar), phase & 1, ctx, abort));
    };
    const int tok = p.token(r);
    const float sx = p.scale_l2;
    int x = 0, units = 0, merges = 0;  // this half's steps and units
    for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, sm.units.wait(i, ctx, abort))) return;
        const LineUnit u = sm.units.u[i % UNITS];
        __syncwarp();
        if (lane == 0) sm.units.release(i);
        const int n = u.end - u.begin;
        if (n == 0) return;
        const int tokens = u.s.n - u.u * p.line.tokens - (FEW ? 0 : half * p.tokens);
        if (FEW ? half >= n : tokens <= 0) continue;
        const bool in = r < p.rows && tok < tokens;
        const int head = u.h * p.G + r - tok * p.G;
        const float sink = p.sinks && in ? sink_log2(__ldg(p.sinks + head)) : 0.f;
        float m = NOTHING, l = 0.f;
        bool far = false;   // some row's m is so large that fp32 must subtract it exactly
        bool fresh = true;  // some row has seen no key yet
        const int first = u.begin + (FEW ? half : 0);
#pragma unroll 1
        for (int j = first; j < u.end; j += FEW ? 2 : 1) {
            const int nch = chunks(u, j);
#pragma unroll 1
            for (int c = 0; c < nch; ++c, ++x) {
                if (!wait(sm.s_full[half][x & 1], x >> 1)) return;
                tc_fence_after();
                const int kpos0 = j * STATE_KEYS + c * CHUNK;
                const uint32_t s_tmem = tmem + (uint32_t)((x & 1) * CHUNK);
                const int there = u.s.len - kpos0;  // keys from here on
                const bool key0 = p.sink_mode == 1 && kpos0 == 0;
                uint32_t xs[2][32];
                auto load = [&]() {
                    tmem_ld32(s_tmem, xs[0]);
                    tmem_ld32(s_tmem + 32u, xs[1]);
                    tc_wait_ld();
                    if (there < CHUNK) {
#pragma unroll
                        for (int e = 0; e < CHUNK; ++e) hide_unless(xs[e >> 5][e & 31], e < there);
                    }
                };
                // m from the row's 64 keys, and O and l in its terms
                auto move = [&]() -> bool {
                    float mx = -INFINITY;
#pragma unroll
                    for (int e = 0; e < CHUNK; e += 2)
                        mx = max3(mx, e == 0 && key0 ? -INFINITY : __uint_as_float(xs[e >> 5][e & 31]),
                                  __uint_as_float(xs[e >> 5][(e & 31) + 1]));
                    float top = mx * sx;
                    if (key0) top = fmaxf(top, __uint_as_float(xs[0][0]) * sx + sink);
                    const float mn = fmaxf(m, top), alpha = ex2(m - mn);
                    m = mn;
                    l *= alpha;
                    fresh = __any_sync(0xffffffffu, m == NOTHING);
                    far = __any_sync(0xffffffffu, m != NOTHING && fabsf(m) > FAR);
                    if (j > first || c > 0) {
                        if (!wait(sm.pv_done[half][(x - 1) & 1], (x - 1) >> 1)) return false;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t o[32];
                            tmem_ld32(tmem + O_COL + 32u * q, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(tmem + O_COL + 32u * q, o);
                        }
                    }
                    return true;
                };
                uint32_t pw[32];
                float sum;
                bool moves = fresh;
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    load();
                    if (moves && !move()) return;
                    // P of the row's 64 keys with m as it is, and their sum
                    float fx = sx, off = m == NOTHING ? 0.f : -m;
                    bool bias = key0;
                    if (far) {  // x - m in two roundings, as move() has them: never above 0 there
#pragma unroll
                        for (int e = 0; e < CHUNK; ++e) {
                            float y = __uint_as_float(xs[e >> 5][e & 31]) * sx;
                            if (e == 0 && bias) y += sink;
                            xs[e >> 5][e & 31] = __float_as_uint(y + off);
                        }
                        fx = 1.f, off = 0.f, bias = false;
                    }
                    const uint64_t f2 = f2_pack(fx, fx), off2 = f2_pack(off, off);
                    uint64_t part[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
                    for (int e = 0; e < CHUNK; e += 2) {
                        float a, b;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(xs[e >> 5][e & 31]),
                                                 __uint_as_float(xs[e >> 5][(e & 31) + 1])),
                                         f2, off2),
                                  a, b);
                        if (e == 0 && bias) a += sink;
                        a = ex2(a);
                        b = ex2(b);
                        part[e >> 1 & 1] = f2_add(part[e >> 1 & 1], f2_pack(a, b));
                        pw[e >> 1] = pack_bf16x2(a, b);
                    }
                    float a, b;
                    f2_unpack(f2_add(part[0], part[1]), a, b);
                    sum = a + b;
                    // (after a move no value is above 2^(1/4), so there is no third pass)
                    moves = pass == 0 && __any_sync(0xffffffffu, sum > SUM_LIMIT);
                    if (!moves) break;
                }
                l += sum;
                tmem_st32(s_tmem, pw);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[half][x & 1]));
            }
        }
        // ---- epilogue
        if (!wait(sm.o_full[half], units)) return;
        ++units;
        tc_fence_after();
        const bool joined = FEW && n > 1;  // both halves worked on the unit
        if (joined && half) {
            if (merges >= 1 && !wait(sm.mg_empty, merges - 1)) return;
            ++merges;
            if (r < FEW_ROWS) sm.ml[r] = make_float2(m, l);
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tmem_ld32(tmem + O_COL + 32u * q, o);
                tc_wait_ld();
                if (r < FEW_ROWS)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *merge_at<D>(sm, r, 8 * q + e) =
                            make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                        __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm.mg_full));
                mbar_arrive(smem_u32(&sm.o_empty[half]));
            }
            continue;
        }
        float a0 = 1.f, a1 = 0.f;  // the halves' weights
        if (joined) {
            if (!wait(sm.mg_full, merges)) return;
            ++merges;
            const float2 other = sm.ml[min(r, FEW_ROWS - 1)];
            const float top = fmaxf(m, other.x);
            a0 = ex2(m - top);
            a1 = ex2(other.x - top);
            m = top;
            l = l * a0 + other.y * a1;
        }
        const bool part = u.cut();
        float inv = l == 0.f ? 0.f : 1.f / l;
        const int rr = FEW ? r : half * p.rows + r;
        const size_t slot = ((size_t)blockIdx.x * 2 + (u.begin > 0 ? 0 : 1)) * ROWS + rr;
        float *prow = reinterpret_cast<float *>(p.ws + plan_rows_offset(ROWS)) + slot * D;
        const size_t orow =
            (size_t)(u.s.t0 + u.u * p.line.tokens + (FEW ? 0 : half * p.tokens) + tok) * p.H + head;
        if (in && part) {
            part_sums(p.ws)[slot] = make_float2(m, l);
        } else if (in) {
            float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
            if (p.sink_mode == 2) with_null_sink(sink, lse2, inv);
            if (p.lse) p.lse[orow] = lse2 * LN2;
        }
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tmem + O_COL + 32u * q, o);
            tc_wait_ld();
            if (joined) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 v = *merge_at<D>(sm, min(r, FEW_ROWS - 1), 8 * q + e);
                    o[4 * e] = __float_as_uint(__uint_as_float(o[4 * e]) * a0 + v.x * a1);
                    o[4 * e + 1] = __float_as_uint(__uint_as_float(o[4 * e + 1]) * a0 + v.y * a1);
                    o[4 * e + 2] = __float_as_uint(__uint_as_float(o[4 * e + 2]) * a0 + v.z * a1);
                    o[4 * e + 3] = __float_as_uint(__uint_as_float(o[4 * e + 3]) * a0 + v.w * a1);
                }
            }
            if (in && part) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(prow + 32 * q + e) = make_float4(
                        __uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                        __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            } else if (in) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = pack_bf16x2(__uint_as_float(o[e + 2 * k]) * inv,
                                           __uint_as_float(o[e + 2 * k + 1]) * inv);
                    *reinterpret_cast<uint4 *>(p.o + orow * D + 32 * q + e) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (joined) mbar_arrive(smem_u32(&sm.mg_empty));
            mbar_arrive(smem_u32(&sm.o_empty[half]));
        }
    }
}

template <int D, bool FEW>
__global__ void __launch_bounds__(NTHREADS, 1)
cross_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
             const __grid_constant__ CUtensorMap tv, const __grid_constant__ CrossParams p,
             const __grid_constant__ DevCtx ctx) {
    extern __shared__ __align__(1024) uint8_t dsmem[];
    using S = Smem<D>;
    S &sm = *reinterpret_cast<S *>(dsmem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (smem_u32(dsmem) & 1023u) {  // the swizzle is anchored to 1024-byte boundaries
        if (threadIdx.x == 0) record_error(ctx, DEVERR_LAYOUT);
        return;
    }
    if (warp == 2) {  // a lane a barrier
        if (lane < S::R) {
            mbar_init(smem_u32(&sm.full[lane]), 1);
            mbar_init(smem_u32(&sm.empty[lane]), FEW ? 1 : 2);  // the halves' MMAs
            mbar_init(smem_u32(&sm.raw[lane]), 1);
        }
        if (lane < 2) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&sm.s_full[lane][b]), 1);
                mbar_init(smem_u32(&sm.p_full[lane][b]), p.warps);
                mbar_init(smem_u32(&sm.pv_done[lane][b]), 1);
            }
            mbar_init(smem_u32(&sm.o_full[lane]), 1);
            mbar_init(smem_u32(&sm.o_empty[lane]), p.warps);
            mbar_init(smem_u32(&sm.drain[lane]), 1);
            mbar_init(smem_u32(&sm.drain[2 + lane]), 1);
        }
        if (lane == 0) {
            mbar_init(smem_u32(&sm.q_full), 1);
            mbar_init(smem_u32(&sm.q_empty), 2);
            mbar_init(smem_u32(&sm.mg_full), p.warps);
            mbar_init(smem_u32(&sm.mg_empty), p.warps);
            sm.abort = 0;
            sm.issued = 0;
        }
        sm.units.init(4 + 1 + 2 * p.warps, lane);  // MMA issuers, tails, softmax
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sm.tmem_base), TMEM_COLS);
        tmem_relinquish();
    }
    // rows of Q that no box writes: their S is 0
    for (int half = 0; half < (FEW ? 1 : 2); ++half)
        for (int c = 0; c < S::NH; ++c)
            for (int e = p.rows * 8 + threadIdx.x; e < 128 * 8; e += NTHREADS)
                *reinterpret_cast<uint4 *>(sm.q[half] + c * S::PART + e * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    line_start<false>(p.line, sm.line, ctx);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // registers: 256 threads x 56 + 256 x 200 = the 512 x 128 of the launch
    if (warp < SOFTMAX) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            load_tiles<D, FEW>(p, &tq, &tk, &tv, sm, ctx);
        } else if (warp == 2) {
            clear_tails<D>(sm, ctx);
        } else if (warp < 4) {
            issue_s<D, FEW>(p, sm, tmem, warp >> 1, ctx);
        } else if (warp < 6) {
            issue_pv<D, FEW>(p, sm, tmem, warp & 1, ctx);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        softmax<D, FEW>(p, sm, tmem, ctx);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort == TIMED_OUT) record_error(ctx, DEVERR_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Whether a sequence's rows of a KV head are few enough for the form in which the halves take
// every other tile.
bool few_rows(int max_q_len, int G) { return (long long)max(1, max_q_len) * G <= FEW_ROWS; }

template <int D, bool FEW>
cudaError_t launch(const CrossArgs &a, const DevInfo &dev, cudaStream_t s) {
    constexpr int ROWS = FEW ? FEW_ROWS : 256;
    const int G = a.H / a.Hkv;
    CrossParams p{};
    p.H = a.H;
    p.G = G;
    p.tokens = FEW ? min(FEW_ROWS / G, max(1, a.max_q_len)) : 128 / G;
    p.rows = p.tokens * G;
    p.warps = (p.rows + 31) / 32;
    p.line = LineArgs{a.cu_seqlens, a.kv_starts, a.kv_lens, a.B, a.T, a.S, a.Hkv,
                      FEW ? p.tokens : 2 * p.tokens, FEW ? 1 : 3,
                      a.workspace && a.workspace_bytes >= plan_workspace(ROWS, D)};
    p.scale_l2 = a.scale * LOG2E;
    p.sinks = a.sinks;
    p.sink_mode = a.sink_mode;
    p.o = static_cast<__nv_bfloat16 *>(a.o);
    p.lse = a.lse;
    p.ws = static_cast<uint8_t *>(a.workspace);
    const uint32_t g = (uint32_t)G;
    while ((1ull << p.g_shift) < g) ++p.g_shift;
    p.g_mul = (uint32_t)((((1ull << p.g_shift) - g) << 32) / g + 1);
    CUtensorMap tq, tk, tv;
    if (!map_rows(&tq, a.q, a.q_stride, a.H, D, a.T, G, p.tokens) ||
        !map_rows(&tk, a.k, a.k_stride, a.Hkv, D, a.S, 1, STATE_KEYS) ||
        !map_rows(&tv, a.v, a.v_stride, a.Hkv, D, a.S, 1, STATE_KEYS))
        return cudaErrorInvalidValue;
    static_assert(sizeof(Smem<D>) <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = ensure_smem_attr((const void *)cross_kernel<D, FEW>, sizeof(Smem<D>), dev);
    if (e != cudaSuccess) return e;
    const int grid = min(dev.sm_count, MAX_PIECES);
    if (verbose())
        fprintf(stderr, "sattn: cross_kernel<%d, %d> grid=%d rows=%d split=%d\n", D, (int)FEW, grid,
                p.rows, p.line.split);
    cross_kernel<D, FEW><<<grid, NTHREADS, sizeof(Smem<D>), s>>>(tq, tk, tv, p, make_ctx(dev));
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.line.split) return e;
    PagedArgs j{};  // what the join looks at
    j.H = a.H;
    j.Hkv = a.Hkv;
    j.d = a.d;
    j.sinks = a.sinks;
    j.sink_mode = a.sink_mode;
    j.o = a.o;
    j.lse = a.lse;
    j.workspace = a.workspace;
    return launch_paged_join(j, ROWS, grid, s);
}

}  // namespace

size_t cross_tc_workspace(int max_q_len, int G, int d) {
    return plan_workspace(few_rows(max_q_len, G) ? FEW_ROWS : 256, d);
}

cudaError_t launch_cross_tc(const CrossArgs &a, const DevInfo &dev, cudaStream_t s) {
    if (few_rows(a.max_q_len, a.H / a.Hkv))
        return a.d == 64 ? launch<64, true>(a, dev, s) : launch<128, true>(a, dev, s);
    return a.d == 64 ? launch<64, false>(a, dev, s) : launch<128, false>(a, dev, s);
}

}  // namespace sattn
