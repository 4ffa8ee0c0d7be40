// Key weights of cross attention on the tensor cores (tcgen05), bf16.
//
// What a key receives is a sum over query rows, so the products are taken the other way round,
// S^T = K Q^T: keys are the 128 rows of an MMA, a thread each, query rows its columns, and
//   w += sum over columns of 2^(S^T scale log2(e) - lse log2(e))
// stays in the thread: no sum across threads, no order that changes. Query rows are tokens
// times the heads of a KV group, fetched as boxes of G heads and floor(N / G) tokens.
//
// A unit is 512 keys of a sequence and KV head, four tiles of 128 with a group of four warps
// each; a step is a tile of N query rows, which all four use: a query tile comes from L2, and one
// for a tile of keys alone would take all of its bandwidth. N is 32, 64 or 128, by the rows
// that a sequence has: single tokens then read the keys and next to nothing else.
// One persistent CTA per SM over an equal piece of the line of units (states_plan.cuh);
// the sums of a unit that is cut go to the workspace and are added up by a second launch.
// Roles: warp 0 units and TMA; 1, 2 the products of two tiles each; 3 the rows' denominators;
// 4-19 the tiles' sums.
//
// Sums are fp32, one running sum a key, in the order of the steps, of ex2.approx's 2^-22.
//
// Bound, many rows: products, exponentials and instructions of the sums would each take about
// 2050 cycles a step of 512 keys by 128 rows; it takes 3590, tensor pipe and exponential unit
// 62 and 61 % busy, as a tile's S cannot be made again before its sums have read it and TMEM has no
// room for a second. With d = 64, half the products, 3310 cycles, exponentials 67 %: it is
// the sums' turn that counts. 8 prompts of 100 to 2000 queries over 1000 to 8000 states, 32 heads on
// 8, d = 128: 173 us, 1.34 PFLOP/s, 0.70 of the bf16 peak; d = 64 153 us. With inputs that L2 does
// not hold yet 184 and 160. (Two tiles a unit, a group of warps each, its
// rows' denominators loaded by itself: 252. The tile that is ready first issued first: 187.)
// Bound, few rows: the memory. 64 single tokens over 257 to 6404 states: 90 us with the second
// launch, 5.4 TB/s; with d = 64, added up, 56 us (128 tokens 91 written, and 117 before
// neighbouring heads were taken side by side, states_plan.cuh).
#include <math.h>
#include <stdio.h>

#include "paged_plan.cuh"
#include "states_plan.cuh"

namespace sattn {
namespace {

constexpr int NTHREADS = 640;
constexpr int SUMS = 4;    // first warp of the sums
constexpr int UNITS = 4;   // units handed on ahead
constexpr int TILES = UNIT_TILES, UNIT_KEYS = TILES * STATE_KEYS;
constexpr int LR = 4;                // steps whose denominators are ahead
// lse in size from which its rounding counts: where it is off by a thousandth and more, a
// weight is taken no larger than 1 (of lse 10^10 it could be 2^1000)
constexpr float LARGE = 1 << 14;
constexpr uint32_t TMEM_COLS = 512;  // 128 a tile

struct WeightParams {
    LineArgs line;
    int H, G, rows;    // rows: of a query tile that hold tokens
    uint32_t n;        // and columns of its product
    const float *lse;
    float scale_l2;
    const float *sinks;  // of key 0, or nullptr
    float *weights;
    int accumulate;
    uint8_t *ws;
    uint32_t g_mul, g_shift;

    // row / G for 0 <= row < 2^31 (as PlanArgs::token)
    __device__ __forceinline__ int token(int row) const {
        return (int)((__umulhi(g_mul, (uint32_t)row) + (uint32_t)row) >> g_shift);
    }
};

template <int D> struct alignas(1024) Smem {
    static constexpr int NH = D / 64;            // 64-column parts of a row
    static constexpr uint32_t PART = 128 * 128;  // 128 rows of 64 bf16
    static constexpr uint32_t TILE_BYTES = NH * PART;
    static constexpr int KR = D == 128 ? 1 : 2;  // tiles of keys ahead, for each of a unit's
    static constexpr int QR = D == 128 ? 3 : 6;  // tiles of queries
    uint8_t k[TILES][KR][TILE_BYTES];
    uint8_t q[QR][TILE_BYTES];
    float lse[LR][128];  // -lse log2(e), -inf where a row does not count
    int cols[LR];        // the step's rows; ~rows where one does not count, or has a large lse
    LineStart line;
    LineRing<UNITS> units;
    uint64_t k_full[TILES][KR], k_empty[TILES][KR], q_full[QR], q_empty[QR];
    uint64_t lse_full[LR], lse_empty[LR], s_full[TILES], s_empty[TILES], drain[2];
    uint32_t tmem_base;
    int abort;
};

// Workspace: PlanNote [pieces], sums [pieces][2][UNIT_KEYS] (part 0 of a piece is its first
// unit if that began earlier, part 1 its last unit if that begins here and goes on). In a note
// t0 is the unit's first row of the states, nrows its keys.
constexpr size_t SUMS_OFFSET = MAX_PIECES * sizeof(PlanNote);
constexpr size_t WORKSPACE = SUMS_OFFSET + (size_t)MAX_PIECES * 2 * UNIT_KEYS * sizeof(float);

// Keys of the unit's tile g.
__device__ __forceinline__ int keys_of(const LineUnit &u, int g) {
    return min(STATE_KEYS, u.s.len - u.u * UNIT_KEYS - g * STATE_KEYS);
}

template <int D>
__device__ void load_tiles(const WeightParams &p, const CUtensorMap *tq, const CUtensorMap *tk,
                           Smem<D> &sm, const DevCtx &ctx) {
    using S = Smem<D>;
    if ((threadIdx.x & 31) != 0) return;
    volatile int *abort = &sm.abort;
    LineIter<true> it(p.line, sm.line);
    if (p.line.split) {
        PlanNote n{};
        if (it.live) {
            const LineUnit &u = it.u;
            n.cont = u.begin > 0;
            n.through = u.begin > 0 && u.end < u.steps;
            n.t0 = u.s.s0 + u.u * UNIT_KEYS;
            n.h = p.line.head(u.h);
            n.nrows = min(UNIT_KEYS, u.s.len - u.u * UNIT_KEYS);
        }
        reinterpret_cast<PlanNote *>(p.ws)[blockIdx.x] = n;
    }
    int kt[TILES] = {}, qt = 0, index = 0;  // loads; units
    bool ok = true;
#pragma unroll 1
    for (; it.live && ok; it.next(p.line, sm.line)) {
        LineUnit u = it.u;
        u.h = p.line.head(u.h);
        ok = sm.units.put(index++, u, ctx, abort);
#pragma unroll
        for (int g = 0; g < TILES; ++g) {
            if (!ok || keys_of(u, g) <= 0) continue;
            const int st = kt[g] % S::KR, use = kt[g] / S::KR;
            if (use >= 1) ok = bar_wait(smem_u32(&sm.k_empty[g][st]), (use - 1) & 1, ctx, abort);
            if (!ok) continue;
            const uint32_t bar = smem_u32(&sm.k_full[g][st]);
            mbar_arrive_expect_tx(bar, S::TILE_BYTES);
#pragma unroll
            for (int c = 0; c < S::NH; ++c)
                tma_load_3d(smem_u32(sm.k[g][st]) + c * S::PART, tk, bar, 64 * c, u.h,
                            u.s.s0 + u.u * UNIT_KEYS + g * STATE_KEYS);
            ++kt[g];
        }
#pragma unroll 1
        for (int j = u.begin; j < u.end && ok; ++j) {
            const int st = qt % S::QR, use = qt / S::QR;
            if (use >= 1) ok = bar_wait(smem_u32(&sm.q_empty[st]), (use - 1) & 1, ctx, abort);
            if (!ok) break;
            const uint32_t bar = smem_u32(&sm.q_full[st]);
            mbar_arrive_expect_tx(bar, (uint32_t)(S::NH * p.rows * 128));
#pragma unroll
            for (int c = 0; c < S::NH; ++c)
                tma_load_3d(smem_u32(sm.q[st]) + c * p.n * 128, tq, bar, 64 * c, u.h * p.G,
                            u.s.t0 + j * p.line.tokens);
            ++qt;
        }
    }
    if (ok) {
        LineUnit last{};
        sm.units.put(index, last, ctx, abort);
    }
    int zero = 0;  // copies in flight land before the CTA leaves
#pragma unroll 1
    for (int st = 0; st < S::KR; ++st)
#pragma unroll
        for (int g = 0; g < TILES; ++g)
            if (st < kt[g])
                bar_wait(smem_u32(&sm.k_full[g][st]), (kt[g] - 1 - st) / S::KR & 1, ctx, &zero);
#pragma unroll 1
    for (int st = 0; st < S::QR && st < qt; ++st)
        bar_wait(smem_u32(&sm.q_full[st]), (qt - 1 - st) / S::QR & 1, ctx, &zero);
}

// The denominators of the steps' query rows: a warp, four steps' loads at a time.
template <int D>
__device__ void load_lse(const WeightParams &p, Smem<D> &sm, const DevCtx &ctx) {
    const int lane = threadIdx.x & 31;
    volatile int *abort = &sm.abort;
    int tok[4], head[4];  // of rows lane, lane + 32, ..
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        tok[e] = p.token(lane + 32 * e);
        head[e] = lane + 32 * e - tok[e] * p.G;
    }
    int q = 0;  // steps
    for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, sm.units.wait(i, ctx, abort))) return;
        const LineUnit u = sm.units.u[i % UNITS];
        __syncwarp();
        if (lane == 0) sm.units.release(i);
        if (u.begin == u.end) return;
#pragma unroll 1
        for (int j0 = u.begin; j0 < u.end; j0 += 4) {
            float x[4][4];
            uint32_t rows = 0;  // bit 4 s + e: x[s][e] is a row's
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = (j0 + s) * p.line.tokens + tok[e];
                    x[s][e] = INFINITY;
                    if (j0 + s < u.end && lane + 32 * e < p.rows && t < u.s.n) {
                        x[s][e] = __ldg(p.lse + (size_t)(u.s.t0 + t) * p.H + u.h * p.G + head[e]);
                        rows |= 1u << (4 * s + e);
                    }
                }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (j0 + s >= u.end) break;
                const int b = q % LR;
                if (q >= LR && !__all_sync(0xffffffffu, bar_wait(smem_u32(&sm.lse_empty[b]),
                                                                 (q / LR - 1) & 1, ctx, abort)))
                    return;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sm.lse[b][lane + 32 * e] = isinf(x[s][e]) ? -INFINITY : -x[s][e] * LOG2E;
                bool odd = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    odd |= fabsf(x[s][e]) > LARGE && rows >> (4 * s + e) & 1;
                odd = __any_sync(0xffffffffu, odd);
                const int cols = min(p.line.tokens, u.s.n - (j0 + s) * p.line.tokens) * p.G;
                if (lane == 0) sm.cols[b] = odd ? ~cols : cols;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.lse_full[b]));
                ++q;
            }
        }
    }
}

// The products of tiles 2 w and 2 w + 1: a warp.
template <int D>
__device__ void issue(const WeightParams &p, Smem<D> &sm, uint32_t tmem, int w, const DevCtx &ctx) {
    using S = Smem<D>;
    const uint32_t idesc = idesc_bf16_f32(128, p.n, 0, 0);
    volatile int *abort = &sm.abort;
    if (ctx.stall) bar_wait(smem_u32(&sm.drain[w]), 0, ctx, abort);  // test hook: runs out
    const uint64_t dk = desc_rows<128>(smem_u32(sm.k[2 * w][0]));
    const uint64_t dq = desc_rows<128>(smem_u32(sm.q[0]));
    auto wait = [&](uint64_t &bar, int phase) {
        return bar_wait(smem_u32(&bar), phase & 1, ctx, abort);
    };
    int kt[2] = {0, 0}, x[2] = {0, 0}, qt = 0;  // the tiles' loads and steps; loads of queries
    bool ok = true;
    for (int i = 0; ok; ++i) {
        if (!(ok = __all_sync(0xffffffffu, sm.units.wait(i, ctx, abort)))) break;
        const LineUnit u = sm.units.u[i % UNITS];
        const int n = u.end - u.begin;
        const int mine = keys_of(u, 2 * w + 1) > 0 ? 2 : keys_of(u, 2 * w) > 0 ? 1 : 0;  // tiles
        __syncwarp();
        if (elect_one()) sm.units.release(i);
        if (n == 0) break;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j, ++qt) {
            const int st = qt % S::QR;
            ok = __all_sync(0xffffffffu, wait(sm.q_full[st], qt / S::QR));
            if (!mine && ok && elect_one()) mbar_arrive(smem_u32(&sm.q_empty[st]));
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                if (a >= mine || !ok) continue;
                const int g = 2 * w + a, ks = kt[a] % S::KR;
                if (j == 0) ok = wait(sm.k_full[g][ks], kt[a] / S::KR);
                if (x[a] >= 1) ok = ok && wait(sm.s_empty[g], x[a] - 1);
                if (!(ok = __all_sync(0xffffffffu, ok))) continue;
                tc_fence_after();
                const uint64_t kd = dk + (uint64_t)((a * S::KR + ks) * (S::TILE_BYTES >> 4));
                const uint64_t qd = dq + (uint64_t)(st * (S::TILE_BYTES >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc_mma_f16(tmem + (uint32_t)(g * 128),
                                   kd + (uint64_t)((kk >> 2) * (S::PART >> 4) + 2 * (kk & 3)),
                                   qd + (uint64_t)((kk >> 2) * (p.n * 128 >> 4) + 2 * (kk & 3)),
                                   idesc, kk > 0);
                    tc_commit(smem_u32(&sm.s_full[g]));
                    if (a == mine - 1) tc_commit(smem_u32(&sm.q_empty[st]));
                    if (j == n - 1) tc_commit(smem_u32(&sm.k_empty[g][ks]));
                }
                ++x[a];
                kt[a] += j == n - 1;
            }
        }
    }
    __syncwarp();
    if (elect_one()) tc_commit(smem_u32(&sm.drain[w]));  // every MMA is done before TMEM goes
    int zero = 0;
    bar_wait(smem_u32(&sm.drain[w]), 0, ctx, &zero);
}

// 0 at most; a NaN stays
__device__ __forceinline__ float cap(float y) { return y > 0.f ? 0.f : y; }

// The sum of 2^(x sx + l) over 32 columns, l from shared memory.
__device__ __forceinline__ float sum32(const uint32_t (&xs)[32], uint64_t sx, const float *lse) {
    uint64_t part[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(lse + e);
        float a0, a1, a2, a3;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(xs[e]), __uint_as_float(xs[e + 1])), sx,
                         f2_pack(l.x, l.y)), a0, a1);
        f2_unpack(f2_fma(f2_pack(__uint_as_float(xs[e + 2]), __uint_as_float(xs[e + 3])), sx,
                         f2_pack(l.z, l.w)), a2, a3);
        part[0] = f2_add(part[0], f2_pack(ex2(a0), ex2(a1)));
        part[1] = f2_add(part[1], f2_pack(ex2(a2), ex2(a3)));
    }
    float a0, a1;
    f2_unpack(f2_add(part[0], part[1]), a0, a1);
    return a0 + a1;
}

// The same of all columns of a step with such rows: without those that do not count, whose
// query may hold anything, and no more than 1 of each; with the sinks of key 0 for the thread that
// has it. (A call, told by the sign of the step's rows: with its code inside the loop of the
// other steps 64 single tokens of d = 64 take 59 us instead of 56.)
__device__ __noinline__ float sum_apart(const WeightParams &p, uint32_t tmem, int cols,
                                        const float *lse, const float *sinks) {
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < cols; c += 32) {
        uint32_t xs[32];
        tmem_ld32(tmem + (uint32_t)c, xs);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const int col = c + e;
            const float l = lse[col];  // (-inf behind the last column too)
            float y = fmaf(__uint_as_float(xs[e]), p.scale_l2, l);
            if (sinks) y += state_sink(__ldg(sinks + col - p.token(col) * p.G));
            sum += l == -INFINITY ? 0.f : ex2(cap(y));
        }
    }
    return sum;
}

// The sums of tile g.
template <int D>
__device__ void sum_up(const WeightParams &p, Smem<D> &sm, uint32_t tmem_base, const DevCtx &ctx) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = (warp - SUMS) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tmem = tmem_base + (uint32_t)(g * 128) + ((uint32_t)(quarter * 32) << 16);
    volatile int *abort = &sm.abort;
    auto wait = [&](uint64_t &bar, int phase) {
        return __all_sync(0xffffffffu, bar_wait(smem_u32(&bar), phase & 1, ctx, abort));
    };
    const float sx = p.scale_l2;
    const uint64_t sx2 = f2_pack(sx, sx);
    int q = 0, x = 0;  // steps; this tile's steps
    for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, sm.units.wait(i, ctx, abort))) return;
        const LineUnit u = sm.units.u[i % UNITS];
        __syncwarp();
        if (lane == 0) sm.units.release(i);
        if (u.begin == u.end) return;
        const int keys = keys_of(u, g);
        const bool first = p.sinks && u.u == 0 && g == 0 && quarter == 0;  // lane 0 has key 0
        const size_t at = (size_t)u.h * p.line.S + u.s.s0 + u.u * UNIT_KEYS + g * STATE_KEYS + r;
        float old = 0.f, w = 0.f;
        if (p.accumulate && !u.cut() && r < keys) old = p.weights[at];
#pragma unroll 1
        for (int j = u.begin; j < u.end; ++j, ++q) {
            const int b = q % LR;
            if (!wait(sm.lse_full[b], q / LR)) return;
            if (keys <= 0) {  // no phase is passed over
                if (lane == 0) mbar_arrive(smem_u32(&sm.lse_empty[b]));
                continue;
            }
            if (!wait(sm.s_full[g], x)) return;
            ++x;
            tc_fence_after();
            const float *lse = sm.lse[b];
            const int cols = sm.cols[b];
            float sum = 0.f;
            if (cols > 96 && !first) {  // the next 32 columns come while these are summed
                uint32_t xs[2][32];
                tmem_ld32(tmem, xs[0]);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c < 3) tmem_ld32(tmem + 32u * (c + 1), xs[(c + 1) & 1]);
                    if (c == 3 && cols < 128) {  // columns of no row may hold anything
#pragma unroll
                        for (int e = 0; e < 32; ++e) hide_unless(xs[1][e], 96 + e < cols);
                    }
                    sum += sum32(xs[c & 1], sx2, lse + 32 * c);
                    if (c < 3) tc_wait_ld();
                    if (c == 2) {  // S has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty[g]));
                    }
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < cols; c += 32) {
                    uint32_t xs[32];
                    tmem_ld32(tmem + (uint32_t)c, xs);
                    tc_wait_ld();
                    if (cols - c < 32) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) hide_unless(xs[e], e < cols - c);
                    }
                    if (!first) {
                        sum += sum32(xs, sx2, lse + c);
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int col = c + e, h = col - p.token(col) * p.G;
                        const float z = lane == 0 ? state_sink(__ldg(p.sinks + u.h * p.G + h)) : 0.f;
                        const float y = fmaf(__uint_as_float(xs[e]), sx, lse[col]);
                        sum += ex2(y == -INFINITY ? y : y + z);  // (whatever the sink)
                    }
                }
                if (cols < 0)
                    sum = sum_apart(p, tmem, ~cols, lse,
                                    first && lane == 0 ? p.sinks + u.h * p.G : nullptr);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty[g]));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.lse_empty[b]));
            w += sum;
        }
        if (keys <= 0) continue;
        if (u.cut()) {
            float *part = reinterpret_cast<float *>(p.ws + SUMS_OFFSET) +
                          ((size_t)blockIdx.x * 2 + (u.begin > 0 ? 0 : 1)) * UNIT_KEYS;
            part[g * STATE_KEYS + r] = w;
        } else if (r < keys) {
            p.weights[at] = old + w;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1)
weights_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ WeightParams p, const __grid_constant__ DevCtx ctx) {
    extern __shared__ __align__(1024) uint8_t dsmem[];
    using S = Smem<D>;
    S &sm = *reinterpret_cast<S *>(dsmem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (smem_u32(dsmem) & 1023u) {  // the swizzle is anchored to 1024-byte boundaries
        if (threadIdx.x == 0) record_error(ctx, DEVERR_LAYOUT);
        return;
    }
    if (warp == 0) {  // a lane a barrier
        if (lane < TILES) {
#pragma unroll
            for (int i = 0; i < S::KR; ++i) {
                mbar_init(smem_u32(&sm.k_full[lane][i]), 1);
                mbar_init(smem_u32(&sm.k_empty[lane][i]), 1);
            }
            mbar_init(smem_u32(&sm.s_full[lane]), 1);
            mbar_init(smem_u32(&sm.s_empty[lane]), 4);
        }
        if (lane < LR) {
            mbar_init(smem_u32(&sm.lse_full[lane]), 1);
            mbar_init(smem_u32(&sm.lse_empty[lane]), 4 * TILES);
        }
        if (lane < S::QR) {
            mbar_init(smem_u32(&sm.q_full[lane]), 1);
            mbar_init(smem_u32(&sm.q_empty[lane]), 2);
        }
        if (lane < 2) mbar_init(smem_u32(&sm.drain[lane]), 1);
        if (lane == 0) sm.abort = 0;
        sm.units.init(2 + 1 + 4 * TILES, lane);
        fence_mbar_init();
        __syncwarp();
    } else if (warp == 1) {
        tmem_alloc(smem_u32(&sm.tmem_base), TMEM_COLS);
        tmem_relinquish();
    } else if (warp == 2 && lane < 2) {
        prefetch_tmap(lane == 0 ? &tk : &tq);
    }
    if (!line_by_warp(p.line))
        line_start<true>(p.line, sm.line, reinterpret_cast<long long *>(sm.lse), ctx);
    tc_fence_before();
    set_up(warp == 0);
    tc_fence_after();
    if (warp == 0 && line_by_warp(p.line)) line_start_warp<true>(p.line, sm.line, ctx);
    const uint32_t tmem = warp == 0 ? 0u : sm.tmem_base;  // (the loader has not waited for it)
    if (warp == 0) {
        load_tiles<D>(p, &tq, &tk, sm, ctx);
        __syncwarp();
    } else if (warp < 3) {
        issue<D>(p, sm, tmem, warp - 1, ctx);
    } else if (warp == 3) {
        load_lse<D>(p, sm, ctx);
    } else {
        sum_up<D>(p, sm, tmem, ctx);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort == TIMED_OUT) record_error(ctx, DEVERR_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Adds up the sums of units that were cut, in the order of their pieces: block i takes the unit
// that the boundary behind CTA i's piece cuts, if that is the first inside the unit.
__global__ void __launch_bounds__(UNIT_KEYS)
add_kernel(const uint8_t *ws, int grid, int side, int S, float *weights, int accumulate) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PlanNote *notes = reinterpret_cast<const PlanNote *>(ws);
    const float *sums = reinterpret_cast<const float *>(ws + SUMS_OFFSET);
    const int c = blockIdx.x + side, key = threadIdx.x;
    const PlanNote me = notes[c], prev = notes[c - side];
    if (!me.cont || key >= me.nrows || (prev.cont && prev.through)) return;
    float w = sums[((size_t)(c - side) * 2 + 1) * UNIT_KEYS + key] + sums[(size_t)c * 2 * UNIT_KEYS + key];
    bool on = me.through;
    for (int i = c + side; on && i < grid; i += side) {
        w += sums[(size_t)i * 2 * UNIT_KEYS + key];
        on = notes[i].through;
    }
    float *at = weights + (size_t)me.h * S + me.t0 + key;
    *at = accumulate ? *at + w : w;
}

template <int D>
cudaError_t launch(const KeyWeightArgs &a, const DevInfo &dev, cudaStream_t s) {
    const int G = a.H / a.Hkv, n = max(1, a.max_q_len);
    const long long need = (long long)n * G;
    WeightParams p{};
    p.H = a.H;
    p.G = G;
    p.n = need <= 32 ? 32 : need <= 64 ? 64 : 128;
    const int tokens = min((int)p.n / G, n);
    p.rows = tokens * G;
    const bool split = a.workspace && a.workspace_bytes >= WORKSPACE;
    p.line = LineArgs{a.cu_seqlens, a.kv_starts, a.kv_lens, a.B, a.T, a.S, a.Hkv, tokens, 0,
                      TILES, 1, TILES, split};
    const int side = p.n < 128 && a.Hkv % 2 == 0 && dev.sm_count > 1 ? 2 : 1;
    const int grid = line_grid(p.line, min(dev.sm_count, MAX_PIECES), side);
    p.lse = a.lse;
    p.scale_l2 = a.scale * LOG2E;
    p.sinks = a.sink_mode == 1 ? a.sinks : nullptr;
    p.weights = a.weights;
    p.accumulate = a.accumulate;
    p.ws = static_cast<uint8_t *>(a.workspace);
    const uint32_t g = (uint32_t)G;
    while ((1ull << p.g_shift) < g) ++p.g_shift;
    p.g_mul = (uint32_t)((((1ull << p.g_shift) - g) << 32) / g + 1);
    CUtensorMap tq, tk;
    if (!map_rows(&tq, a.q, a.q_stride, a.H, D, a.T, G, tokens) ||
        !map_rows(&tk, a.k, a.k_stride, a.Hkv, D, a.S, 1, STATE_KEYS))
        return cudaErrorInvalidValue;
    static_assert(sizeof(Smem<D>) <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = ensure_smem_attr((const void *)weights_kernel<D>, sizeof(Smem<D>), dev);
    if (e != cudaSuccess) return e;
    if (verbose())
        fprintf(stderr, "sattn: weights_kernel<%d> grid=%d n=%u rows=%d split=%d\n", D, grid, p.n,
                p.rows, p.line.split);
    weights_kernel<D><<<grid, NTHREADS, sizeof(Smem<D>), s>>>(tq, tk, p, make_ctx(dev));
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.line.split || grid <= side) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid - side));
    cfg.blockDim = dim3(UNIT_KEYS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, add_kernel, static_cast<const uint8_t *>(p.ws), grid, side, a.S,
                              a.weights, a.accumulate);
}

}  // namespace

size_t weights_tc_workspace() { return WORKSPACE; }

cudaError_t launch_weights_tc(const KeyWeightArgs &a, const DevInfo &dev, cudaStream_t s) {
    return a.d == 64 ? launch<64>(a, dev, s) : launch<128>(a, dev, s);
}

}  // namespace sattn
