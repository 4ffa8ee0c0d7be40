// Attention of many tokens a sequence over the paged e4m3 cache (tcgen05).
//
// A unit is 256 query rows (tokens times the heads of a KV group) in two halves
// of 128, the rows of the MMAs; both halves use each 128-key tile. Here the
// products bound the time, so operands are what the tensor core takes at full
// rate with next to no loss:
//  * S = Q K^T takes K's codes as they are. Q is scaled by a power of two a row
//    (its largest value then lies in [128, 256)) and split, q = hi + lo with
//    hi = e4m3(q), lo = e4m3(q - hi): together 8 significant bits, exactly a
//    bf16's, down to 2^-10 of the row's largest value, and an error of at most 2^-18 of that
//    below. Both products go into one accumulator; two e4m3 MMAs take the time
//    of one in f16.
//  * O += P V: a probability needs more range than two e4m3 terms have, so V's
//    codes are widened to f16 in shared memory (exact), once a tile for 256
//    rows, and P is rounded to f16: 2^(7 + x - m) <= 2^15, so 2^-12
//    relative down to 2^-21 of the largest weight and at most 2^-32 of it below.
// S, O and the row sums are fp32.
//
// The keys are taken 64 at a time:
//   S [128 x 64] of a half into TMEM, one of two buffers
//   x = S * (scale log2(e) * k_scale) + log2(v_scale): the value's scale goes
//       into the exponent, so V's codes need none; the row sum divides it out.
//       Both are one number for a page, that is for 16 columns or more
//   P = 2^(7 + x - m), f16, over the first columns of S's own buffer
//   O += P V, P from TMEM
// m is the maximum of a row's first keys and stays unless 64 keys' P sum up to more than
// 2^15: P is computed on trust in one pass over S that looks for no maximum,
// and where the sum says that this was wrong m moves, O is rescaled and the pass
// is repeated. TMEM: S / P 2 x 2 x 64 columns, O 2 x D: all 512 for D = 128, hence
// the shared columns of S and P.
//
// One persistent CTA per SM over an equal piece of the tiles (paged_plan.cuh):
//   warp 0       the units; TMA: tiles of K and V, two rings of STAGES
//   warps 1, 3   S of the halves, two steps ahead of the softmax
//   warps 8, 10  P V of the halves
//   warp 2       the pages' scales
//   warps 4-7    widening: V's codes to f16 tiles (two buffers)
//   warps 12-15, 16-19   Q, softmax and epilogue of the halves, a thread a row
//
// Bound: the chain of a step, S ready -> 64 exponentials a thread -> P V -> the S
// that takes P's columns, about 1900 cycles where the products need 1300. For 2048 tokens
// behind 30720 cached ones (32 heads on 8, d = 128) 844 us, 1.26 PFLOP/s; the
// products alone would take 549. Prompts of 61 .. 1500 tokens 220 us: a unit costs about
// 15000 cycles by itself (Q, the first maximum, O); 8 us of them are the look at each unit's
// value scales. 88 to 108 bytes a thread are spilled, in which role the compiler does not say.
// Measured against 839 us for the first, before the units of far scales:
//   one thread for both products of a half            939 us (an MMA takes its
//     thread 65 to 80 cycles to issue, a commit or a wait that is met 100 to 200)
//   the same, every index kept up instead of computed   875 us
//   S of 128 keys at once, in one buffer               1077 us
//   two threads a row, 32 keys each                    1028 us (no registers left
//     to have the next loads in flight)
//   Q by the widening warps, one unit ahead             854 us, the prompts 309
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdio.h>

#include "paged_mma.cuh"
#include "paged_plan.cuh"

namespace sattn {
namespace {

constexpr int ROWS = 256;
constexpr int NTHREADS = 640;
constexpr int SOFTMAX = 12;  // first softmax warp
constexpr int STAGES = 3;
constexpr int SRING = 8;
// A unit's own cost in tiles, of about 3800 cycles each: with 3, 4 and 5 the prompts
// above take 221, 211 and 213 us.
constexpr int EXTRA = 4;
constexpr int UNITS = 4;  // units handed on ahead
constexpr float BASE = 7.f;       // P = 2^(BASE + x - m)
constexpr float SUM_LIMIT = 32768.f;  // m moves when 64 keys' P sum up to more
constexpr float FAR = 1 << 20;  // m up to which x - m may be taken in one rounding

struct PrefillParams {
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

template <int D> struct alignas(1024) Smem {
    static constexpr uint32_t HALF = 128 * 128;  // 128 rows of 64 f16
    static constexpr int NH = D / 64;            // such column halves a tile
    uint8_t q[2][2][128 * D];  // half; hi, lo
    uint8_t k[STAGES][TILE * D];
    uint8_t v[STAGES][TILE * D];
    uint8_t v16[2][NH * HALF];
    float4 sc[SRING][8];
    int zero[SRING];  // a visible page of the tile has a zero value scale
    PlanStart plan;
    UnitRing<ROWS, UNITS> units;
    uint64_t k_full[STAGES], k_empty[STAGES], v8_full[STAGES], v8_empty[STAGES];
    uint64_t v_full[2], v_empty[2];
    uint64_t sc_full[SRING], sc_empty[SRING];
    uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], o_empty[2], drain[4];
    uint32_t tmem_base;
    int abort;
};
constexpr uint32_t TMEM_COLS = 512, HALF_COLS = 256, O_COL = 128;
constexpr int SUB = 64;  // keys a step

// kind::f16, f16 operands, fp32 accumulate; b_mn: B is stored with N contiguous.
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t b_mn) {
    return (1u << 4) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
template <int D>
__device__ void load_tiles(const PrefillParams &p, const CUtensorMap *tk, const CUtensorMap *tv,
                           Smem<D> &sm, const DevCtx &ctx) {
    const int lane = threadIdx.x & 31;
    const int per_tile = TILE >> p.page_shift, chunk = 32 >> (7 - p.page_shift);
    const uint32_t page_bytes = (uint32_t)p.page * D;
    int t = 0;  // tiles
    bool ok = true;
    bool bad = false;
    if (lane == 0) {
        prefetch_tmap(tk);
        prefetch_tmap(tv);
    }
    UnitIter<ROWS> it(p.plan, sm.plan);
    if (p.plan.split && lane == 0) write_note(it, p.ws);
    int index = 0;
#pragma unroll 1
    for (; it.live && ok; it.next(p.plan, sm.plan)) {
        const Unit<ROWS> &u = it.u;
        if (u.begin == u.end) continue;
        if (lane == 0) ok = sm.units.put(index, u, ctx, &sm.abort);
        ++index;
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        for (int c = u.begin; c < u.end && ok; c += chunk) {
            const int j = (u.t_first + c) * per_tile + lane;
            const int pid = c + lane / per_tile < u.end
                                ? page_of(p.page_table, p.max_pages, p.num_pages, p.page_shift, u, j)
                                : -1;
            bad |= pid == -2;
            const int row = pid < 0 ? p.rows_total : (pid * p.plan.Hkv + u.h) * p.page;
            const int nt = min(chunk, u.end - c);
            for (int i = 0; i < nt && ok; ++i, ++t) {
                const int st = t % STAGES, use = t / STAGES;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t full = smem_u32(kv ? &sm.v8_full[st] : &sm.k_full[st]);
                    const uint32_t empty = smem_u32(kv ? &sm.v8_empty[st] : &sm.k_empty[st]);
                    const uint32_t dst = smem_u32(kv ? sm.v[st] : sm.k[st]);
                    bool go = true;
                    if (lane == 0) {
                        if (use >= 1) go = bar_wait(empty, (use - 1) & 1, ctx, &sm.abort);
                        if (go) mbar_arrive_expect_tx(full, TILE * D);
                    }
                    ok = __shfl_sync(0xffffffffu, go ? 1 : 0, 0) != 0;
                    if (!ok) break;
                    const int s = lane - i * per_tile;
                    if (s >= 0 && s < per_tile)
                        tma_load_2d(dst + (uint32_t)s * page_bytes, kv ? tv : tk, full, 0, row);
                }
            }
        }
    }
    if (lane == 0 && ok) {
        Unit<ROWS> last{};
        sm.units.put(index, last, ctx, &sm.abort);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(ctx, DEVERR_INDEX);
    if (lane == 0) {  // copies in flight land before the CTA leaves
        int zero = 0;
#pragma unroll 1
        for (int i = 1; i <= STAGES && i <= t; ++i) {
            bar_wait(smem_u32(&sm.k_full[(t - i) % STAGES]), ((t - i) / STAGES) & 1, ctx, &zero);
            bar_wait(smem_u32(&sm.v8_full[(t - i) % STAGES]), ((t - i) / STAGES) & 1, ctx, &zero);
        }
    }
}

template <int D>
__device__ void load_scales(const PrefillParams &p, Smem<D> &sm, const DevCtx &ctx) {
    const int lane = threadIdx.x & 31;
    const int per_tile = TILE >> p.page_shift, chunk = 32 >> (7 - p.page_shift);
    int t = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
        ok = __all_sync(0xffffffffu, sm.units.wait(i, ctx, &sm.abort));
        if (!ok) break;
        Unit<ROWS> &u = sm.units.u[i % UNITS];
        if (u.begin == u.end) break;
        for (int c = u.begin; c < u.end && ok; c += chunk) {
            const int j = (u.t_first + c) * per_tile + lane;
            const int pid = c + lane / per_tile < u.end
                                ? page_of(p.page_table, p.max_pages, p.num_pages, p.page_shift, u, j)
                                : -1;
            const float4 s = page_scales(p.k_scale, p.v_scale, pid, p.plan.Hkv, u.h);
            if (c == u.begin) {
                // before the first, whether any of the unit's is far: eight pages a lane in flight
                bool far = pid >= 0 && far_log2(s.y);
                const int end = (u.t_first + u.end) * per_tile;
#pragma unroll 1
                for (int j1 = j + 32; j1 - lane < end; j1 += 256) {
                    int id[8];
                    float vs[8];
#pragma unroll
                    for (int a = 0; a < 8; ++a)
                        id[a] = j1 + 32 * a < end
                                    ? page_of(p.page_table, p.max_pages, p.num_pages, p.page_shift,
                                              u, j1 + 32 * a)
                                    : -1;
#pragma unroll
                    for (int a = 0; a < 8; ++a)
                        vs[a] = id[a] < 0 ? 1.f
                                          : __ldg(p.v_scale + (size_t)id[a] * p.plan.Hkv + u.h);
#pragma unroll
                    for (int a = 0; a < 8; ++a) far = far || far_scale(vs[a]);
                }
                far = __any_sync(0xffffffffu, far);
                if (lane == 0 && far) u.far = 1;
            }
            const int nt = min(chunk, u.end - c);
            for (int a = 0; a < nt; ++a, ++t) {
                const int st = t % SRING, use = t / SRING;
                if (use >= 1)
                    ok = bar_wait(smem_u32(&sm.sc_empty[st]), (use - 1) & 1, ctx, &sm.abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const int sl = lane - a * per_tile;
                const bool here = sl >= 0 && sl < per_tile;
                if (here) sm.sc[st][sl] = s;
                const bool zero = __any_sync(0xffffffffu, here && pid >= 0 && s.w == 0.f);
                if (lane == 0) sm.zero[st] = zero;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.sc_full[st]));
            }
        }
        __syncwarp();
        if (lane == 0) sm.units.release(i);
    }
}

// Widens tiles; 128 threads. Returns early when a wait gives up
// (no named barriers here, so every warp may leave by itself).
template <int D>
__device__ void widen(const PrefillParams &p, Smem<D> &sm, const DevCtx &ctx) {
    constexpr int UR = D / 16;             // 16-code units a row
    constexpr int PER = TILE * UR / 128;   // units a thread, a tile
    const int tid = threadIdx.x - 128, lane = tid & 31;
    volatile int *abort = &sm.abort;
    // unit i * 128 + tid of a tile: the row moves on by a multiple of 8, so its
    // place in the swizzle stays. The second column half's lanes store their two
    // 16-byte units in the other order, so that the halves' units fall into
    // different banks.
    const int r0 = tid / UR, un = tid % UR;
    const bool sw = D == 128 && un >= 4;
    const uint32_t half = (uint32_t)(un >> 2) * Smem<D>::HALF, first = 2 * (un & 3) + (sw ? 1 : 0);
    const uint32_t at0 = half + sw128_offset(r0, first), at1 = half + sw128_offset(r0, first ^ 1);
    int t = 0;  // tiles
    for (int i = 0;; ++i) {
        if (!sm.units.wait(i, ctx, abort)) return;
        Unit<ROWS> &u = sm.units.u[i % UNITS];
        if (u.begin == u.end) return;
        for (int j = u.begin; j < u.end; ++j, ++t) {
            const int b = t & 1, use = t >> 1, st = t % STAGES, ss = t % SRING;
            const int kpos0 = (u.t_first + j) * TILE;
            const bool edge = kpos0 < u.ilo || kpos0 + TILE - 1 > u.ihi;
            if (!bar_wait(smem_u32(&sm.v8_full[st]), (t / STAGES) & 1, ctx, abort)) return;
            if (!bar_wait(smem_u32(&sm.sc_full[ss]), (t / SRING) & 1, ctx, abort)) return;
            uint4 *src = reinterpret_cast<uint4 *>(sm.v[st]) + tid;
            // values that no row sees may hold anything, NaN codes too, and the MMA
            // multiplies them by 0; a zero scale drops the values
            if (edge || sm.zero[ss]) {
#pragma unroll 1
                for (int i = 0; i < PER; ++i) {
                    const int r = r0 + i * (128 / UR), key = kpos0 + r;
                    uint4 x = src[i * 128];
                    const bool hidden = key < u.lo || key > u.hi;
                    if (hidden || sm.sc[ss][r >> p.page_shift].w == 0.f) {
                        // (NaN times a scale of 0 is NaN)
                        if (!hidden && without_nan(x)) u.nan_values = u.nan_zero = 1;
                        src[i * 128] = make_uint4(0, 0, 0, 0);
                    } else if ((key < u.ilo || key > u.ihi) && without_nan(x)) {
                        src[i * 128] = x;
                        u.nan_values = 1;
                    }
                }
            }
            if (use >= 1 && !bar_wait(smem_u32(&sm.v_empty[b]), (use - 1) & 1, ctx, abort)) return;
            constexpr int B = 4;  // units in registers at a time
#pragma unroll 1
            for (int i0 = 0; i0 < PER; i0 += B) {
                uint4 x[B];
#pragma unroll
                for (int i = 0; i < B; ++i) x[i] = src[(i0 + i) * 128];
                uint8_t *dst = sm.v16[b] + i0 * (128 / UR) * 128;
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const uint4 a =
                        make_uint4(e4m3x2_to_f16x2(x[i].x), e4m3x2_to_f16x2(x[i].x >> 16),
                                   e4m3x2_to_f16x2(x[i].y), e4m3x2_to_f16x2(x[i].y >> 16));
                    const uint4 c =
                        make_uint4(e4m3x2_to_f16x2(x[i].z), e4m3x2_to_f16x2(x[i].z >> 16),
                                   e4m3x2_to_f16x2(x[i].w), e4m3x2_to_f16x2(x[i].w >> 16));
                    uint8_t *row = dst + i * (128 / UR) * 128;
                    *reinterpret_cast<uint4 *>(row + at0) = sw ? c : a;
                    *reinterpret_cast<uint4 *>(row + at1) = sw ? a : c;
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(&sm.v_full[b]));
            mbar_arrive(smem_u32(&sm.v8_empty[st]));
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.sc_empty[ss]));
        }
        if (lane == 0) sm.units.release(i);
    }
}

// S of one half: S of step x goes to buffer x & 1, when P V of step x - 2 has read its P.
template <int D>
__device__ void issue_s(Smem<D> &sm, uint32_t tmem, int half, const DevCtx &ctx) {
    constexpr uint32_t IDESC = idesc_e4m3_f32(128, SUB, 0, 0);
    volatile int *abort = &sm.abort;
    if (ctx.stall) bar_wait(smem_u32(&sm.drain[half]), 0, ctx, abort);  // test hook: runs out
    const uint64_t dq = desc_rows<D>(smem_u32(sm.q[half][0])), dk = desc_rows<D>(smem_u32(sm.k[0]));
    const uint32_t cols = tmem + (uint32_t)half * HALF_COLS;
    auto wait = [&](uint64_t &bar, int phase) {
        return bar_wait(smem_u32(&bar), phase & 1, ctx, abort);
    };
    int x = 0, t = 0, ec = 0;  // steps, tiles, units
    bool ok = true;
    for (int i = 0; ok; ++i) {
        if (!(ok = sm.units.wait(i, ctx, abort))) break;
        const Unit<ROWS> &u = sm.units.u[i % UNITS];
        const int n = u.end - u.begin, s0 = u.sub_begin() - 2 * u.begin,
                  s1 = u.sub_end() - 2 * u.begin;
        const bool none = half && u.nrows <= 128;
        sm.units.release(i);
        if (n == 0) break;
        if (none) {  // no rows in this half: its share in freeing the stages
            for (int j = 0; j < n && ok; ++j, ++t) {
                ok = wait(sm.k_full[t % STAGES], t / STAGES);
                mbar_arrive(smem_u32(&sm.k_empty[t % STAGES]));
            }
            continue;
        }
        ok = wait(sm.q_full[half], ec);
#pragma unroll 1
        for (int k = s0; k < s1 && ok; ++k, ++x) {
            const int st = t % STAGES, b = x & 1;
            // The tile's scales too, so that who finds S finds them: a commit orders the MMAs
            // alone, so this thread arrives on S's barrier for what it has seen itself.
            if (k == s0 || !(k & 1))
                ok = wait(sm.k_full[st], t / STAGES) && wait(sm.sc_full[t % SRING], t / SRING);
            if (x >= 2) ok = ok && wait(sm.pv_done[half][b], (x >> 1) - 1);
            if (!ok) break;
            mbar_arrive(smem_u32(&sm.s_full[half][b]));
            tc_fence_after();
            const uint64_t kd = dk + (uint64_t)(st * (TILE * D >> 4) + (k & 1) * (SUB * D >> 4));
#pragma unroll
            for (int kk = 0; kk < 2 * D / 32; ++kk) {  // hi, then lo
                const int lo = kk / (D / 32), c = kk % (D / 32);
                mma_f8(cols + (uint32_t)(b * SUB), dq + (uint64_t)(lo * (128 * D >> 4) + 2 * c),
                       kd + (uint64_t)(2 * c), IDESC, kk > 0);
            }
            tc_commit(smem_u32(&sm.s_full[half][b]));
            if ((k & 1) || k == s1 - 1) {
                tc_commit(smem_u32(&sm.k_empty[st]));
                ++t;
            }
        }
        ++ec;
    }
    tc_commit(smem_u32(&sm.drain[half]));  // every MMA is done before TMEM goes
    int zero = 0;
    bar_wait(smem_u32(&sm.drain[half]), 0, ctx, &zero);
}

// P V of one half.
template <int D>
__device__ void issue_pv(Smem<D> &sm, uint32_t tmem, int half, const DevCtx &ctx) {
    constexpr uint32_t IDESC = idesc_f16_f32(128, D, 1);
    constexpr uint32_t HALF = Smem<D>::HALF, BYTES = Smem<D>::NH * HALF;
    volatile int *abort = &sm.abort;
    const uint64_t dv = smem_desc_sw128(smem_u32(sm.v16[0]), HALF, 1024u);
    const uint32_t cols = tmem + (uint32_t)half * HALF_COLS;
    auto wait = [&](uint64_t &bar, int phase) {
        return bar_wait(smem_u32(&bar), phase & 1, ctx, abort);
    };
    int x = 0, t = 0, ec = 0;  // steps, tiles, units
    bool ok = true;
    for (int i = 0; ok; ++i) {
        if (!(ok = sm.units.wait(i, ctx, abort))) break;
        const Unit<ROWS> &u = sm.units.u[i % UNITS];
        const int n = u.end - u.begin, s0 = u.sub_begin() - 2 * u.begin,
                  s1 = u.sub_end() - 2 * u.begin;
        const bool none = half && u.nrows <= 128;
        sm.units.release(i);
        if (n == 0) break;
        if (none) {
            for (int j = 0; j < n && ok; ++j, ++t) {
                ok = wait(sm.v_full[t & 1], t >> 1);
                mbar_arrive(smem_u32(&sm.v_empty[t & 1]));
            }
            continue;
        }
#pragma unroll 1
        for (int k = s0; k < s1; ++k, ++x) {
            const int vb = t & 1, b = x & 1;
            if (k == s0 || !(k & 1)) ok = wait(sm.v_full[vb], t >> 1);
            // the first P V overwrites the O that the last unit's epilogue reads
            if (k == s0 && ec >= 1) ok = ok && wait(sm.o_empty[half], ec - 1);
            ok = ok && wait(sm.p_full[half][b], x >> 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vd =
                dv + (uint64_t)(vb * (BYTES >> 4) + (k & 1) * (SUB / 16 * 2048u >> 4));
            const uint32_t pt = cols + (uint32_t)(b * SUB);
#pragma unroll
            for (int kk = 0; kk < SUB / 16; ++kk)
                tc_mma_f16_ts(cols + O_COL, pt + 8u * kk,
                              vd + (uint64_t)(kk * (2048u >> 4)), IDESC, kk > 0 || k > s0);
            tc_commit(smem_u32(&sm.pv_done[half][b]));
            if ((k & 1) || k == s1 - 1) {
                tc_commit(smem_u32(&sm.v_empty[vb]));
                ++t;
            }
        }
        // (the arrival: what the widening warps noted of the unit's values)
        if (ok) mbar_arrive(smem_u32(&sm.o_full[half]));
        tc_commit(smem_u32(&sm.o_full[half]));
        ++ec;
    }
    tc_commit(smem_u32(&sm.drain[2 + half]));
    int zero = 0;
    bar_wait(smem_u32(&sm.drain[2 + half]), 0, ctx, &zero);
}

// The k with the largest |q| 2^k in [128, 256), from that |q|'s bf16 bits.
__device__ __forceinline__ int up_shift(uint32_t top) {
    return top ? max(-120, min(7 - ((int)(top >> 7) - 127), 120)) : 0;
}

// A unit whose row sums are taken apart (far_scale), for a thread's row r, from its Q on: m as
// in the fast steps, but at its maximum in every step; l in terms of n, the maximum of the
// logits alone. A key at a time, a column at a time: such calls are rare, and what the
// fast loop carries along for them costs every call. (Beside that loop a unit's far form costs
// little: chunk below 847 us, as a function that is called 862.) Returns false if a
// wait gave up.
template <int D>
__device__ __forceinline__ bool far_unit(const PrefillParams &p, Smem<D> &sm, const Unit<ROWS> &u,
                                      uint32_t tmem, int half, int t, int done, int units, float qf,
                                      float l, const DevCtx &ctx) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = half * 128 + (warp & 3) * 32 + lane;
    const int tok = p.plan.token(u.row0 + r), head = u.h * p.plan.G + u.row0 + r - tok * p.plan.G;
    const int pos = u.s.len - u.s.n + tok;
    const int first = p.plan.wl < 0 ? 0 : max(0, pos - p.plan.wl);
    const int last = p.plan.causal ? pos : u.s.len - 1;
    const bool in = r < u.nrows;
    const float sink = p.sinks && in ? sink_log2(__ldg(p.sinks + head)) : 0.f;
    auto wait = [&](uint64_t &bar, int phase) {
        return __all_sync(0xffffffffu, bar_wait(smem_u32(&bar), phase & 1, ctx, &sm.abort));
    };
    float m = NOTHING, n = NOTHING;
    const int s0 = u.sub_begin(), s1 = u.sub_end();
    int kpos0 = u.t_first * TILE + s0 * SUB;
#pragma unroll 1
    for (int k = s0; k < s1; ++k, ++done, t += !(k & 1), kpos0 += SUB) {
        const int ss = t % SRING, b = done & 1;
        const uint32_t s_tmem = tmem + (uint32_t)(b * SUB);
        if (!wait(sm.s_full[half][b], done >> 1)) return false;
        tc_fence_after();
        // the logit of key e, and its page's log2 scale
        auto logit = [&](int e, float &lv) {
            const float4 s = sm.sc[ss][((k & 1) * SUB + e) >> p.page_shift];
            const int key = kpos0 + e;
            float y = tmem_ld1(s_tmem + (uint32_t)e) * (s.x * qf);
            if (p.sink_mode == 1 && key == 0) y += sink;
            lv = s.y;
            return key < first || key > last || s.y == -INFINITY ? -INFINITY : y;
        };
        float top = m;
#pragma unroll 1
        for (int e = 0; e < SUB; ++e) {
            float lv;
            const float y = logit(e, lv), nn = fmaxf(n, y);
            l = fmaf(l, ex2(n - nn), ex2(y - nn + BASE));
            n = nn;
            top = fmaxf(top, y + lv);
        }
        if (__any_sync(0xffffffffu, top > m) && k > s0) {
            if (!wait(sm.pv_done[half][b ^ 1], (done - 1) >> 1)) return false;
            tc_fence_after();
            const float alpha = ex2(m - top);
#pragma unroll 1
            for (int c = 0; c < D; ++c)
                tmem_st1(tmem + O_COL + (uint32_t)c, tmem_ld1(tmem + O_COL + (uint32_t)c) * alpha);
        }
        m = top;
#pragma unroll 1
        for (int e = 0; e < SUB; e += 2) {  // P over S's first columns, behind what is read
            float lv0, lv1;
            const float y0 = logit(e, lv0), y1 = logit(e + 1, lv1);
            tmem_st1(s_tmem + (uint32_t)(e >> 1),
                     __uint_as_float(pack_f16x2(ex2(y0 + lv0 - m + BASE), ex2(y1 + lv1 - m + BASE))));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&sm.p_full[half][b]));
            if ((k & 1) || k == s1 - 1) mbar_arrive(smem_u32(&sm.sc_empty[ss]));
        }
    }
    if (!wait(sm.o_full[half], units)) return false;
    tc_fence_after();
    const bool part = u.begin > 0 || u.end < u.ntiles;
    float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
    const size_t slot = ((size_t)blockIdx.x * 2 + (u.begin > 0 ? 0 : 1)) * ROWS + r;
    float *prow = reinterpret_cast<float *>(p.ws + plan_rows_offset(ROWS)) + slot * D;
    const size_t orow = (size_t)(u.s.t0 + tok) * p.H + head;
    if (in && part) {
        part_sums(p.ws)[slot] = make_float2(n, l * (1.f / (1 << (int)BASE)));
    } else if (in) {
        float lse2 = l == 0.f ? -INFINITY : n - BASE + __log2f(l);
        if (p.sink_mode == 2) with_null_sink(sink, lse2, inv);
        if (p.lse) p.lse[orow] = lse2 * LN2;
    }
    // 2^(m - n) is a value scale's size: in two steps, as it may leave fp32's range
    const float root = ex2(0.5f * (m - n));
    inv *= root;
    uint32_t nan[D / 32] = {};  // columns that are NaN
    if ((u.nan_values || u.nan_zero) && in)
        each_partial_key<D>(p, u, first, last, [&](int, const uint8_t *codes) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
#pragma unroll 1
                for (int e = 0; e < 32; ++e)
                    nan[w] |= (__ldg(codes + 32 * w + e) & 0x7f) == 0x7f ? 1u << e : 0u;
        });
#pragma unroll 1
    for (int c = 0; c < D; ++c) {
        float o = tmem_ld1(tmem + O_COL + (uint32_t)c) * root * inv;
        uint32_t word = nan[0];
#pragma unroll
        for (int w = 1; w < D / 32; ++w) word = c >> 5 == w ? nan[w] : word;
        if (word >> (c & 31) & 1) o = NAN;
        if (in && part) prow[c] = o;
        else if (in) p.o[orow * D + c] = __float2bfloat16_rn(o);
        __syncwarp();
    }
    tc_fence_before();
    return true;
}

template <int D, int CW>  // CW: columns that share a page's scales (16 or 32)
__device__ void softmax(const PrefillParams &p, Smem<D> &sm, uint32_t tmem_base,
                        const DevCtx &ctx) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = (warp - SOFTMAX) >> 2, quarter = warp & 3;
    const int r = half * 128 + quarter * 32 + lane;  // row of the unit
    const uint32_t tmem =
        tmem_base + (uint32_t)half * HALF_COLS + ((uint32_t)(quarter * 32) << 16);
    volatile int *abort = &sm.abort;
    auto wait = [&](uint64_t &bar, int phase) {
        return __all_sync(0xffffffffu, bar_wait(smem_u32(&bar), phase & 1, ctx, abort));
    };
    int t0 = 0, done = 0, units = 0;  // CTA's tiles; this half's steps and units
    for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, sm.units.wait(i, ctx, abort))) return;
        const Unit<ROWS> &u = sm.units.u[i % UNITS];
        const int n = u.end - u.begin, G = p.plan.G;
        if (n == 0) return;
        if (half && u.nrows <= 128) {  // nothing in this half: keep the scales' ring going
            for (int j = 0; j < n; ++j) {
                const int ss = (t0 + j) % SRING;
                if (!wait(sm.sc_full[ss], (t0 + j) / SRING)) return;
                if (lane == 0) mbar_arrive(smem_u32(&sm.sc_empty[ss]));
            }
            t0 += n;
            __syncwarp();
            if (lane == 0) sm.units.release(i);
            continue;
        }
        // What is needed now and then is computed now and then: a register that the
        // steps do not have spills, and there is next to no L1 beside the tiles.
        auto token = [&]() { return p.plan.token(u.row0 + r); };
        auto in_unit = [&]() { return r < u.nrows; };
        // the row's keys; a row past the unit's last sees what it likes (not written)
        auto last_key = [&]() {
            return p.plan.causal ? u.s.len - u.s.n + token() : u.s.len - 1;
        };
        auto first_key = [&]() {
            return p.plan.wl < 0 ? 0 : max(0, u.s.len - u.s.n + token() - p.plan.wl);
        };
        auto sink = [&]() {
            return p.sinks && in_unit()
                       ? sink_log2(__ldg(p.sinks + u.h * G + u.row0 + r - token() * G))
                       : 0.f;
        };
        // ---- Q of the warp's 32 rows, a power of two times each, split. The half's Q tile
        // is free: this warp has seen the last S that reads it. CH lanes a row, 16 bytes
        // each, so that a load is whole lines (a row a thread: 4000 cycles more a unit)
        float qf, l;
        {
            constexpr int CH = D / 8, RL = 32 / CH, ITEMS = 32 / RL, B = 8;  // RL: rows a load
            const int c = lane % CH, first = r - lane + lane / CH;
            // (in registers: a store to the tile would have them read again)
            const int row0 = u.row0, rows = u.nrows, h0 = u.h * G;
            const __nv_bfloat16 *src = p.q + (size_t)u.s.t0 * p.q_stride + 8 * c;
            uint32_t mine = 0;  // of the thread's own row: its largest |q|, as bf16 bits
#pragma unroll 1
            for (int i0 = 0; i0 < ITEMS; i0 += B) {
                uint4 x[B];
                uint32_t top[B];
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const int rr = first + (i0 + i) * RL, row = row0 + rr, tok = p.plan.token(row);
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (rr < rows)
                        x[i] = __ldg(reinterpret_cast<const uint4 *>(
                            src + (size_t)tok * p.q_stride + (size_t)(h0 + row - tok * G) * D));
                }
#pragma unroll
                for (int i = 0; i < B; ++i)
                    top[i] = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                      __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
#pragma unroll
                for (int o = 1; o < CH; o <<= 1)
#pragma unroll
                    for (int i = 0; i < B; ++i)
                        top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    top[i] = max(top[i] >> 16, top[i] & 0xffffu);
                    const uint32_t of_row = __shfl_sync(0xffffffffu, top[i], lane % RL * CH);
                    if (lane / RL == i0 + i) mine = of_row;
                }
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const int rr = first + (i0 + i) * RL;
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    const float up = __uint_as_float((uint32_t)(127 + up_shift(top[i])) << 23);
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // by way of f16, which holds a scaled bf16 down to 2^-24
                        const uint32_t ab = pack_f16x2(__uint_as_float(w[e] << 16) * up,
                                                       __uint_as_float(w[e] & 0xffff0000u) * up);
                        const uint32_t h = e4m3x2_of_f16x2(ab);
                        const uint32_t l2 =
                            e4m3x2_of_f16x2(difference_f16x2(ab, e4m3x2_to_f16x2(h)));
                        hi[e >> 1] = e & 1 ? hi[e >> 1] | h << 16 : h;
                        lo[e >> 1] = e & 1 ? lo[e >> 1] | l2 << 16 : l2;
                    }
                    const uint32_t at = sw_offset<D>(rr & 127, c >> 1) + 8 * (c & 1);
                    *reinterpret_cast<uint2 *>(sm.q[half][0] + at) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(sm.q[half][1] + at) = make_uint2(lo[0], lo[1]);
                }
            }
            l = mine >= 0x7f80u ? NAN : 0.f;  // an inf or a NaN spoils the row
            qf = p.scale_l2 * __uint_as_float((uint32_t)(127 - up_shift(mine)) << 23);
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(&sm.q_full[half]));
        }
        // (the unit's scales are looked at before its first tile's are handed on)
        if (!wait(sm.sc_full[t0 % SRING], t0 / SRING)) return;
        if (__builtin_expect(u.far, 0)) {
            if (!far_unit<D>(p, sm, u, tmem, half, t0, done, units, qf, l, ctx)) return;
            done += u.sub_end() - u.sub_begin();
            t0 += n;
            ++units;
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm.o_empty[half]));
                sm.units.release(i);
            }
            continue;
        }
        float m = NOTHING;
        bool far = false;  // some row's m is so large that fp32 must subtract it exactly
        bool fresh = true;  // some row has seen no key yet
        const int s0 = u.sub_begin(), s1 = u.sub_end();
        int t = t0, kpos0 = u.t_first * TILE + s0 * SUB;  // tile, and the step's first key
#pragma unroll 1
        for (int k = s0; k < s1; ++k, ++done, t += !(k & 1), kpos0 += SUB) {
            const int ss = t % SRING, in_tile = (k & 1) * SUB;
            const uint32_t s_tmem = tmem + (uint32_t)((done & 1) * SUB);
            const bool mask = kpos0 < u.ilo || kpos0 + SUB - 1 > u.ihi;
            const bool key0 = p.sink_mode == 1 && kpos0 == 0;
            if (!wait(sm.s_full[half][done & 1], done >> 1)) return;
            tc_fence_after();
            // the pages' scales as S and x take them: f above 0 (a zero key scale makes
            // it 0), since a masked S is -inf
            constexpr int NW = SUB / CW;
            float sx[NW], sy[NW], sz[NW];
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 s = sm.sc[ss][(in_tile + w * CW) >> p.page_shift];
                sx[w] = fmaxf(s.x * qf, FLT_MIN), sy[w] = s.y, sz[w] = s.z;
            }
            uint32_t xs[2][32];
            auto load = [&]() {
                tmem_ld32(s_tmem, xs[0]);
                tmem_ld32(s_tmem + 32u, xs[1]);
                tc_wait_ld();
                if (mask) {
                    // bit e: the row sees key e
                    const int a = max(0, first_key() - kpos0), z = min(SUB - 1, last_key() - kpos0);
                    const uint64_t seen = a > z ? 0 : (~0ull >> (SUB - 1 - z)) & (~0ull << a);
#pragma unroll
                    for (int e = 0; e < SUB; ++e)
                        hide_unless(xs[e >> 5][e & 31],
                                    (uint32_t)(seen >> (e & 32)) & (1u << (e & 31)));
                }
            };
            // m from the row's 64 keys, and O and l in its terms
            auto move = [&]() -> bool {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int e = w * CW; e < w * CW + CW; e += 2)
                        mx = max3(mx, e == 0 && key0 ? -INFINITY
                                                     : __uint_as_float(xs[e >> 5][e & 31]),
                                  __uint_as_float(xs[e >> 5][(e & 31) + 1]));
                    top = fmaxf(top, fmaf(mx, sx[w], sy[w]));
                    if (w == 0 && key0)
                        top = fmaxf(top, fmaf(__uint_as_float(xs[0][0]), sx[0], sy[0]) + sink());
                }
                const float mn = fmaxf(m, top), alpha = ex2(m - mn);
                m = mn;
                l *= alpha;
                fresh = __any_sync(0xffffffffu, m == NOTHING);
                far = __any_sync(0xffffffffu, m != NOTHING && fabsf(m) > FAR);
                if (k > s0) {
                    if (!wait(sm.pv_done[half][(done - 1) & 1], (done - 1) >> 1)) return false;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tmem + O_COL + 32u * c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(tmem + O_COL + 32u * c, o);
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
                const float base = m == NOTHING ? BASE : BASE - m;
                float raw = 0.f;
                bool bias = key0;
                sum = 0.f;
                float fx[NW], off[NW];
#pragma unroll
                for (int w = 0; w < NW; ++w) fx[w] = sx[w], off[w] = sy[w] + base;
                if (far) {  // x - m in two roundings, as move() has them: never above 0 there
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
#pragma unroll
                        for (int e = w * CW; e < w * CW + CW; ++e) {
                            float x = fmaf(__uint_as_float(xs[e >> 5][e & 31]), sx[w], sy[w]);
                            if (e == 0 && bias) x += sink();
                            xs[e >> 5][e & 31] = __float_as_uint(x - m);
                        }
                        fx[w] = 1.f, off[w] = BASE;
                    }
                    bias = false;
                }
#pragma unroll
                for (int w = 0; w < SUB; w += CW) {
                    const uint64_t f2 = f2_pack(fx[w / CW], fx[w / CW]);
                    const uint64_t off2 = f2_pack(off[w / CW], off[w / CW]);
                    uint64_t part = f2_pack(0.f, 0.f);
#pragma unroll
                    for (int e = w; e < w + CW; e += 2) {
                        float a, b;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(xs[e >> 5][e & 31]),
                                                 __uint_as_float(xs[e >> 5][(e & 31) + 1])),
                                         f2, off2),
                                  a, b);
                        if (e == 0 && bias) a += sink();
                        a = ex2(a);
                        b = ex2(b);
                        part = f2_add(part, f2_pack(a, b));
                        pw[e >> 1] = pack_f16x2(a, b);
                    }
                    float a, b;
                    f2_unpack(part, a, b);
                    raw += a + b;
                    sum = fmaf(a + b, sz[w / CW], sum);
                }
                // no value is above the sum, so below the limit none has left f16's range;
                // and after a move none is above 2^(BASE + 1/4), so there is no third pass
                moves = pass == 0 && __any_sync(0xffffffffu, raw > SUM_LIMIT);
                if (!moves) break;
            }
            l += sum;
            tmem_st32(s_tmem, pw);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm.p_full[half][done & 1]));
                if ((k & 1) || k == s1 - 1) mbar_arrive(smem_u32(&sm.sc_empty[ss]));
            }
        }
        t0 += n;
        // ---- epilogue
        if (!wait(sm.o_full[half], units)) return;
        ++units;
        tc_fence_after();
        const bool part = u.begin > 0 || u.end < u.ntiles;
        float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
        const size_t slot = ((size_t)blockIdx.x * 2 + (u.begin > 0 ? 0 : 1)) * ROWS + r;
        float *prow = reinterpret_cast<float *>(p.ws + plan_rows_offset(ROWS)) + slot * D;
        const bool in = in_unit();
        const int tok = token();
        const size_t orow = (size_t)(u.s.t0 + tok) * p.H + u.h * G + u.row0 + r - tok * G;
        if (in) {
            if (part) {
                part_sums(p.ws)[slot] = make_float2(m, l * (1.f / (1 << (int)BASE)));
            } else {
                float lse2 = l == 0.f ? -INFINITY : m - BASE + __log2f(l);
                if (p.sink_mode == 2) with_null_sink(sink(), lse2, inv);
                if (p.lse) p.lse[orow] = lse2 * LN2;
            }
        }
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tmem + O_COL + 32u * c, o);
            tc_wait_ld();
            if (u.nan_values && in) {
                uint32_t cols = 0;  // columns that are NaN
                each_partial_key<D>(p, u, first_key(), last_key(), [&](int, const uint8_t *codes) {
                    const uint32_t *at = reinterpret_cast<const uint32_t *>(codes) + 8 * c;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i)  // a bit a code
                        cols |= ((nan_codes(__ldg(at + i)) & 0x08040201u) * 0x01010101u >> 24)
                                << (4 * i);
                });
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (cols >> e & 1) o[e] = 0x7fffffffu;
            }
            if (in && part) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(prow + 32 * c + e) = make_float4(
                        __uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                        __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            } else if (in) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = pack_bf16x2(__uint_as_float(o[e + 2 * i]) * inv,
                                           __uint_as_float(o[e + 2 * i + 1]) * inv);
                    *reinterpret_cast<uint4 *>(p.o + orow * D + 32 * c + e) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            __syncwarp();
        }
        tc_fence_before();
        if (lane == 0) {
            mbar_arrive(smem_u32(&sm.o_empty[half]));
            sm.units.release(i);
        }
    }
}

template <int D, int CW>
__global__ void __launch_bounds__(NTHREADS, 1)
prefill_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               const __grid_constant__ PrefillParams p, const __grid_constant__ DevCtx ctx) {
    extern __shared__ __align__(1024) uint8_t dsmem[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(dsmem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (smem_u32(dsmem) & 1023u) {  // the swizzle is anchored to 1024-byte boundaries
        if (threadIdx.x == 0) record_error(ctx, DEVERR_LAYOUT);
        return;
    }
    if (warp == 2) {  // a lane a barrier: one thread would take longer than the plan
        if (lane < STAGES) {
            mbar_init(smem_u32(&sm.k_full[lane]), 1);
            mbar_init(smem_u32(&sm.k_empty[lane]), 2);  // both halves' MMAs
            mbar_init(smem_u32(&sm.v8_full[lane]), 1);
            mbar_init(smem_u32(&sm.v8_empty[lane]), 128);
        }
        if (lane < 2) {
            mbar_init(smem_u32(&sm.v_full[lane]), 128);
            mbar_init(smem_u32(&sm.v_empty[lane]), 2);
            mbar_init(smem_u32(&sm.drain[lane]), 1);
            mbar_init(smem_u32(&sm.drain[2 + lane]), 1);
            mbar_init(smem_u32(&sm.q_full[lane]), 128);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&sm.s_full[lane][b]), 2);  // the issuer and its MMAs
                mbar_init(smem_u32(&sm.p_full[lane][b]), 4);
                mbar_init(smem_u32(&sm.pv_done[lane][b]), 1);
            }
            mbar_init(smem_u32(&sm.o_full[lane]), 2);
            mbar_init(smem_u32(&sm.o_empty[lane]), 4);
        }
        if (lane < SRING) {
            mbar_init(smem_u32(&sm.sc_full[lane]), 1);
            mbar_init(smem_u32(&sm.sc_empty[lane]), 8 + 4);  // softmax and widening warps
        }
        if (lane == 0) sm.abort = 0;
        sm.units.init(4 + 1 + 4 + 8, lane);  // MMA issuers, scales, widening, softmax
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sm.tmem_base), TMEM_COLS);
        tmem_relinquish();
    }
    plan_start<ROWS>(p.plan, sm.plan, ctx);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // registers: 384 threads x 48 + 256 x 168 = the 640 x 96 of the launch
    if (warp < SOFTMAX) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 0) {
            load_tiles<D>(p, &tk, &tv, sm, ctx);
        } else if (warp == 2) {
            load_scales<D>(p, sm, ctx);
        } else if (warp < 4) {
            if (lane == 0) issue_s<D>(sm, tmem, warp >> 1, ctx);
            __syncwarp();
        } else if (warp < 8) {
            widen<D>(p, sm, ctx);
        } else if (!(warp & 1)) {
            if (lane == 0) issue_pv<D>(sm, tmem, (warp >> 1) & 1, ctx);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        softmax<D, CW>(p, sm, tmem, ctx);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort == TIMED_OUT) record_error(ctx, DEVERR_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int D, int CW>
cudaError_t launch(const PagedArgs &a, const DevInfo &dev, cudaStream_t s) {
    CUtensorMap tk, tv;
    if (!map_cache(&tk, a.k_cache, a,
                   D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
        !map_cache(&tv, a.v_cache, a, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    const size_t smem = sizeof(Smem<D>);
    static_assert(sizeof(Smem<D>) <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = ensure_smem_attr((const void *)prefill_kernel<D, CW>, smem, dev);
    if (e != cudaSuccess) return e;
    const int grid = dev.sm_count < MAX_PIECES ? dev.sm_count : MAX_PIECES;
    const bool split = a.workspace && a.workspace_bytes >= plan_workspace(ROWS, D);
    PrefillParams p{plan_args(a, split, EXTRA), static_cast<const __nv_bfloat16 *>(a.q), a.q_stride,
                    a.v_cache, a.k_scale, a.v_scale, a.page_table, a.H, a.num_pages, a.page,
                    page_shift(a.page), a.max_pages, a.num_pages * a.Hkv * a.page,
                    a.scale * LOG2E, a.sinks, a.sink_mode, static_cast<__nv_bfloat16 *>(a.o),
                    a.lse, static_cast<uint8_t *>(a.workspace)};
    if (verbose())
        fprintf(stderr, "sattn: paged prefill_kernel<%d, %d> grid=%d smem=%zu split=%d\n", D, CW,
                grid, smem, (int)split);
    prefill_kernel<D, CW><<<grid, NTHREADS, smem, s>>>(tk, tv, p, make_ctx(dev));
    e = cudaGetLastError();
    if (e != cudaSuccess || !split) return e;
    return launch_paged_join(a, ROWS, grid, s);
}

}  // namespace

size_t paged_prefill_workspace(int d) { return plan_workspace(ROWS, d); }

cudaError_t launch_paged_prefill(const PagedArgs &a, const DevInfo &dev, cudaStream_t s) {
    if (a.d == 64) return a.page == 16 ? launch<64, 16>(a, dev, s) : launch<64, 32>(a, dev, s);
    return a.page == 16 ? launch<128, 16>(a, dev, s) : launch<128, 32>(a, dev, s);
}

}  // namespace sattn
