// Cross attention to encoder states on the tensor cores (tcgen05), bf16.
//
// Query rows are tokens times the heads of a KV group, token-major, fetched as boxes of G heads and
// floor(128 / G) tokens, so that any group size fills the 128 rows of an MMA. The states
// come as tiles of 128 keys, K and V in turn through one ring of shared memory.
//   S = Q K^T   [128 x 128] into TMEM
//   P = 2^(S scale log2(e) - m), bf16, 64 keys at a time over the columns of S that
//       have been read; l += its sum, unrounded
//   O += P V    P from TMEM, 64 keys at a time: while the second half of P is computed the
//       product with the first runs. (bf16 because V is: an MMA's operands have one type. It takes
//       a bf16 output's error from 1.65e-3 to 2.2e-3 of its size.)
// m is the maximum of a row's first 64 keys and stays unless 64 keys' P sum up to more than
// 2^15: P is computed on trust in one pass over S that looks for no maximum, and where the
// sum says that this was wrong m moves, O is rescaled and the pass is repeated.
// V rows behind the sequence's last state are zeroed in shared memory (the MMA multiplies them
// by P = 0, and they may be NaN).
//
// One persistent CTA per SM over an equal piece of the line of units (states_plan.cuh), two
// halves that work in turn, so that one's softmax runs beside the other's products:
//   many rows   a unit is 256 rows; both halves use every tile
//   FEW         a unit is FEW (32 or 64) rows at most; the halves take every other tile, and
//               the rows stand in the MMA's 128 more than once, so that each warp of a
//               half takes some of a step's keys: its P is 0 for the others, and the O of its lanes
//               a sum over its own keys. Every warp runs a softmax of its own (eight in
//               all, or four with 64 rows); they are joined at a unit's end. What bounds is the
//               memory, and a tile's chain of products and exponentials, a row a thread,
//               takes longer than its load.
// The pieces of a unit that is cut between CTAs are joined by a second launch.
// Roles: warp 0 units and TMA; 1, 3 S of the halves; 4, 5 P V; 2 the last V tile's rows;
// 6, 7 (FEW) the sums over a unit's streams; 8-11, 12-15 softmax and epilogue, a thread a row.
//
// Bound, many rows: the chain from S over exponentials and the store of P to the next product, of
// two softmax warps a scheduler. 4097 queries over 16411 states, 32 heads on 8, take 3240 cycles a
// tile of 128 keys (256 rows) with d = 128 and 3110 with d = 64, where operand reads and products
// halve and no unit of the SM is above 46 % busy (the MMA unit with its operand reads 46, its
// products 34, exponentials 34, issue 44; counters at 2048 over 8192). With d = 128 that unit is
// at 74 %: S of 64 keys takes 48 cycles an MMA where 128 would take 32 for as many (Q is read again
// for each), 2560 cycles a tile with the TMA writes. d = 128: 725 to 740 us, 1.5 PFLOP/s, 0.78 of
// the bf16 peak, and less where the clock falls under the load; d = 64: 663 us. 16 prompts of 17 to 900 queries over 257 to 4100 states: 181 us,
// d = 64 159, of which the join of cut units is 11 and a unit by itself (first maximum, O) 2 tiles'
// time.
// Measured on the way, us for the first with d = 128:
//   MMAs issued by single threads, S of 128 keys in one buffer a half       1016
//     the same by converged warps that elect a lane (states_plan.cuh)        945
//     and the halves made to take turns (P V and the next S of one, then
//     of the other; else both wait for products at the same time)            780
//   S of 64 keys in two buffers, no turns                                    736
//   P stored before its sum is looked at                                     725
// Bound, few rows: the memory, 7.2 TB/s while tiles stream; 64 single tokens over 257 to 6404
// states 150 us, 6.3 TB/s, with d = 64 83 us, 5.7 TB/s; a unit costs 2200 cycles by itself. One
// token over 1601 states 14.3 us, where a trivial kernel takes 4: the plan (3000 cycles of dependent
// loads and divisions), the first tile, one step, the join, in a row. (Joined by the last
// piece to arrive, its two warps that add up the streams, and without the launch: the same for
// this one token; 8 tokens of 32 heads over 1500 states 57 us, with the launch 21; 60 rows of one
// KV head over 16000 states 333 and 37.)
#include <math.h>
#include <stdio.h>

#include "paged_plan.cuh"
#include "states_plan.cuh"

namespace sattn {
namespace {

constexpr int NTHREADS = 512;
constexpr int SOFTMAX = 8;   // first softmax warp
constexpr int UNITS = 4;     // units handed on ahead
constexpr int ADDERS = 2;    // warps that add up a unit's streams (FEW)
// What a step costs; with one half's rows alone 0.63 of it. A unit by itself: 2 steps, 1 or
// 3 in the FEW form (by cycles of CTAs with other shares of each).
constexpr int COST = 8, LESS = 5;
constexpr int CHUNK = 64;    // keys whose P is handed on at a time
constexpr float SUM_LIMIT = 32768.f;  // m moves when 64 keys' P sum up to more
constexpr float FAR = 1 << 20;  // m up to which x - m may be taken in one rounding
// (d = 64 leaves room for a third buffer of S a half: no gain where it was tried)
constexpr uint32_t TMEM_COLS = 512, HALF_COLS = 256, O_COL = 128;

struct CrossParams {
    LineArgs line;
    int H, G, tokens;  // tokens: of a half's rows
    int rows;          // tokens * G
    float scale_l2;
    const float *sinks;
    int sink_mode;
    __nv_bfloat16 *o;
    int o_wide;  // o is on a 32-byte boundary
    float *lse;
    uint8_t *ws;
    uint32_t g_mul, g_shift;

    // row / G for 0 <= row < 2^31 (as PlanArgs::token)
    __device__ __forceinline__ int token(int row) const {
        return (int)((__umulhi(g_mul, (uint32_t)row) + (uint32_t)row) >> g_shift);
    }
};

// A piece's note for the join launch: of the unit that begins in it and goes on behind it, its
// first token, KV head, rows (0: there is none) and parts.
struct JoinNote {
    int t0, h, rows, parts;
};
static_assert(sizeof(JoinNote) <= sizeof(PlanNote), "the notes' part of the workspace");

template <int D> struct alignas(1024) Smem {
    static constexpr int NH = D / 64;                     // 64-column parts of a row
    static constexpr uint32_t PART = 128 * 128;           // 128 rows of 64 bf16
    static constexpr uint32_t TILE_BYTES = NH * PART;
    static constexpr int R = D == 128 ? 5 : 12;           // ring of K and V tiles
    uint8_t q[2][TILE_BYTES];  // (FEW: q[1] takes the warps' O at a unit's end)
    uint8_t kv[R][TILE_BYTES];
    LineStart line;
    LineRing<UNITS> units;
    float2 ml[256];  // FEW: the streams' m and l
    uint64_t full[R], empty[R], raw[R];
    uint64_t q_full, q_empty, meet, out_full, out_empty;
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

template <int D, int FEW>
__device__ void load_tiles(const CrossParams &p, const CUtensorMap *tq,
                                           const CUtensorMap *tk, const CUtensorMap *tv,
                                           Smem<D> &sm, const DevCtx &ctx) {
    using S = Smem<D>;
    if ((threadIdx.x & 31) != 0) return;
    volatile int *abort = &sm.abort;
    LineIter<false> it(p.line, sm.line);
    JoinNote *note = reinterpret_cast<JoinNote *>(p.ws) + blockIdx.x;
    if (p.line.split) *note = JoinNote{};
    int t = 0, index = 0, queries = 0;  // loads into the ring; units; loads of Q
    uint32_t raws = 0, on_raw = 0;      // bit i: raw[i]'s phase; slot i's last load counts there
    bool ok = true;
#pragma unroll 1
    for (; it.live && ok; it.next(p.line, sm.line)) {
        LineUnit u = it.u;
        u.h = p.line.head(u.h);
        ok = sm.units.put(index, u, ctx, abort);
        if (p.line.split && u.begin == 0 && u.end < u.steps)
            *note = JoinNote{u.s.t0 + u.u * p.line.tokens, u.h,
                             min(p.line.tokens, u.s.n - u.u * p.line.tokens) * p.G, u.parts};
        const bool tail = ragged(u);
        auto ask = [&]() {  // for the unit's queries
            if (index >= 1) ok = ok && bar_wait(smem_u32(&sm.q_empty), (index - 1) & 1, ctx, abort);
            if (!ok) return;
            const uint32_t bar = smem_u32(&sm.q_full);
            const int tok = u.s.t0 + u.u * p.line.tokens;
            const bool two = !FEW && u.s.n - u.u * p.line.tokens > p.tokens;
            constexpr int COPIES = FEW ? 128 / FEW : 2;
            mbar_arrive_expect_tx(bar, (FEW ? COPIES : two ? 2 : 1) * S::NH * p.rows * 128);
#pragma unroll
            for (int i = 0; i < COPIES; ++i)
                if (FEW || i == 0 || two)
#pragma unroll
                    for (int c = 0; c < S::NH; ++c)
                        tma_load_3d(smem_u32(sm.q[FEW ? 0 : i]) + c * S::PART + i * FEW * 128, tq, bar,
                                    64 * c, u.h * p.G, tok + (FEW ? 0 : i * p.tokens));
            ++queries;
        };
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
                // Q behind the first K; later ones' behind the first tile, which need not wait for it
                if (j == u.begin && kv == (index > 0)) ask();
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
template <int D, int FEW>
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
template <int D, int FEW>
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

__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
}
// C columns of S, and the C / 2 of P.
template <int C> __device__ __forceinline__ void load_s(uint32_t at, uint32_t (&x)[C]) {
#pragma unroll
    for (int i = 0; i < C / 16; ++i) {
        uint32_t r[16];
        tmem_ld16(at + 16u * i, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[16 * i + e] = r[e];
    }
}
template <> __device__ __forceinline__ void load_s<64>(uint32_t at, uint32_t (&x)[64]) {
    tmem_ld32(at, *reinterpret_cast<uint32_t (*)[32]>(&x[0]));
    tmem_ld32(at + 32u, *reinterpret_cast<uint32_t (*)[32]>(&x[32]));
}
template <int C> __device__ __forceinline__ void store_p(uint32_t at, const uint32_t (&w)[C / 2]) {
#pragma unroll
    for (int i = 0; i < C / 16; ++i) tmem_st8(at + 8u * i, w + 8 * i);
}
template <> __device__ __forceinline__ void store_p<64>(uint32_t at, const uint32_t (&w)[32]) {
    tmem_st32(at, w);
}

// Eight words to a 32-byte boundary, a whole sector: rows are written a thread each, and
// halves of sectors cost L2 a pass each.
__device__ __forceinline__ void store32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// A row's running softmax over its columns of S, C at a time.
struct Row {
    float m, l;
    bool far;    // some row's m is so large that fp32 must subtract it exactly
    bool fresh;  // some row has seen no key yet
};

// One step: P of the C columns x, packed, to store(), and their sum into l. `there`: how many of the
// columns are keys; key0: the first is the sequence's first, with a biased logit. rescale(alpha)
// is called (by whole warps) where m moves and O with it; returns false if that gave up.
template <int C, typename F, typename G>
__device__ __forceinline__ bool weigh(Row &row, uint32_t (&x)[C], float sx, int there, bool key0,
                                      float sink, F rescale, G store) {
    if (there < C) {
#pragma unroll
        for (int e = 0; e < C; ++e) hide_unless(x[e], e < there);
    }
    bool moves = row.fresh;
    float sum;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        // the first pass's P has landed before the second's goes to the same columns: nothing
        // else orders two stores
        if (pass > 0) tc_wait_st();
        if (moves) {  // m from these columns, and O and l in its terms
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < C; e += 2)
                mx = max3(mx, e == 0 && key0 ? -INFINITY : __uint_as_float(x[e]),
                          __uint_as_float(x[e + 1]));
            float top = __fmul_rn(mx, sx);
            if (key0) top = fmaxf(top, __fadd_rn(__fmul_rn(__uint_as_float(x[0]), sx), sink));
            const float mn = fmaxf(row.m, top), alpha = ex2(row.m - mn);
            row.m = mn;
            row.l *= alpha;
            row.fresh = __any_sync(0xffffffffu, row.m == NOTHING);
            row.far = __any_sync(0xffffffffu, row.m != NOTHING && fabsf(row.m) > FAR);
            if (!rescale(alpha)) return false;
        }
        // P with m as it is, and its sum, which is looked at while P is on its way: x is
        // still here should m have to move
        uint32_t pw[C / 2];
        const float off = row.m == NOTHING ? 0.f : -row.m;
        // x - m in two roundings, as m has them: never above 0 there. (One rounding, an fma, would
        // differ from m by half a step of it, and 2^ of that.)
        if (row.far) {
            sum = 0.f;
#pragma unroll
            for (int e = 0; e < C; e += 2) {
                float a = __fmul_rn(__uint_as_float(x[e]), sx);
                if (e == 0 && key0) a = __fadd_rn(a, sink);
                a = ex2(__fadd_rn(a, off));
                const float b = ex2(__fadd_rn(__fmul_rn(__uint_as_float(x[e + 1]), sx), off));
                sum += a + b;
                pw[e >> 1] = pack_bf16x2(a, b);
            }
            store(pw);
        } else {
            const uint64_t f2 = f2_pack(sx, sx), off2 = f2_pack(off, off);
            uint64_t part[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
            for (int e = 0; e < C; e += 2) {
                float a, b;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), f2, off2),
                          a, b);
                if (e == 0 && key0) a += sink;
                a = ex2(a);
                b = ex2(b);
                part[e >> 1 & 1] = f2_add(part[e >> 1 & 1], f2_pack(a, b));
                pw[e >> 1] = pack_bf16x2(a, b);
            }
            store(pw);
            float a, b;
            f2_unpack(f2_add(part[0], part[1]), a, b);
            sum = a + b;
        }
        // (after a move no value is above 2^(1/4), so there is no third pass)
        moves = pass == 0 && __any_sync(0xffffffffu, sum > SUM_LIMIT);
        if (!moves) break;
    }
    row.l += sum;
    return true;
}

// O of the warp's lanes times alpha.
template <int D> __device__ __forceinline__ void scale_o(uint32_t at, float alpha) {
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(at + 32u * q, o);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
        tmem_st32(at + 32u * q, o);
    }
}

template <int D>
__device__ void softmax_many(const CrossParams &p, Smem<D> &sm, uint32_t tmem_base,
                             const DevCtx &ctx) {
    constexpr int ROWS = 256;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = (warp - SOFTMAX) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the half
    const uint32_t tmem = tmem_base + (uint32_t)half * HALF_COLS + ((uint32_t)(quarter * 32) << 16);
    volatile int *abort = &sm.abort;
    auto wait = [&](uint64_t &bar, int phase) {
        return __all_sync(0xffffffffu, bar_wait(smem_u32(&bar), phase & 1, ctx, abort));
    };
    const int tok = p.token(r);
    int x = 0, units = 0;  // this half's steps and units
    for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, sm.units.wait(i, ctx, abort))) return;
        const LineUnit u = sm.units.u[i % UNITS];
        __syncwarp();
        if (lane == 0) sm.units.release(i);
        if (u.begin == u.end) return;
        const int tokens = u.s.n - u.u * p.line.tokens - half * p.tokens;
        if (tokens <= 0) continue;
        const bool in = r < p.rows && tok < tokens;
        const int head = u.h * p.G + r - tok * p.G;
        const float sink = p.sinks && in ? state_sink(__ldg(p.sinks + head)) : 0.f;
        Row row = {NOTHING, 0.f, false, true};
#pragma unroll 1
        for (int j = u.begin; j < u.end; ++j) {
            const int nch = chunks(u, j);
#pragma unroll 1
            for (int c = 0; c < nch; ++c, ++x) {
                const int kpos0 = j * STATE_KEYS + c * CHUNK;
                const uint32_t s_tmem = tmem + (uint32_t)((x & 1) * CHUNK);
                if (!wait(sm.s_full[half][x & 1], x >> 1)) return;
                tc_fence_after();
                uint32_t xs[CHUNK];
                load_s(s_tmem, xs);
                tc_wait_ld();
                if (!weigh(row, xs, p.scale_l2, u.s.len - kpos0, p.sink_mode == 1 && kpos0 == 0, sink,
                           [&](float alpha) {
                               if (j == u.begin && c == 0) return true;  // no O yet
                               if (!wait(sm.pv_done[half][(x - 1) & 1], (x - 1) >> 1)) return false;
                               tc_fence_after();
                               scale_o<D>(tmem + O_COL, alpha);
                               return true;
                           },
                           [&](const uint32_t(&w)[CHUNK / 2]) { store_p<CHUNK>(s_tmem, w); }))
                    return;
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
        const bool part = u.cut();
        float inv = row.l == 0.f ? 0.f : 1.f / row.l;
        const size_t slot =
            ((size_t)blockIdx.x * 2 + (u.begin > 0 ? 0 : 1)) * ROWS + half * p.rows + r;
        float *prow = reinterpret_cast<float *>(p.ws + plan_rows_offset(ROWS)) + slot * D;
        const size_t orow =
            (size_t)(u.s.t0 + u.u * p.line.tokens + half * p.tokens + tok) * p.H + head;
        if (in && part) {
            part_sums(p.ws)[slot] = make_float2(row.m, row.l);
        } else if (in) {
            float lse2 = row.l == 0.f ? -INFINITY : row.m + log2f(row.l);
            if (p.sink_mode == 2) with_null_sink(sink, lse2, inv);
            if (p.lse) p.lse[orow] = lse2 * LN2;
        }
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tmem + O_COL + 32u * q, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
            if (in && part) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) store32(prow + 32 * q + e, o + e);
            } else if (in) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    w[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                __nv_bfloat16 *at = p.o + orow * D + 32 * q;
                if (p.o_wide) {
                    store32(at, w);
                    store32(at + 16, w + 8);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4 *>(at + 2 * e) =
                            make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                }
            }
            __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.o_empty[half]));
    }
}

template <int D> __device__ __forceinline__ void store_row(__nv_bfloat16 *o, const float *acc, int lane) {
    constexpr int E = D / 32;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) w[e / 2] = pack_bf16x2(acc[e], acc[e + 1]);
    if constexpr (E == 4) *reinterpret_cast<uint2 *>(o + lane * E) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(o + lane * E) = w[0];
}

// Where the streams' O of a unit's rows lie in shared memory: `cap` rows, `width` columns at a time.
template <int D, int FEW> struct Out {
    static constexpr int STREAMS = 256 / FEW;
    int cap, width;
    float4 *buffer;
    __device__ __forceinline__ Out(const CrossParams &p, Smem<D> &sm) {
        cap = p.rows <= 8 ? 8 : p.rows <= 16 ? 16 : FEW;
        width = min(D, (int)Smem<D>::TILE_BYTES / (STREAMS * cap * 4));
        buffer = reinterpret_cast<float4 *>(sm.q[1]);
    }
    // A warp adds up 2^shift pieces of 16 bytes of 32 / 2^shift rows at a time
    __device__ __forceinline__ int shift() const { return 29 - __clz(width); }
    // 16-byte piece c of row r of a stream (neighbouring rows' in different banks)
    __device__ __forceinline__ float4 *piece(int stream, int r, int c) const {
        const int n = width / 4, sw = min(n, 8) - 1;
        return buffer + (stream * cap + r) * n + (c ^ (r & sw));
    }
};

template <int D, int FEW>
__device__ void softmax_few(const CrossParams &p, Smem<D> &sm, uint32_t tmem_base,
                            const DevCtx &ctx) {
    constexpr int COPIES = 128 / FEW, C = CHUNK / COPIES;  // of the rows; a warp's columns of a step
    constexpr int STREAMS = 2 * COPIES;                    // softmaxes of a row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = (warp - SOFTMAX) >> 2, quarter = warp & 3;
    const int copy = quarter * 32 / FEW, r = (quarter * 32 + lane) % FEW, stream = half * COPIES + copy;
    const uint32_t tmem = tmem_base + (uint32_t)half * HALF_COLS + ((uint32_t)(quarter * 32) << 16);
    volatile int *abort = &sm.abort;
    auto wait = [&](uint64_t &bar, int phase) {
        return __all_sync(0xffffffffu, bar_wait(smem_u32(&bar), phase & 1, ctx, abort));
    };
    const Out<D, FEW> out(p, sm);
    const int tok = p.token(r);
    int x = 0, units = 0, meets = 0, outs = 0;  // this half's steps and units; all units, passes
    for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, sm.units.wait(i, ctx, abort))) return;
        const LineUnit u = sm.units.u[i % UNITS];
        __syncwarp();
        if (lane == 0) sm.units.release(i);
        const int n = u.end - u.begin;
        if (n == 0) return;
        const int rows = min(p.tokens, u.s.n - u.u * p.line.tokens) * p.G;  // of the unit
        const int head = u.h * p.G + r - tok * p.G;
        // of key 0, or of the denominator
        const float bias = p.sinks && r < rows ? state_sink(__ldg(p.sinks + head)) : 0.f;
        Row row = {NOTHING, 0.f, false, true};
        const int first = u.begin + half;
#pragma unroll 1
        for (int j = first; j < u.end; j += 2) {
            const int nch = chunks(u, j);
#pragma unroll 1
            for (int c = 0; c < nch; ++c, ++x) {
                const int kpos0 = j * STATE_KEYS + c * CHUNK + copy * C;
                const uint32_t s_tmem = tmem + (uint32_t)((x & 1) * CHUNK);
                if (!wait(sm.s_full[half][x & 1], x >> 1)) return;
                tc_fence_after();
                uint32_t xs[C];
                load_s(s_tmem + (uint32_t)(copy * C), xs);
                tc_wait_ld();
                {  // the other warps' keys
                    const uint32_t zero[C / 2] = {};
#pragma unroll
                    for (int k = 1; k < COPIES; ++k)
                        store_p<C>(s_tmem + (uint32_t)(((copy + k) % COPIES) * (C / 2)), zero);
                }
                if (!weigh(row, xs, p.scale_l2, u.s.len - kpos0, p.sink_mode == 1 && kpos0 == 0, bias,
                           [&](float alpha) {
                               if (j == first && c == 0) return true;  // no O yet
                               if (!wait(sm.pv_done[half][(x - 1) & 1], (x - 1) >> 1)) return false;
                               tc_fence_after();
                               scale_o<D>(tmem + O_COL, alpha);
                               return true;
                           },
                           [&](const uint32_t(&w)[C / 2]) {
                               store_p<C>(s_tmem + (uint32_t)(copy * (C / 2)), w);
                           }))
                    return;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[half][x & 1]));
            }
        }
        // ---- the unit's end. Every thread weighs its stream's O by 2^(m - the row's m) / the
        // row's sum; they go through shared memory to the warps that add them up
        const bool worked = half < n, cut = u.cut();
        if (outs >= 1 && !wait(sm.out_empty, outs - 1)) return;  // the last unit's are added up
        sm.ml[stream * FEW + r] = make_float2(row.m, row.l);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.meet));
        if (!wait(sm.meet, meets++)) return;
        float m = NOTHING, z = 0.f;
        {
            float2 v[STREAMS];
#pragma unroll
            for (int st = 0; st < STREAMS; ++st) {
                v[st] = sm.ml[st * FEW + r];
                m = fmaxf(m, v[st].x);
            }
#pragma unroll
            for (int st = 0; st < STREAMS; ++st) z = fmaf(v[st].y, ex2(v[st].x - m), z);
        }
        // (__log2f and __fdividef for O alone, a bf16: off by 2^-21)
        float lse2 = z == 0.f ? -INFINITY : m + __log2f(z), inv = z == 0.f ? 0.f : __fdividef(1.f, z);
        if (!cut && p.sink_mode == 2) with_null_sink(bias, lse2, inv);
        const float f = ex2(row.m - m) * inv;
        if (stream == 0 && r < rows) {
            if (cut) {
                part_sums(p.ws)[((size_t)blockIdx.x * 2 + (u.begin > 0 ? 0 : 1)) * FEW + r] =
                    make_float2(m, z);
            } else if (p.lse) {
                if (p.sink_mode == 2) {
                    const float top = fmaxf(m, bias);
                    z = fmaf(z, ex2(m - top), ex2(bias - top));
                    m = top;
                }
                p.lse[(size_t)(u.s.t0 + u.u * p.line.tokens + tok) * p.H + head] =
                    z == 0.f ? -INFINITY : (m + log2f(z)) * LN2;
            }
        }
        if (worked) {
            if (!wait(sm.o_full[half], units)) return;
            ++units;
            tc_fence_after();
        }
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += out.width, ++outs) {
            if (c0 > 0 && !wait(sm.out_empty, outs - 1)) return;
#pragma unroll 1
            for (int c = 0; c < out.width; c += 16) {
                uint32_t o[16];
                if (worked) {
                    tmem_ld16(tmem + O_COL + (uint32_t)(c0 + c), o);
                    tc_wait_ld();
                }
                if (r < rows) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *out.piece(stream, r, c / 4 + e) =
                            worked ? make_float4(__uint_as_float(o[4 * e]) * f,
                                                 __uint_as_float(o[4 * e + 1]) * f,
                                                 __uint_as_float(o[4 * e + 2]) * f,
                                                 __uint_as_float(o[4 * e + 3]) * f)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (worked && c0 + out.width >= D) mbar_arrive(smem_u32(&sm.o_empty[half]));
                mbar_arrive(smem_u32(&sm.out_full));
            }
        }
    }
}

// Adds up the streams of a unit's rows, a lane 16 bytes of a row, and writes them.
template <int D, int FEW>
__device__ void add_up(const CrossParams &p, Smem<D> &sm, int w, const DevCtx &ctx) {
    constexpr int STREAMS = 256 / FEW;
    const int lane = threadIdx.x & 31;
    volatile int *abort = &sm.abort;
    auto wait = [&](uint64_t &bar, int phase) {
        return __all_sync(0xffffffffu, bar_wait(smem_u32(&bar), phase & 1, ctx, abort));
    };
    const Out<D, FEW> out(p, sm);
    const int shift = out.shift(), c = lane & ((1 << shift) - 1), each = 32 >> shift;
    int outs = 0;
    for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, sm.units.wait(i, ctx, abort))) return;
        const LineUnit u = sm.units.u[i % UNITS];
        __syncwarp();
        if (lane == 0) sm.units.release(i);
        if (u.begin == u.end) return;
        const int rows = min(p.tokens, u.s.n - u.u * p.line.tokens) * p.G;
        const bool cut = u.cut();
        const size_t slot0 = ((size_t)blockIdx.x * 2 + (u.begin > 0 ? 0 : 1)) * FEW;
        const int t0 = u.s.t0 + u.u * p.line.tokens;
        auto orow = [&](int q) {  // of the output
            const int tq = p.token(q);
            return (size_t)(t0 + tq) * p.H + u.h * p.G + q - tq * p.G;
        };
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += out.width, ++outs) {
            if (!wait(sm.out_full, outs)) return;
#pragma unroll 1
            for (int q = w * each + (lane >> shift); q < rows; q += ADDERS * each) {
                float4 acc = *out.piece(0, q, c);
#pragma unroll
                for (int st = 1; st < STREAMS; ++st) {
                    const float4 x = *out.piece(st, q, c);
                    acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
                }
                if (cut)
                    *reinterpret_cast<float4 *>(
                        reinterpret_cast<float *>(p.ws + plan_rows_offset(FEW)) + (slot0 + q) * D +
                        c0 + 4 * c) = acc;
                else
                    *reinterpret_cast<uint2 *>(p.o + orow(q) * D + c0 + 4 * c) =
                        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.out_empty));
        }
    }
}

template <int D, int FEW>
__global__ void __launch_bounds__(NTHREADS, 1)
cross_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
             const __grid_constant__ CUtensorMap tv, const __grid_constant__ CrossParams p,
             const __grid_constant__ DevCtx ctx) {
    extern __shared__ __align__(1024) uint8_t dsmem[];
    using S = Smem<D>;
    S &sm = *reinterpret_cast<S *>(dsmem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.line.split) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (smem_u32(dsmem) & 1023u) {  // the swizzle is anchored to 1024-byte boundaries
        if (threadIdx.x == 0) record_error(ctx, DEVERR_LAYOUT);
        return;
    }
    if (warp == 0) {  // a lane a barrier
        if (lane < S::R) {
            mbar_init(smem_u32(&sm.full[lane]), 1);
            mbar_init(smem_u32(&sm.empty[lane]), FEW ? 1 : 2);  // the halves' MMAs
            mbar_init(smem_u32(&sm.raw[lane]), 1);
        }
        if (lane < 2) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&sm.s_full[lane][b]), 1);
                mbar_init(smem_u32(&sm.p_full[lane][b]), 4);
                mbar_init(smem_u32(&sm.pv_done[lane][b]), 1);
            }
            mbar_init(smem_u32(&sm.o_full[lane]), 1);
            mbar_init(smem_u32(&sm.o_empty[lane]), 4);
            mbar_init(smem_u32(&sm.drain[lane]), 1);
            mbar_init(smem_u32(&sm.drain[2 + lane]), 1);
        }
        if (lane == 0) {
            mbar_init(smem_u32(&sm.q_full), 1);
            mbar_init(smem_u32(&sm.q_empty), 2);
            mbar_init(smem_u32(&sm.meet), 8);
            mbar_init(smem_u32(&sm.out_full), 8);
            mbar_init(smem_u32(&sm.out_empty), ADDERS);
            sm.abort = 0;
            sm.issued = 0;
        }
        sm.units.init(4 + 1 + 8 + (FEW ? ADDERS : 0), lane);  // MMA issuers, tails, softmax
        fence_mbar_init();
        __syncwarp();
    } else if (warp == 1) {
        tmem_alloc(smem_u32(&sm.tmem_base), TMEM_COLS);
        tmem_relinquish();
    } else if (warp == 3 && lane < 3) {
        prefetch_tmap(lane == 0 ? &tk : lane == 1 ? &tv : &tq);
    } else if (warp >= SOFTMAX) {  // rows of Q that no box writes: their S is 0
        constexpr int COPIES = FEW ? 128 / FEW : 2, ROWS = FEW ? FEW : 128;
        const int free = (ROWS - p.rows) * 8;
        for (int i = 0; i < COPIES * S::NH; ++i)
            for (int e = threadIdx.x - SOFTMAX * 32; e < free; e += NTHREADS - SOFTMAX * 32)
                *reinterpret_cast<uint4 *>(sm.q[FEW ? 0 : i / S::NH] + i % S::NH * S::PART +
                                           ((FEW ? i / S::NH * FEW : 0) + p.rows) * 128 + e * 16) =
                    make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (!line_by_warp(p.line))
        line_start<false>(p.line, sm.line, reinterpret_cast<long long *>(sm.ml), ctx);
    tc_fence_before();
    set_up(warp == 0);
    tc_fence_after();
    if (warp == 0 && line_by_warp(p.line)) line_start_warp<false>(p.line, sm.line, ctx);
    const uint32_t tmem = warp == 0 ? 0u : sm.tmem_base;  // (the loader has not waited for it)
    // registers: 256 threads x 88 + 256 x 168 = the 512 x 128 of the launch
    if (warp < SOFTMAX) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) {
            load_tiles<D, FEW>(p, &tq, &tk, &tv, sm, ctx);
        } else if (warp == 2) {
            clear_tails<D>(sm, ctx);
        } else if (warp < 4) {
            issue_s<D, FEW>(p, sm, tmem, warp >> 1, ctx);
        } else if (warp < 6) {
            issue_pv<D, FEW>(p, sm, tmem, warp & 1, ctx);
        } else if (FEW) {
            add_up<D, FEW ? FEW : 32>(p, sm, warp - 6, ctx);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        if constexpr (FEW > 0) softmax_few<D, FEW>(p, sm, tmem, ctx);
        else softmax_many<D>(p, sm, tmem, ctx);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort == TIMED_OUT) record_error(ctx, DEVERR_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Joins the parts of cut units, a programmatic dependent of the kernel that wrote them: block x
// has the unit that is cut behind piece x, a warp a row of it. w_i = z_i 2^(m_i - m),
// lse = m + log2 sum_i w_i (+ the null logit), o = sum_i w_i o_i / sum_i w_i, in the order of the
// pieces, the columns spread over the lanes. Few parts (nearly all units of many rows have two):
// every lane weighs them all, sums and rows come in one round of loads, and what bounds is
// the instructions; more: lane i holds part i's sums, and it is latency that counts, so K rows
// are on their way at a time.
constexpr int JOIN_THREADS = 256;
template <int D, int K>
__global__ void __launch_bounds__(JOIN_THREADS)
cross_join(const uint8_t *ws, int slots, int side, int H, int G, uint32_t g_mul, uint32_t g_shift,
           const float *sinks, int null_sink, __nv_bfloat16 *o, float *lse) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int E = D / 32, BLOCKS = MAX_PIECES / 32;
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * (JOIN_THREADS / 32) + (threadIdx.x >> 5);
    const JoinNote n = reinterpret_cast<const JoinNote *>(ws)[blockIdx.x];
    if (r >= n.rows) return;
    // part i of the unit: the last of CTA x, then the first of x + side, x + 2 side, ..
    auto slot = [&](int i) { return ((size_t)(blockIdx.x + i * side) * 2 + (i == 0 ? 1 : 0)) * slots + r; };
    const float2 *sums = reinterpret_cast<const float2 *>(ws + plan_sums_offset());
    const float *rows = reinterpret_cast<const float *>(ws + plan_rows_offset(slots)) + lane * E;
    const int tok = (int)((__umulhi(g_mul, (uint32_t)r) + (uint32_t)r) >> g_shift), head = n.h * G + r - tok * G;
    const size_t out = (size_t)(n.t0 + tok) * H + head;
    const float null = null_sink ? state_sink(__ldg(sinks + head)) : -INFINITY;
    auto load = [&](int i, float (&x)[E]) {
        const float *at = rows + slot(i) * D;
        if constexpr (E == 4) *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(at);
        else *reinterpret_cast<float2 *>(x) = *reinterpret_cast<const float2 *>(at);
    };
    float acc[E] = {}, x[K][E], m = fmaxf(null, NOTHING), z;
    if (n.parts <= 4) {
        float2 part[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            part[d] = make_float2(NOTHING, 0.f);
            if (d >= n.parts) continue;
            part[d] = sums[slot(d)];
            load(d, x[d]);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) m = fmaxf(m, part[d].x);
        z = ex2(null - m);  // (0 without a null logit)
#pragma unroll
        for (int d = 0; d < 4; ++d) z += part[d].y *= ex2(part[d].x - m);
        // (over their sum, so that values near fp32's largest do not overflow)
        const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            if (d < n.parts)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(part[d].y * inv, x[d][e], acc[e]);
        store_row<D>(o + out * D, acc, lane);
        if (lse && lane == 0) lse[out] = z == 0.f ? -INFINITY : (m + log2f(z)) * LN2;
        return;
    }
    auto get = [&](int i) { return i < n.parts ? sums[slot(i)] : make_float2(NOTHING, 0.f); };
    const float2 mine = get(lane);
    m = fmaxf(m, mine.x);
    if (n.parts > 32) {
#pragma unroll
        for (int b = 1; b < BLOCKS; ++b) m = fmaxf(m, get(32 * b + lane).x);
    }
    m = warp_max(m);
    float w = mine.y * ex2(mine.x - m);
    z = w;
    if (n.parts > 32) {
#pragma unroll
        for (int b = 1; b < BLOCKS; ++b) {
            const float2 s = get(32 * b + lane);
            z += s.y * ex2(s.x - m);
        }
    }
    z = warp_sum(z) + ex2(null - m);
    const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll 1
    for (int i0 = 0; i0 < n.parts; i0 += 32) {
        if (i0 > 0) {
            const float2 s = get(i0 + lane);
            w = s.y * ex2(s.x - m);
        }
        w *= inv;
        const int cnt = min(32, n.parts - i0);
#pragma unroll 1
        for (int k = 0; k < cnt; k += K) {
#pragma unroll
            for (int d = 0; d < K; ++d)
                if (k + d < cnt) load(i0 + k + d, x[d]);
#pragma unroll
            for (int d = 0; d < K; ++d) {
                const float f = __shfl_sync(0xffffffffu, w, k + d & 31);
                if (k + d < cnt)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, x[d][e], acc[e]);
            }
        }
    }
    store_row<D>(o + out * D, acc, lane);
    if (lse && lane == 0) lse[out] = z == 0.f ? -INFINITY : (m + log2f(z)) * LN2;
}

// Rows of a unit in the FEW form, or 0 where a sequence has more of a KV head.
int few_rows(int max_q_len, int G) {
    const long long rows = (long long)max(1, max_q_len) * G;
    return rows <= 32 ? 32 : rows <= 64 ? 64 : 0;
}

template <int D, int FEW>
cudaError_t launch(const CrossArgs &a, const DevInfo &dev, cudaStream_t s) {
    constexpr int ROWS = FEW ? FEW : 256;
    const int G = a.H / a.Hkv;
    CrossParams p{};
    p.H = a.H;
    p.G = G;
    p.tokens = FEW ? min(FEW / G, max(1, a.max_q_len)) : 128 / G;
    p.rows = p.tokens * G;
    const bool split = a.workspace && a.workspace_bytes >= plan_workspace(ROWS, D);
    p.line = LineArgs{a.cu_seqlens, a.kv_starts, a.kv_lens, a.B, a.T, a.S, a.Hkv,
                      FEW ? p.tokens : 2 * p.tokens, FEW ? 0 : p.tokens, COST, FEW ? COST : LESS,
                      FEW ? (D == 128 ? 1 : 3) * COST : 2 * COST, split};
    // (many rows are not bound by the memory: no gain)
    const int side = FEW && a.Hkv % 2 == 0 && dev.sm_count > 1 ? 2 : 1;
    const int grid = line_grid(p.line, min(dev.sm_count, MAX_PIECES), side);
    p.scale_l2 = a.scale * LOG2E;
    p.sinks = a.sinks;
    p.sink_mode = a.sink_mode;
    p.o = static_cast<__nv_bfloat16 *>(a.o);
    p.o_wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
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
    if (verbose())
        fprintf(stderr, "sattn: cross_kernel<%d, %d> grid=%d rows=%d split=%d\n", D, FEW, grid,
                p.rows, p.line.split);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = sizeof(Smem<D>);
    cfg.stream = s;
    e = cudaLaunchKernelEx(&cfg, cross_kernel<D, FEW>, tq, tk, tv, p, make_ctx(dev));
    if (e != cudaSuccess || !split) return e;
    constexpr int K = FEW ? 8 : 4;  // (of 256 rows there are few parts, and warps enough)
    cfg.gridDim = dim3((unsigned)grid, (unsigned)(p.rows * (FEW ? 1 : 2) + 7) / 8);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cross_join<D, K>, (const uint8_t *)p.ws, ROWS, side, a.H, G, p.g_mul, p.g_shift, a.sinks,
                              (int)(a.sink_mode == 2), p.o, a.lse);
}

}  // namespace

size_t cross_tc_workspace(int max_q_len, int G, int d) {
    const int few = few_rows(max_q_len, G);
    return plan_workspace(few ? few : 256, d);
}

cudaError_t launch_cross_tc(const CrossArgs &a, const DevInfo &dev, cudaStream_t s) {
    const int few = few_rows(a.max_q_len, a.H / a.Hkv);
    if (a.d == 64)
        return few == 32   ? launch<64, 32>(a, dev, s)
               : few == 64 ? launch<64, 64>(a, dev, s)
                           : launch<64, 0>(a, dev, s);
    return few == 32   ? launch<128, 32>(a, dev, s)
           : few == 64 ? launch<128, 64>(a, dev, s)
                       : launch<128, 0>(a, dev, s);
}

}  // namespace sattn
