// How the tensor-core kernels over encoder states share out their work.
//
// A unit is a tile of one sequence and KV head with all that it meets: a tile of query rows
// with its steps over 128-key tiles (the attention), or 512 keys with their steps over tiles
// of query rows (KEYS: the key weights). Units are numbered sequence by sequence, KV
// head by KV head; their steps in a row, by what one costs (the last unit of a head, whose
// tiles are not all there, less), and before each unit's steps `extra` for what a
// unit costs by itself, form one line that is cut into equal pieces, one a CTA. A
// piece may begin and end inside a unit: a ragged batch then keeps every SM busy for the
// same time, whatever its lengths, and a few units spread over all SMs. Where the memory
// bounds, two CTAs take a piece side by side, of a group of two heads one each: a token's rows of
// both lie next to each other, and come from memory as one. (64 tokens over 257 to 6400 states of
// 8 KV heads, d = 64: 94 us with pieces of one head, 83 so, and 23 more where L2 fetched rows of
// other heads and lost them (map_rows); d = 128, rows of twice the length: 152 and 150.) The
// pieces of a unit that is cut leave partial results in the workspace, which are joined in a
// fixed order. Everything is computed from the lengths on the device, so a
// call needs no host copy of them and can be captured and replayed with other lengths.
#pragma once

#include "internal.h"
#include "paged_mma.cuh"
#include "states.cuh"

namespace sattn {

constexpr int STATE_KEYS = 128;  // keys a tile
constexpr int UNIT_TILES = 4;    // and tiles in a unit of keys

struct LineArgs {
    const int32_t *cu, *starts, *lens;
    int B, T, S, Hkv;  // Hkv: heads, or groups of them that CTAs take side by side
    int tokens;  // of a tile of query rows
    int half;    // tokens up to which such a tile costs less
    int cost, less;  // a step's cost, and with such a tile
    int extra;   // a unit's own cost
    int split;   // 0: no workspace, pieces end at unit boundaries
    int side;    // CTAs that share a piece, a head of a group each
    int pieces;
    uint32_t mul, shift;  // x / pieces = (high(mul x) + x) >> shift for 0 <= x < 2^31

    __device__ __forceinline__ int piece() const { return side == 2 ? blockIdx.x >> 1 : blockIdx.x; }
    // The CTA's head of group h.
    __device__ __forceinline__ int head(int h) const { return side == 2 ? 2 * h + (blockIdx.x & 1) : h; }
};

struct LineUnit {
    StateSeq s;
    int b, h, u, nu;     // sequence, KV head, unit of its nu
    int steps;           // at least one (an empty one's is masked)
    int one, last;       // a step's cost, and in the last of a head's units
    int begin, end;      // the steps of this piece, 0 .. steps
    int parts;           // pieces of a unit that begins in this one (not KEYS)
    __device__ __forceinline__ bool cut() const { return begin > 0 || end < steps; }
    __device__ __forceinline__ int step_cost() const { return u == nu - 1 ? last : one; }
};

// Sequence b's units; false if it has none.
template <bool KEYS>
__device__ __forceinline__ bool line_seq(const LineArgs &a, int b, LineUnit &u, bool &bad) {
    u.b = b;
    bad = !load_states(a.cu, a.starts, a.lens, b, a.T, a.S, u.s);
    if (bad) return false;
    constexpr int TILE_KEYS = KEYS ? UNIT_TILES * STATE_KEYS : STATE_KEYS;
    const int keys = (int)(((uint32_t)u.s.len + TILE_KEYS - 1) / TILE_KEYS);
    const int rows = (int)(((uint32_t)u.s.n + a.tokens - 1) / (uint32_t)a.tokens);
    u.nu = KEYS ? keys : rows;
    u.steps = max(1, KEYS ? rows : keys);
    u.one = a.cost;
    if (KEYS)  // of UNIT_TILES, so many are there
        u.last = (u.s.len - (keys - 1) * TILE_KEYS + STATE_KEYS - 1) / STATE_KEYS * a.less;
    else
        u.last = u.s.n - (rows - 1) * a.tokens <= a.half ? a.less : a.cost;
    return u.nu > 0;
}
// The line of one KV head of that sequence.
__device__ __forceinline__ long long line_head(const LineArgs &a, const LineUnit &u) {
    return (long long)u.nu * ((long long)u.steps * u.one + a.extra) -
           (long long)u.steps * (u.one - u.last);
}

// What a CTA starts from (in shared memory).
struct LineStart {
    long long x0, x1;  // its piece of the line
    long long ustart;  // where the unit that holds x0 starts
    long long per;     // positions a piece
    LineUnit u;
};

// a / b for a >= 0, b > 0. Small ones (almost all) by way of fp32: the quotient of two numbers
// below 2^22 is off by less than 1 there, and is put right. A CTA has four divisions, one
// after the other, to make before its first load, of 150 to 200 cycles in integers.
__device__ __forceinline__ long long line_div(long long a, long long b) {
    if ((a | b) >> 22) return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
    int q = (int)__fdividef((float)(int)a, (float)(int)b);
    const int r = (int)a - q * (int)b;
    return q + (r >= (int)b) - (r < 0);
}
// The piece that position x of the line lies in.
__device__ __forceinline__ int line_piece(const LineStart &ls, long long x) {
    return (int)line_div(x, ls.per);
}
__device__ __forceinline__ long long warp_prefix64(long long v) {  // over the lanes up to this one
    const int lane = threadIdx.x & 31;
    if (__all_sync(0xffffffffu, v < 1 << 26)) {
        int x = (int)v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += w;
        }
        return x;
    }
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const long long w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

// The CTA's piece of a line of that length.
__device__ __forceinline__ void line_ends(const LineArgs &a, LineStart &ls, long long total,
                                          bool writes, long long &x0, long long &x1) {
    const long long up = total + a.pieces - 1;
    long long per = up >> 31 ? up / a.pieces
                             : (__umulhi(a.mul, (uint32_t)up) + (uint32_t)up) >> a.shift;
    per = max(per, (long long)a.cost);  // so that no piece between others lacks a step
    x0 = min(total, a.piece() * per);
    x1 = min(total, x0 + per);
    if (writes) {
        ls.x0 = x0;
        ls.x1 = x1;
        ls.per = per;
    }
}
// The unit of position x0, which lies in sequence u.b, whose line starts at `before`.
__device__ __forceinline__ void line_unit(const LineArgs &a, LineStart &ls, LineUnit &u,
                                          long long x0, long long before) {
    const long long head = line_head(a, u), one = (long long)u.steps * u.one + a.extra;
    u.h = (int)line_div(x0 - before, head);
    before += u.h * head;
    u.u = min(u.nu - 1, (int)line_div(x0 - before, one));
    ls.u = u;
    ls.ustart = before + u.u * one;
}

// Batches that one warp plans (line_start_warp), a lane a few sequences: the loading warp does it
// while the others set up what they need, and starts its loads without meeting them.
constexpr int LINE_WARP = 128;
__device__ __forceinline__ bool line_by_warp(const LineArgs &a) { return a.B <= LINE_WARP; }

template <bool KEYS>
__device__ __forceinline__ void line_start_warp(const LineArgs &a, LineStart &ls, const DevCtx &ctx) {
    const int lane = threadIdx.x & 31;
    const int per = (a.B + 31) >> 5, b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
    LineUnit u;
    bool bad = false, wrong;
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        if (line_seq<KEYS>(a, b, u, wrong)) mine += a.Hkv * line_head(a, u);
        bad |= wrong;
    }
    if (bad && blockIdx.x == 0) record_error(ctx, DEVERR_SEQLENS);
    const long long upto = warp_prefix64(mine);
    long long before = upto - mine, x0, x1;
    line_ends(a, ls, __shfl_sync(0xffffffffu, upto, 31), lane == 0, x0, x1);
    if (x0 < x1 && x0 >= before && x0 < upto) {
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            if (per > 1 && !line_seq<KEYS>(a, b, u, wrong)) continue;
            const long long all = a.Hkv * line_head(a, u);
            if (x0 < before + all) {
                line_unit(a, ls, u, x0, before);
                break;
            }
            before += all;
        }
    }
    __syncwarp();
}

// The same by the whole CTA (a whole number of warps, 640 threads at most), with a number a
// warp in shared memory; ends with a barrier.
template <bool KEYS>
__device__ __forceinline__ void line_start(const LineArgs &a, LineStart &ls, long long *warps,
                                           const DevCtx &ctx) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    LineUnit u;
    bool bad = false;
    long long x0, x1;
    const int per = (a.B + (int)blockDim.x - 1) / (int)blockDim.x;  // sequences a thread
    const int b0 = (int)min((long long)a.B, (long long)tid * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        bool wrong;
        if (line_seq<KEYS>(a, b, u, wrong)) mine += a.Hkv * line_head(a, u);
        bad |= wrong;
    }
    if (bad && blockIdx.x == 0) record_error(ctx, DEVERR_SEQLENS);
    const long long inc = warp_prefix64(mine);
    if (lane == 31) warps[warp] = inc;
    __syncthreads();
    const long long ws = warp_prefix64(lane < nw ? warps[lane] : 0);
    long long before = inc - mine;
    if (warp > 0) before += __shfl_sync(0xffffffffu, ws, warp - 1);
    line_ends(a, ls, __shfl_sync(0xffffffffu, ws, 31), tid == 0, x0, x1);
    if (x0 < x1 && x0 >= before && x0 < before + mine) {
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            bool wrong;
            if (!line_seq<KEYS>(a, b, u, wrong)) continue;
            const long long all = a.Hkv * line_head(a, u);
            if (x0 < before + all) {
                line_unit(a, ls, u, x0, before);
                break;
            }
            before += all;
        }
    }
    __syncthreads();
}

// The CTA's set-up is done: the loading warp (0) arrives when its barriers are there and goes
// on, the others wait for it and for one another.
__device__ __forceinline__ void set_up(bool loader) {
    if (loader) asm volatile("barrier.cta.arrive 1, %0;" ::"r"(blockDim.x) : "memory");
    else asm volatile("barrier.cta.sync 1, %0;" ::"r"(blockDim.x) : "memory");
}

// Walks the units of a CTA's piece.
template <bool KEYS> struct LineIter {
    LineUnit u;
    long long ustart, x1;  // where u starts on the line
    bool live;

    __device__ __forceinline__ LineIter(const LineArgs &a, const LineStart &ls) {
        x1 = ls.x1;
        live = ls.x0 < x1;
        if (!live) return;
        u = ls.u;
        ustart = ls.ustart;
        // a step is the piece's that its first position lies in
        const long long into = ls.x0 - ustart - a.extra, w = u.step_cost();
        u.begin = into <= 0 ? 0 : (int)line_div(into + w - 1, w);
        // uncut, the unit is all of the piece's that its first step lies in
        if (!a.split && u.begin > 0) u.begin = u.steps;
        clip(a, ls);
        if (live && u.begin == u.end) next(a, ls);
    }
    // The steps of u in this piece.
    __device__ __forceinline__ void clip(const LineArgs &a, const LineStart &ls) {
        const long long t0 = ustart + a.extra, w = u.step_cost();
        live = live && t0 + u.begin * w < x1;
        u.end = u.steps;
        u.parts = 1;
        if (!live || !a.split) return;
        if (t0 + (u.steps - 1) * w >= x1) u.end = (int)line_div(x1 - t0 + w - 1, w);
        if (!KEYS && u.begin == 0 && u.end < u.steps)
            u.parts = line_piece(ls, t0 + (u.steps - 1) * w) - a.piece() + 1;
    }
    // To the next unit of the line; there may be none behind this piece.
    __device__ __forceinline__ void next(const LineArgs &a, const LineStart &ls) {
        live = u.end == u.steps;
        if (!live) return;
        ustart += (long long)u.steps * u.step_cost() + a.extra;
        if (++u.u == u.nu) {
            u.u = 0;
            if (++u.h == a.Hkv) {
                u.h = 0;
                int b = u.b + 1;
                bool bad;
#pragma unroll 1
                while (b < a.B && !line_seq<KEYS>(a, b, u, bad)) ++b;
                if (b >= a.B) {
                    live = false;
                    return;
                }
            }
        }
        u.begin = 0;
        clip(a, ls);
    }
};

// The units in shared memory: the loading warp walks them and hands them on, the
// other roles read what they need. A unit without steps ends the piece.
template <int N> struct LineRing {
    LineUnit u[N];
    uint64_t full[N], empty[N];

    __device__ __forceinline__ void init(int readers, int lane) {  // a warp
        if (lane < N) {
            mbar_init(smem_u32(&full[lane]), 1);
            mbar_init(smem_u32(&empty[lane]), readers);
        }
    }
    // One thread: unit number i.
    __device__ __forceinline__ bool put(int i, const LineUnit &x, const DevCtx &ctx,
                                        volatile int *abort) {
        if (i >= N && !bar_wait(smem_u32(&empty[i % N]), (i / N - 1) & 1, ctx, abort)) return false;
        u[i % N] = x;
        mbar_arrive(smem_u32(&full[i % N]));
        return true;
    }
    __device__ __forceinline__ bool wait(int i, const DevCtx &ctx, volatile int *abort) {
        return bar_wait(smem_u32(&full[i % N]), (i / N) & 1, ctx, abort);
    }
    __device__ __forceinline__ void release(int i) { mbar_arrive(smem_u32(&empty[i % N])); }
};

// One lane of a converged warp, the same each time. MMAs are issued by whole warps that branch
// on this: their operands then stay in uniform registers (issued in a role of a single
// thread, each MMA takes that thread 65 to 115 cycles).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(e));
    return e != 0;
}

// A count in shared memory that one thread raises and others wait for.
__device__ __forceinline__ void count_set(uint32_t at, int v) {
    asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ int count_get(uint32_t at) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
// Waits until the count is at least n, as bar_wait waits for a phase.
__device__ __forceinline__ bool count_wait(uint32_t at, int n, const DevCtx &ctx,
                                           volatile int *abort) {
    if (count_get(at) >= n) return true;
    const uint32_t limit = (uint32_t)min(ctx.wait_ns, (uint64_t)4000000000u);
    uint32_t t0, t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
#pragma unroll 1
    do {
        if (count_get(at) >= n) return true;
        if (*abort) return false;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    } while (t - t0 <= limit);
    *abort = TIMED_OUT;
    return false;
}

// Shares the line out to `grid` CTAs, `side` of them a piece; returns the CTAs in use.
inline int line_grid(LineArgs &a, int grid, int side) {
    a.side = side;
    a.Hkv /= side;
    a.pieces = grid / side;
    a.shift = 0;
    while ((1ll << a.shift) < a.pieces) ++a.shift;
    a.mul = (uint32_t)((((1ull << a.shift) - a.pieces) << 32) / (uint32_t)a.pieces + 1);
    return a.pieces * side;
}

// Rows of heads x d elements, `stride` elements apart, as boxes of 64 columns, `heads_box`
// heads and `rows_box` rows. A row of 64 is half of what L2 would fetch by default: it would read
// a neighbouring head's as well, which may be gone before it is used.
inline bool map_rows(CUtensorMap *m, const void *p, int64_t stride, int heads, int d, int rows,
                     int heads_box, int rows_box) {
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)heads, (uint64_t)rows};
    const uint64_t strides[2] = {(uint64_t)d * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {64, (uint32_t)heads_box, (uint32_t)rows_box};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims,
                             strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                             d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                     : CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
}

}  // namespace sattn
