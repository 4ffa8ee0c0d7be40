// How the tensor-core kernels of the paged cache share out their work.
//
// A unit is up to ROWS query rows of one sequence and KV head (rows run
// token-major over the tokens and the heads of the group, so any group size
// fills a unit) with the 128-key tiles that any of them can see. Units are
// numbered sequence by sequence, KV head by KV head; their tiles in a row, and
// before each unit's tiles `extra` for what a unit costs by itself, form one
// line that is cut into equal pieces, one a CTA. A piece may
// begin and end inside a unit: a ragged batch then keeps every SM busy for the
// same time, whatever its lengths, and one long sequence spreads over all SMs.
// A unit that lies in one piece is finished there; the pieces of a unit that
// is cut write partial results (normalised rows and their log2 denominators)
// to the workspace, and they are joined in a fixed order.
// Everything is computed from the lengths on the device, so a call needs no
// host copy of them and can be captured and replayed with other lengths.
#pragma once

#include <math.h>

#include "internal.h"
#include "paged.cuh"
#include "paged_mma.cuh"

namespace sattn {

constexpr int TILE = 128;           // keys per tile
constexpr float NOTHING = -3.4e38f;  // maximum of a row that has seen no key yet

struct PlanArgs {
    const int32_t *cu, *lens;
    int B, T, G, Hkv, page, causal, wl;
    long long capacity;  // positions that the page table holds
    int split;           // 0: no workspace, pieces end at unit boundaries
    int extra;           // a unit's own cost, in tiles
    uint32_t g_mul, g_shift;

    // row / G for 0 <= row < 2^31: with s = ceil(log2 G) and
    // mul = 2^32 (2^s - G) / G + 1, row / G = (high(mul row) + row) >> s.
    __device__ __forceinline__ int token(int row) const {
        return (int)((__umulhi(g_mul, (uint32_t)row) + (uint32_t)row) >> g_shift);
    }
};

__host__ inline PlanArgs plan_args(const PagedArgs &a, int split, int extra) {
    const uint32_t G = (uint32_t)(a.H / a.Hkv);
    uint32_t s = 0;
    while ((1ull << s) < G) ++s;
    const uint32_t mul = (uint32_t)((((1ull << s) - G) << 32) / G + 1);
    return PlanArgs{a.cu_seqlens, a.kv_lens, a.B, a.T, (int)G, a.Hkv, a.page, a.causal,
                    a.window_left, (long long)a.max_pages * a.page, split, extra, mul, s};
}

// One unit's rows and keys.
template <int ROWS> struct Unit {
    PagedSeq s;
    int b, h, rt, nrt;     // sequence, KV head, row tile of its nrt
    int row0, nrows;       // rows of the sequence's n * G that the unit takes
    int lo, hi;            // first and last key that any of its rows sees
    int ilo, ihi;          // keys that all of them see
    int t_first, ntiles;   // tiles of the sequence; ntiles >= 1 (an empty unit's is masked)
    int begin, end;        // the tiles of this piece, 0 .. ntiles
    int c0, parts;         // of a cut unit: its first piece, and how many
    int nan_values;        // set where a key that not every row sees has NaN value codes
    int nan_zero;          // and where one of a page with a value scale of 0 has
    int far;               // set where a page's value scale is far (far_scale)

    // The same piece in halves of tiles, less the halves that no row sees.
    __device__ __forceinline__ int sub_begin() const {
        return 2 * begin + (begin == 0 && (lo & (TILE - 1)) >= TILE / 2 ? 1 : 0);
    }
    __device__ __forceinline__ int sub_end() const {
        return 2 * end - (end == ntiles && (hi & (TILE - 1)) < TILE / 2 ? 1 : 0);
    }
    __device__ __forceinline__ int pos(const PlanArgs &p, int row) const {
        return s.len - s.n + p.token(row);
    }

    __device__ __forceinline__ void set_rows(const PlanArgs &p, int rt_) {
        rt = rt_;
        row0 = rt * ROWS;
        nrows = min(ROWS, s.n * p.G - row0);
        const int p0 = pos(p, row0), p1 = pos(p, row0 + nrows - 1);
        lo = p.wl < 0 ? 0 : max(0, p0 - p.wl);
        ilo = p.wl < 0 ? 0 : max(0, p1 - p.wl);
        hi = p.causal ? p1 : s.len - 1;
        ihi = p.causal ? p0 : s.len - 1;
        t_first = lo / TILE;
        ntiles = hi < lo ? 1 : hi / TILE - t_first + 1;
        nan_values = nan_zero = far = 0;
    }
};

template <int ROWS>
__device__ __forceinline__ bool plan_seq(const PlanArgs &p, int b, Unit<ROWS> &u) {
    u.b = b;
    if (!load_seq(p.cu, p.lens, b, p.T, p.capacity, u.s)) return false;
    u.nrt = (int)(((long long)u.s.n * p.G + ROWS - 1) / ROWS);
    return true;
}

// Line length of one head of a sequence: of its row tiles rt, rt + step, ...
template <int ROWS>
__device__ __forceinline__ long long seq_tiles(const PlanArgs &p, Unit<ROWS> &u, int rt, int step) {
    long long sum = 0;
#pragma unroll 1
    for (; rt < u.nrt; rt += step) {
        u.set_rows(p, rt);
        sum += u.ntiles + p.extra;
    }
    return sum;
}
__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Sums over the lanes up to this one.
__device__ __forceinline__ long long warp_prefix(long long v) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const long long w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

// What a CTA starts from (in shared memory).
struct PlanStart {
    long long x0, x1;  // its piece of the line
    long long total, ustart;  // the line; where the unit that holds x0 starts
    int pieces, b, h, rt;
    long long wsum[32];
    long long before;  // line before the sequences b0 .. b1 - 1, in which x0 lies
    int b0, b1;
};

// The piece that position x of the line lies in.
static __device__ __noinline__ int piece_of(long long x, int pieces, long long total) {
    return (int)(((x + 1) * pieces - 1) / total);
}
static __device__ __noinline__ long long piece_start(long long total, int c, int pieces) {
    return total * c / pieces;
}

// The CTA's piece of a line of that length.
__device__ __forceinline__ void plan_piece(PlanStart &ps, long long total, bool writes,
                                           long long &x0, long long &x1) {
    const int pieces = (int)min((long long)gridDim.x, max(1ll, total));
    const int c = min((int)blockIdx.x, pieces);
    if (total < (1 << 23)) {  // c <= 256: 32-bit division
        x0 = (uint32_t)total * (uint32_t)c / (uint32_t)pieces;
        x1 = (uint32_t)total * (uint32_t)min(c + 1, pieces) / (uint32_t)pieces;
    } else {
        x0 = piece_start(total, c, pieces);
        x1 = piece_start(total, min(c + 1, pieces), pieces);
    }
    if (writes) {
        ps.x0 = x0;
        ps.x1 = x1;
        ps.total = total;
        ps.pieces = pieces;
        ps.b = ps.h = ps.rt = 0;  // (in bounds even if the lengths change meanwhile)
        ps.ustart = x0;
    }
}

// The head and unit of position x0 in sequence u.b, whose heads take ph each from `at` on.
template <int ROWS>
__device__ __forceinline__ void plan_unit(const PlanArgs &p, PlanStart &ps, Unit<ROWS> &u,
                                          long long x0, long long at, long long ph) {
    const int lane = threadIdx.x & 31;
    const long long off = x0 - at;
    const int h = min(p.Hkv - 1, max(off, ph) < (1ll << 31) ? (int)((uint32_t)off / (uint32_t)ph)
                                                            : (int)(off / ph));
    at += h * ph;
    if (u.nrt == 1) {
        if (lane == 0) ps.b = u.b, ps.h = h, ps.rt = 0, ps.ustart = at;
        return;
    }
#pragma unroll 1
    for (int r0 = 0; r0 < u.nrt; r0 += 32) {
        int nt = 0;
        if (r0 + lane < u.nrt) {
            u.set_rows(p, r0 + lane);
            nt = u.ntiles + p.extra;
        }
        const long long upto = warp_prefix(nt);
        if (nt > 0 && x0 >= at + upto - nt && x0 < at + upto) {
            ps.b = u.b;
            ps.h = h;
            ps.rt = r0 + lane;
            ps.ustart = at + upto - nt;
        }
        at += __shfl_sync(0xffffffffu, upto, 31);
        if (x0 < at) break;
    }
}

// Up to 32 sequences of few rows: one warp, a lane a sequence, while another sets up the
// barriers. (A request of 1000 positions: 10.5 us; 13.3 with the path below, whose warps
// meet three times, and one thread for the barriers.)
template <int ROWS>
__device__ __forceinline__ void plan_small(const PlanArgs &p, PlanStart &ps, const DevCtx &ctx) {
    const int lane = threadIdx.x & 31;
    Unit<ROWS> u;
    u.nrt = 0;
    bool bad = false;
    long long ph = 0;
    if (lane < p.B) bad = !plan_seq(p, lane, u);
    if (bad) u.nrt = 0;
    if (bad && blockIdx.x == 0) record_error(ctx, DEVERR_SEQLENS);
    if (__any_sync(0xffffffffu, u.nrt > 8)) {  // rows after all: the sequences in turn
#pragma unroll 1
        for (int b = 0; b < p.B; ++b) {
            Unit<ROWS> v;
            if (!plan_seq(p, b, v)) v.nrt = 0;
            const long long sum = warp_sum64(seq_tiles(p, v, lane, 32));
            if (lane == b) ph = sum;
        }
    } else {
        ph = seq_tiles(p, u, 0, 1);
    }
    const long long mine = ph * p.Hkv, upto = warp_prefix(mine), before = upto - mine;
    long long x0, x1;
    plan_piece(ps, __shfl_sync(0xffffffffu, upto, 31), lane == 0, x0, x1);
    __syncwarp();
    if (x0 >= x1) return;
    const int b = __ffs(__ballot_sync(0xffffffffu, x0 >= before && x0 < upto)) - 1;
    if (b < 0) return;
    u.b = b;
    u.s.t0 = __shfl_sync(0xffffffffu, u.s.t0, b);
    u.s.n = __shfl_sync(0xffffffffu, u.s.n, b);
    u.s.len = __shfl_sync(0xffffffffu, u.s.len, b);
    u.nrt = __shfl_sync(0xffffffffu, u.nrt, b);
    plan_unit(p, ps, u, x0, __shfl_sync(0xffffffffu, before, b), __shfl_sync(0xffffffffu, ph, b));
}

// Called by the whole CTA (blockDim.x a multiple of 32); ends with a barrier.
// Small batches are summed a warp a sequence, since one may have many units;
// large ones a thread a run of sequences.
template <int ROWS>
__device__ void plan_start(const PlanArgs &p, PlanStart &ps, const DevCtx &ctx) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    if constexpr (ROWS <= 32) {
        if (p.B <= 32) {
            if (warp == 0) plan_small<ROWS>(p, ps, ctx);
            __syncthreads();
            return;
        }
    }
    const bool by_warp = p.B <= 2 * nw;
    const int workers = by_warp ? nw : (int)blockDim.x, me = by_warp ? warp : tid;
    const int per = (p.B + workers - 1) / workers;
    const int b0 = (int)min((long long)p.B, (long long)me * per), b1 = min(p.B, b0 + per);
    Unit<ROWS> u;
    long long mine = 0;
    bool bad = false;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        if (!plan_seq(p, b, u)) bad = true;
        else mine += seq_tiles(p, u, by_warp ? lane : 0, by_warp ? 32 : 1) * p.Hkv;
    }
    if (bad && blockIdx.x == 0) record_error(ctx, DEVERR_SEQLENS);
    if (by_warp) {  // the lanes' shares, counted once
        mine = warp_sum64(mine);
        if (lane != 31) mine = 0;
    }
    const long long inc = warp_prefix(mine);
    if (lane == 31) ps.wsum[warp] = inc;
    __syncthreads();
    const long long ws = lane < nw ? ps.wsum[lane] : 0, upto = warp_prefix(ws);
    const long long before = __shfl_sync(0xffffffffu, upto - ws, warp) + inc - mine;
    long long x0, x1;
    plan_piece(ps, __shfl_sync(0xffffffffu, upto, 31), tid == 0, x0, x1);
    if (x0 < x1 && x0 >= before && x0 < before + mine) {
        ps.before = before;
        ps.b0 = b0;
        ps.b1 = b1;
    }
    __syncthreads();
    if (warp == 0 && x0 < x1) {  // the sequence, head and unit of x0
        long long at = ps.before, ph = 0;
        int b = ps.b0;
#pragma unroll 1
        for (; b < ps.b1; ++b) {
            if (!plan_seq(p, b, u)) continue;
            ph = warp_sum64(seq_tiles(p, u, lane, 32));
            if (x0 < at + ph * p.Hkv) break;
            at += ph * p.Hkv;
        }
        if (b < ps.b1) plan_unit(p, ps, u, x0, at, ph);
    }
    __syncthreads();
}

// Walks the units of a CTA's piece.
template <int ROWS> struct UnitIter {
    Unit<ROWS> u;
    long long ustart, x1;  // where u starts on the line
    bool live;

    __device__ __forceinline__ UnitIter(const PlanArgs &p, const PlanStart &ps) {
        x1 = ps.x1;
        live = ps.x0 < x1;
        if (!live) return;
        plan_seq(p, ps.b, u);
        u.h = ps.h;
        u.set_rows(p, ps.rt);
        ustart = ps.ustart;
        u.begin = (int)max(0ll, ps.x0 - ustart - p.extra);
        // uncut, the unit is all of the piece's that its first tile lies in
        if (!p.split && u.begin > 0) u.begin = u.ntiles;
        clip(p, ps);
    }
    // The tiles of u in this piece (there may be none of the first unit).
    __device__ __forceinline__ void clip(const PlanArgs &p, const PlanStart &ps) {
        const long long t0 = ustart + p.extra;
        live = live && t0 + u.begin < x1;
        u.end = p.split ? (int)min((long long)u.ntiles, x1 - t0) : u.ntiles;
        u.c0 = 0;
        u.parts = 1;
        if (live && p.split && (u.begin > 0 || u.end < u.ntiles)) {
            u.c0 = piece_of(t0, ps.pieces, ps.total);
            u.parts = piece_of(t0 + u.ntiles - 1, ps.pieces, ps.total) - u.c0 + 1;
        }
    }
    // To the next unit of the line; there may be none behind this piece.
    __device__ __forceinline__ void next(const PlanArgs &p, const PlanStart &ps) {
        live = u.end == u.ntiles;
        if (!live) return;
        ustart += u.ntiles + p.extra;
        int rt = u.rt + 1;
        if (rt == u.nrt) {
            rt = 0;
            if (++u.h == p.Hkv) {
                u.h = 0;
                int b = u.b + 1;
#pragma unroll 1
                for (; b < p.B; ++b)
                    if (plan_seq(p, b, u) && u.s.n > 0) break;
                if (b == p.B) {
                    live = false;
                    return;
                }
            }
        }
        u.set_rows(p, rt);
        u.begin = 0;
        clip(p, ps);
    }
};

// Page of a sequence's page slot j: its id where a key that the unit sees lies
// in it, -1 where none does (the table is not read), -2 for an entry that is no page.
template <int ROWS>
__device__ __forceinline__ int page_of(const int32_t *table, int max_pages, int num_pages,
                                       int shift, const Unit<ROWS> &u, int j) {
    const int first = j << shift;
    if (first > u.hi || first + (1 << shift) <= u.lo) return -1;
    const int pid = __ldg(table + (size_t)u.b * max_pages + j);
    return pid >= 0 && pid < num_pages ? pid : -2;
}

// A page's scales as the softmax takes them: the key scale, the log2 of the
// value scale (-inf hides the page's keys), 1 / the value scale, and whether
// that is not 0: with a zero value scale the keys are weighed as with the least
// scale and the values dropped.
//
// The log2 goes into the exponent of the probabilities, e = x + log2 s with x the logit, and
// 1 / s takes it out of what they add to the row sum l. With scales from 2^-64 to 2^24 what
// is flushed to 0, a probability or the sum at a move of m by more than 2^126, would have
// added 2^-33 of the sum a key at most (2^-126 of e's maximum, 2^88 between the scales, 2^5
// that m lags behind). For a scale beyond (far_scale) 1 / s may be infinite or 0
// and such a loss the whole sum, so in a unit with such a page 2^(x - n) is summed apart,
// with a maximum n of the logits alone: a second pass over S in small slow code, kept out
// of the hot loops (inside one it costs more by being there than by running: up to a tenth
// of a call that never takes it).
__device__ __forceinline__ float4 page_scales(const float *k_scale, const float *v_scale, int pid,
                                              int Hkv, int h) {
    if (pid < 0) return make_float4(1.f, -INFINITY, 0.f, 0.f);
    const size_t at = (size_t)pid * Hkv + h;
    const float vs = __ldg(v_scale + at), e = vs > 0.f ? vs : LEAST_SCALE;
    return make_float4(__ldg(k_scale + at), __log2f(e), __fdividef(1.f, e), vs > 0.f ? 1.f : 0.f);
}

__device__ __forceinline__ bool far_scale(float s) {
    return s > 0.f && !(s >= LEAST_SCALE && s <= 16777216.f);
}
__device__ __forceinline__ bool far_log2(float s) { return !(s >= -64.f && s <= 24.f); }

// NaN value codes of keys that some rows of a unit see and others do not. The MMA
// multiplies every key's values by every row's weight, and 0 * NaN is NaN, so such
// codes are taken out of the tile (without_nan) and put back at the unit's end into
// the rows that see them: each_partial_key calls at(key, codes) for the piece's
// keys from `lo` to `hi` that not every row sees. Pages with a value scale of 0 are
// cleared altogether: where one has a NaN, for their other keys too.
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) {  // 0xff for each NaN code
    return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
}
__device__ __forceinline__ bool without_nan(uint4 &x) {
    const uint4 n = make_uint4(nan_codes(x.x), nan_codes(x.y), nan_codes(x.z), nan_codes(x.w));
    x = make_uint4(x.x & ~n.x, x.y & ~n.y, x.z & ~n.z, x.w & ~n.w);
    return n.x | n.y | n.z | n.w;
}
template <int D, int ROWS, typename Params, typename F>
__device__ __forceinline__ void each_partial_key(const Params &p, const Unit<ROWS> &u, int lo,
                                                 int hi, F at) {
    const int a = max(lo, (u.t_first + u.begin) * TILE);
    const int z = min(hi, (u.t_first + u.end) * TILE - 1);
#pragma unroll 1
    for (int k = a; k <= z; ++k) {
        const bool all_see = k >= u.ilo && k <= u.ihi;
        if (all_see && !u.nan_zero) {
            k = u.ihi;
            continue;
        }
        const int pid = __ldg(p.page_table + (size_t)u.b * p.max_pages + (k >> p.page_shift));
        const size_t ph = (size_t)pid * p.plan.Hkv + u.h;
        if (pid < 0 || pid >= p.num_pages || (all_see && __ldg(p.v_scale + ph) > 0.f)) {
            k |= p.page - 1;  // nothing there for such keys of the page: to the last of them
            if (all_see) k = min(k, u.ihi);
            continue;
        }
        at(k, p.v_cache + (ph * p.page + (k & (p.page - 1))) * D);
    }
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x,
                                            int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

// Tensor map of a cache [pages, Hkv, page, d] as rows of d bytes, one page and head a box.
inline bool map_cache(CUtensorMap *m, const uint8_t *cache, const PagedArgs &a,
                      CUtensorMapSwizzle sw) {
    const uint64_t dims[2] = {(uint64_t)a.d, (uint64_t)a.num_pages * a.Hkv * a.page};
    const uint64_t strides[1] = {(uint64_t)a.d};
    const uint32_t box[2] = {(uint32_t)a.d, (uint32_t)a.page};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(cache), dims,
                             strides, box, sw) == CUDA_SUCCESS;
}
inline int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// The units in shared memory: the loading warp walks them and hands them on, the
// other roles read what they need (their registers are for other things). A unit
// without tiles ends the piece.
template <int ROWS, int N> struct UnitRing {
    Unit<ROWS> u[N];
    uint64_t full[N], empty[N];

    __device__ __forceinline__ void init(int readers, int lane) {  // a warp
        if (lane < N) {
            mbar_init(smem_u32(&full[lane]), 1);
            mbar_init(smem_u32(&empty[lane]), readers);
        }
    }
    // One thread: unit number i (the last one has end == begin).
    __device__ __forceinline__ bool put(int i, const Unit<ROWS> &x, const DevCtx &ctx,
                                        volatile int *abort) {
        if (i >= N && !bar_wait(smem_u32(&empty[i % N]), (i / N - 1) & 1, ctx, abort))
            return false;
        u[i % N] = x;
        mbar_arrive(smem_u32(&full[i % N]));
        return true;
    }
    __device__ __forceinline__ bool wait(int i, const DevCtx &ctx, volatile int *abort) {
        return bar_wait(smem_u32(&full[i % N]), (i / N) & 1, ctx, abort);
    }
    __device__ __forceinline__ void release(int i) { mbar_arrive(smem_u32(&empty[i % N])); }
};

// A piece's note for the join launch: whether it begins inside a unit, whether
// that unit also goes on behind the piece, and which unit it is.
struct PlanNote {
    int cont, through, t0, h, row0, nrows, pad0, pad1;
};

// Workspace: PlanNote [pieces], or the join counters of the decode kernel [pieces];
// (m, z) [pieces][2][ROWS], rows [pieces][2][ROWS][D] (fp32).
// Part 0 of a piece is its first unit if that began earlier, part 1 its last
// unit if that begins here and goes on. Of a part's row: its maximum m, its
// denominator z = sum 2^(x - m) (as one number, m + log2 z, large logits would
// swallow z), and o.
constexpr int MAX_PIECES = 256;
__host__ __device__ constexpr size_t plan_sums_offset() { return MAX_PIECES * sizeof(PlanNote); }
__host__ __device__ constexpr size_t plan_rows_offset(int rows) {
    return plan_sums_offset() + (size_t)MAX_PIECES * 2 * rows * sizeof(float2);
}
__host__ __device__ constexpr size_t plan_workspace(int rows, int d) {
    return plan_rows_offset(rows) + (size_t)MAX_PIECES * 2 * rows * d * 4;
}
__device__ __forceinline__ unsigned *join_counters(uint8_t *ws) {
    return reinterpret_cast<unsigned *>(ws);
}
__device__ __forceinline__ float2 *part_sums(uint8_t *ws) {
    return reinterpret_cast<float2 *>(ws + plan_sums_offset());
}

template <int ROWS>
__device__ __forceinline__ void write_note(const UnitIter<ROWS> &it, uint8_t *ws) {
    PlanNote n{};
    if (it.live) {
        n.cont = it.u.begin > 0;
        n.through = it.u.begin > 0 && it.u.end < it.u.ntiles;
        n.t0 = it.u.s.t0;
        n.h = it.u.h;
        n.row0 = it.u.row0;
        n.nrows = it.u.nrows;
    }
    reinterpret_cast<PlanNote *>(ws)[blockIdx.x] = n;
}

// Joins the pieces of cut units; a programmatic dependent of the kernel that
// wrote them. `rows` rows of d columns per unit, `pieces` CTAs in that launch.
cudaError_t launch_paged_join(const PagedArgs &a, int rows, int pieces, cudaStream_t s);

}  // namespace sattn
