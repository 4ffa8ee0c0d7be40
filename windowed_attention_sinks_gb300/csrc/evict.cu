// Eviction of a sequence's rows by the attention weight that they have received.
//
// evict_select: one block a sequence and KV head picks the `keep` rows that stay: the first
// `first` and the last `last` rows, and of the others the heaviest, the lower row first
// among equal ones. Weights count as max(w, 0) (NaN as 0), so their bits order them;
// the least bits T that still stay are found digit by digit (11, 11 and 10 bits, from the
// top) from histograms of the rows that agree with T so far. Then each warp counts its run of
// rows above T and equal to T, one scan over the warps places them, and the kept rows are
// written in ascending order. The weights are read once into shared memory (the first
// CACHED of a head) and four times from there.
// evict_gather: copies the kept rows of k and v, 16 bytes an item, in the order of the
// output, and zeros behind a sequence's last one.
#include "internal.h"

namespace sattn {
namespace {

constexpr int SELECT = 1024, CACHED = 16384, BINS = 2048;
constexpr int GATHER = 256, AHEAD = 4;

struct SelectSmem {
    uint32_t w[CACHED];
    int bins[BINS];
    int warp_gt[32], warp_eq[32];
    int digit, above;
};

__device__ __forceinline__ uint32_t order_bits(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

// Which bin, counted from the top, holds the k-th row (k >= 1)? `above`: rows in higher bins.
// The whole block; ends with a barrier.
__device__ __forceinline__ void find_bin(SelectSmem &sm, int nbins, int k) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // thread i holds bins top - 2 i and top - 2 i - 1
    const int hi = nbins - 1 - 2 * threadIdx.x;
    const int a = hi >= 0 ? sm.bins[hi] : 0, b = hi >= 1 ? sm.bins[hi - 1] : 0;
    int inc = a + b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) sm.warp_gt[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int v = sm.warp_gt[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        sm.warp_eq[lane] = v;
    }
    __syncthreads();
    const int before = (warp ? sm.warp_eq[warp - 1] : 0) + inc - a - b;
    if (before < k && k <= before + a) {
        sm.digit = hi;
        sm.above = before;
    } else if (before + a < k && k <= before + a + b) {
        sm.digit = hi - 1;
        sm.above = before + a;
    }
    __syncthreads();
}

__global__ void __launch_bounds__(SELECT, 1) evict_select_kernel(EvictArgs a, DevCtx ctx) {
    extern __shared__ __align__(16) uint8_t raw[];
    SelectSmem &sm = *reinterpret_cast<SelectSmem *>(raw);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int start = __ldg(a.kv_starts + b);
    int len = __ldg(a.kv_lens + b);
    if (start < 0 || len < 0 || (long long)start + len > a.S) {
        if (tid == 0) record_error(ctx, DEVERR_SEQLENS);
        len = 0;
    }
    const float *w = a.weights + (size_t)h * a.S + start;
    const size_t out = (size_t)h * a.B * a.keep + (size_t)b * a.keep;
    int32_t *rows = a.rows_out + out;
    float *wout = a.weights_out + out;
    const int kept = min(len, a.keep);
    if (h == 0 && tid == 0) {
        a.out_starts[b] = b * a.keep;
        a.out_lens[b] = kept;
    }
    for (int i = kept + tid; i < a.keep; i += SELECT) {
        rows[i] = -1;
        wout[i] = 0.f;
    }
    if (len <= a.keep) {
        for (int i = tid; i < len; i += SELECT) {
            rows[i] = i;
            wout[i] = __ldg(w + i);
        }
        return;
    }
    const int lo = a.first, hi = len - a.last;  // the rows that compete
    int need = a.keep - a.first - a.last;       // of which so many stay; fewer than there are
    auto bits = [&](int i) { return i < CACHED ? sm.w[i] : order_bits(__ldg(w + i)); };
    for (int i0 = tid; i0 < min(len, CACHED); i0 += 4 * SELECT) {
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[u] = i0 + u * SELECT < len ? __ldg(w + i0 + u * SELECT) : 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + u * SELECT < min(len, CACHED)) sm.w[i0 + u * SELECT] = order_bits(x[u]);
    }
    uint32_t T = 0xffffffffu;  // nothing is above it
    if (need > 0) {
        T = 0;
        constexpr int SHIFT[3] = {21, 10, 0}, WIDTH[3] = {11, 11, 10};
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            const int shift = SHIFT[d], nbins = 1 << WIDTH[d], top = shift + WIDTH[d];
            for (int i = tid; i < nbins; i += SELECT) sm.bins[i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += SELECT) {
                const uint32_t x = bits(i);
                if (top == 32 || x >> top == T >> top) atomicAdd(&sm.bins[x >> shift & (nbins - 1)], 1);
            }
            __syncthreads();
            find_bin(sm, nbins, need);
            T |= (uint32_t)sm.digit << shift;
            need -= sm.above;
        }
    }
    __syncthreads();
    // `need` of the rows equal to T stay, the lowest ones; warp i has a run of rows
    const int per = ((len + 31) / 32 + 31) & ~31, from = min(len, warp * per), to = min(len, from + per);
    auto flags = [&](int i, bool &gt, bool &eq) {
        const bool in = i < to;
        const uint32_t x = in ? bits(i) : 0;
        const bool always = i < lo || i >= hi;
        gt = in && (always || x > T);
        eq = in && !always && x == T;
    };
    int ngt = 0, neq = 0;
    for (int i = from + lane; i - lane < to; i += 32) {
        bool gt, eq;
        flags(i, gt, eq);
        ngt += __popc(__ballot_sync(0xffffffffu, gt));
        neq += __popc(__ballot_sync(0xffffffffu, eq));
    }
    if (lane == 0) {
        sm.warp_gt[warp] = ngt;
        sm.warp_eq[warp] = neq;
    }
    __syncthreads();
    int gt0 = 0, eq0 = 0;
    for (int i = 0; i < warp; ++i) {
        gt0 += sm.warp_gt[i];
        eq0 += sm.warp_eq[i];
    }
    const unsigned below = (1u << lane) - 1;
    for (int i = from + lane; i - lane < to; i += 32) {
        bool gt, eq;
        flags(i, gt, eq);
        const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        const int g = gt0 + __popc(mg & below), q = eq0 + __popc(me & below);
        if (gt || (eq && q < need)) {
            const int at = g + min(q, need);
            rows[at] = i;
            wout[at] = __ldg(w + i);
        }
        gt0 += __popc(mg);
        eq0 += __popc(me);
    }
}

// UNITS: 16-byte units a row.
template <int UNITS> __global__ void __launch_bounds__(GATHER) evict_gather_kernel(EvictArgs a, long long rows) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // an item: 16 bytes of a kept row's key and of its value
    const long long items = rows * UNITS;
    const long long i0 = (long long)blockIdx.x * (GATHER * AHEAD) + threadIdx.x;
    const int64_t ks = a.k_stride / (16 / a.elem), vs = a.v_stride / (16 / a.elem);
    const size_t slots = (size_t)a.B * a.keep;
    uint4 x[AHEAD], y[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
        const long long i = i0 + u * GATHER;
        x[u] = y[u] = make_uint4(0, 0, 0, 0);
        if (i >= items) continue;
        const long long row = i / UNITS;  // slot, head
        const int c = (int)(i % UNITS);
        const long long slot = row / a.Hkv;
        const int h = (int)(row % a.Hkv), b = (int)(slot / a.keep);
        const int at = a.rows_out[(size_t)h * slots + slot];
        if (at < 0) continue;
        const size_t src = (size_t)__ldg(a.kv_starts + b) + at;
        x[u] = __ldg(static_cast<const uint4 *>(a.k) + src * ks + h * UNITS + c);
        y[u] = __ldg(static_cast<const uint4 *>(a.v) + src * vs + h * UNITS + c);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
        const long long i = i0 + u * GATHER;
        if (i >= items) continue;
        static_cast<uint4 *>(a.k_out)[i] = x[u];
        static_cast<uint4 *>(a.v_out)[i] = y[u];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, const DevInfo &dev, cudaStream_t s) {
    cudaError_t e = ensure_smem_attr((const void *)evict_select_kernel, sizeof(SelectSmem), dev);
    if (e != cudaSuccess) return e;
    evict_select_kernel<<<(unsigned)(a.B * a.Hkv), SELECT, sizeof(SelectSmem), s>>>(a, make_ctx(dev));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.B * a.keep * a.Hkv;
    const int units = a.d * a.elem / 16;
    const long long per = GATHER * AHEAD;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows * units + per - 1) / per));
    cfg.blockDim = dim3(GATHER);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (units == 8) return cudaLaunchKernelEx(&cfg, evict_gather_kernel<8>, a, rows);
    if (units == 16) return cudaLaunchKernelEx(&cfg, evict_gather_kernel<16>, a, rows);
    return cudaLaunchKernelEx(&cfg, evict_gather_kernel<32>, a, rows);
}

}  // namespace sattn
