// Eviction of a sequence's rows by the attention weight that they have received.
//
// evict_select: one block a sequence and KV head picks the `keep` rows that stay: the first
// `first` and the last `last` rows, and of the others the heaviest, the lower row first
// among equal ones. Weights count as max(w, 0) (NaN as 0), so their bits order them;
// the least bits T that still stay are found from histograms of the range that they can lie in,
// in 2048 parts, until a part is one number: three rounds at most, of which the later ones
// count few rows. Then each warp counts its run of rows above T
// and equal to T, one scan over the warps places them, and the kept rows are written in
// ascending order. The first CACHED weights of a head are read once into shared memory, and in two
// to five passes from there (the rounds, the counting, the placing); those behind it come from
// global memory in every pass, and a kept row's weight once more when it is written.
// Bound by instructions over few SMs (16000 rows: 16 us, two blocks an SM): load 4 us, the rounds 4,
// the placing 4; digits of the bits as bins 30.
// evict_gather: copies the kept rows of k and v, 16 bytes an item, in the order of the
// output, and zeros behind a sequence's last one. Bound by memory: 64 sequences, 4000 of up to
// 16000 rows of 4 heads kept, d = 64: 82 us for 512 MB, 0.92 of the copy rate.
#include "internal.h"

namespace sattn {
namespace {

constexpr int SELECT = 1024, WARPS = SELECT / 32, CACHED = 16384, LOG_BINS = 11,
              BINS = 1 << LOG_BINS;
constexpr uint32_t ALWAYS = 0xffffffffu;
constexpr int GATHER = 256, AHEAD = 4;

struct SelectSmem {
    alignas(16) uint32_t w[CACHED];
    int bins[BINS];
    int warp_gt[WARPS], warp_eq[WARPS];
    uint32_t warp_most[WARPS];
    int digit, above;
};

__device__ __forceinline__ uint32_t order_bits(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

// Which bin, counted from the top, holds the k-th row (k >= 1)? `above`: rows in higher bins.
// The whole block; the bins are there, and zero behind it.
__device__ __forceinline__ void find_bin(SelectSmem &sm, int k) {
    constexpr int PER = BINS / SELECT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    // thread i holds the bins from top - PER i downwards
    int n[PER], mine = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        n[j] = sm.bins[BINS - 1 - PER * (int)threadIdx.x - j];
        mine += n[j];
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) sm.bins[BINS - 1 - PER * (int)threadIdx.x - j] = 0;
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) sm.warp_gt[warp] = before;
    before -= mine;
    __syncthreads();
    before += __reduce_add_sync(0xffffffffu, lane < warp ? sm.warp_gt[lane] : 0);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (before < k && k <= before + n[j]) {
            sm.digit = BINS - 1 - PER * (int)threadIdx.x - j;
            sm.above = before;
        }
        before += n[j];
    }
    __syncthreads();
}

__global__ void __launch_bounds__(SELECT, 2) evict_select_kernel(EvictArgs a, DevCtx ctx) {
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
    // A row as a number: the weight's bits, more than any weight's for a row that stays anyway.
    auto value = [&](int i, float x) { return i < lo || i >= hi ? ALWAYS : order_bits(x); };
    // f(i, x) with the values of rows i .. i + 3, for the multiples of 4 below len that are this
    // thread's (behind len: 0); a warp's are 128 rows each time, the lanes' in order.
    const int per = ((len + WARPS - 1) / WARPS + 127) & ~127, from = min(len, warp * per),
              to = min(len, from + per);
    auto each = [&](auto f) {
#pragma unroll 2
        for (int i = from + 4 * lane; i - 4 * lane < to; i += 128) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (i + 3 < CACHED) {
                x = *reinterpret_cast<const uint4 *>(sm.w + i);
            } else {
                if (i < to) x.x = value(i, __ldg(w + i));
                if (i + 1 < to) x.y = value(i + 1, __ldg(w + i + 1));
                if (i + 2 < to) x.z = value(i + 2, __ldg(w + i + 2));
                if (i + 3 < to) x.w = value(i + 3, __ldg(w + i + 3));
            }
            const uint32_t v[4] = {x.x, x.y, x.z, x.w};
            f(i, v);
        }
    };
    for (int i = tid; i < BINS; i += SELECT) sm.bins[i] = 0;
    // into shared memory; how many of those that compete are above 0, and their range
    constexpr int U = 8;
    int npos = 0;
    uint32_t least = 0xffffffffu, most = 0;
    for (int i0 = tid; i0 < ((len + 127) & ~127); i0 += U * SELECT) {
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = i0 + u * SELECT < len ? __ldg(w + i0 + u * SELECT) : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * SELECT;
            const uint32_t v = i < len ? value(i, x[u]) : 0;
            if (i < CACHED) sm.w[i] = v;
            if (v - 1 < ALWAYS - 1) {
                ++npos;
                least = min(least, v);
                most = max(most, v);
            }
        }
    }
    npos = __reduce_add_sync(0xffffffffu, npos);
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
        sm.warp_gt[warp] = npos;
        sm.warp_eq[warp] = (int)least;
        sm.warp_most[warp] = most;
    }
    __syncthreads();
    npos = __reduce_add_sync(0xffffffffu, sm.warp_gt[lane]);
    least = __reduce_min_sync(0xffffffffu, (uint32_t)sm.warp_eq[lane]);
    most = __reduce_max_sync(0xffffffffu, sm.warp_most[lane]);
    uint32_t T = 0;
    if (need == 0) {
        T = ALWAYS - 1;  // no weight is above it
    } else if (need > npos) {
        need -= npos;  // so many of those at 0
    } else {
        // the range that T lies in, in BINS parts, until a part is one number
        while (least < most) {
            const int shift = max(0, 32 - __clz(most - least) - LOG_BINS);
            const uint32_t range = most - least;
            __syncthreads();
            each([&](int, const uint32_t(&x)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (x[e] - least <= range) atomicAdd(&sm.bins[(x[e] - least) >> shift], 1);
            });
            find_bin(sm, need);
            need -= sm.above;
            least += (uint32_t)sm.digit << shift;
            most = min(most, least + ((1u << shift) - 1));
        }
        T = least;
    }
    __syncthreads();
    // `need` of the rows equal to T stay, the lowest ones. Rows above T and equal to it
    int ngt = 0, neq = 0;
    each([&](int i, const uint32_t(&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ngt += x[e] > T;
            neq += x[e] == T && i + e < to;
        }
    });
    ngt = __reduce_add_sync(0xffffffffu, ngt);
    neq = __reduce_add_sync(0xffffffffu, neq);
    if (lane == 0) {
        sm.warp_gt[warp] = ngt;
        sm.warp_eq[warp] = neq;
    }
    __syncthreads();
    int gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? sm.warp_gt[lane] : 0);
    int eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? sm.warp_eq[lane] : 0);
    each([&](int i, const uint32_t(&x)[4]) {
        int mine = 0;  // rows above T, and 2^16 times those equal to it
#pragma unroll
        for (int e = 0; e < 4; ++e)
            mine += x[e] > T ? 1 : x[e] == T && i + e < to ? 1 << 16 : 0;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        upto -= mine;
        int g = gt0 + (upto & 0xffff), q = eq0 + (upto >> 16);
        int at[4];
        float kept_w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool gt = x[e] > T, eq = x[e] == T && i + e < to;
            at[e] = gt || (eq && q < need) ? g + min(q, need) : -1;
            if (at[e] >= 0) kept_w[e] = __ldg(w + i + e);
            g += gt;
            q += eq;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (at[e] >= 0) {
                rows[at[e]] = i + e;
                wout[at[e]] = kept_w[e];
            }
        gt0 += all & 0xffff;
        eq0 += all >> 16;
    });
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
