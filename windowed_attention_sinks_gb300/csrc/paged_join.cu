// Joins the partial results of units that were cut between CTAs (the workspace of the paged
// cache's kernels): w_c = z_c 2^(m_c - m), lse = m + log2 sum_c w_c (+ the
// null-logit sink, once), o = sum_c w_c o_c / sum_c w_c, in the order of the pieces.
//
// A warp takes a row of the unit that a piece boundary cuts, if that boundary is the
// first inside the unit (the others leave). Lane i holds piece i's sums,
// the columns are spread over the lanes. The work is a few MB at most, so it is
// latency that counts: notes, denominators and rows are three rounds of loads. Behind
// 2048 tokens over 8192 keys 17 us by itself under a profiler (36 MB from a cold L2);
// with the rows one after the other it took 600 us.
#include <math.h>

#include "paged_plan.cuh"

namespace sattn {
namespace {

constexpr int THREADS = 256;

template <int D>
__global__ void __launch_bounds__(THREADS)
join_kernel(const uint8_t *ws, int rows, int pieces, int H, int G, const float *sinks,
            int null_sink, __nv_bfloat16 *o, float *lse) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PlanNote *notes = reinterpret_cast<const PlanNote *>(ws);
    const int lane = threadIdx.x & 31;
    const int c = blockIdx.x + 1;  // boundary between pieces c - 1 and c
    const int r = blockIdx.y * (THREADS / 32) + (threadIdx.x >> 5);
    // lane i: piece c + i of the unit is cut off in front; and goes on behind
    const PlanNote me = notes[c];
    if (!me.cont || r >= me.nrows) return;
    const PlanNote prev = notes[c - 1];
    if (prev.cont && prev.through) return;
    int parts = 2;  // the last of c - 1, the first of c, and on while they go through
    for (int i0 = c; me.through; i0 += 32) {
        const bool on = i0 + lane < pieces && notes[i0 + lane].cont && notes[i0 + lane].through;
        const unsigned run = __ballot_sync(0xffffffffu, on);
        const int len = run == 0xffffffffu ? 32 : __ffs(~run) - 1;
        parts += len;
        if (len < 32) break;
    }
    const float2 *sums = reinterpret_cast<const float2 *>(ws + plan_sums_offset());
    const float *prow = reinterpret_cast<const float *>(ws + plan_rows_offset(rows));
    constexpr int E = D / 32;
    // piece i of the unit: part 1 of CTA c - 1, then part 0 of c, c + 1, ...
    auto slot = [&](int i) { return (size_t)(c - 1 + i) * 2 + (i == 0 ? 1 : 0); };
    const int row = me.row0 + r;
    const int head = me.h * G + row % G;
    const size_t out = (size_t)(me.t0 + row / G) * H + head;
    const float sink = null_sink ? sink_log2(__ldg(sinks + head)) : -INFINITY;
    float m = fmaxf(sink, NOTHING);
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, sums[slot(i) * rows + r].x);
    m = warp_max(m);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    auto weight = [&](int i) {
        if (i >= parts) return 0.f;
        const float2 s = sums[slot(i) * rows + r];
        return s.y * ex2(s.x - m);
    };
    const float first = weight(lane);
    float z = ex2(sink - m) + warp_sum(first);  // (0 without a sink)
    for (int i0 = 32; i0 < parts; i0 += 32) z += warp_sum(weight(i0 + lane));
    // the weights over their sum, so that values near fp32's largest do not overflow
    const float inv = z == 0.f ? 0.f : 1.f / z;
    for (int i0 = 0; i0 < parts; i0 += 32) {
        const float w = (i0 == 0 ? first : weight(i0 + lane)) * inv;
        const int cnt = min(32, parts - i0);
#pragma unroll 4
        for (int i = 0; i < cnt; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const float *p = prow + (slot(i0 + i) * rows + r) * D + lane * E;
            if (E == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(p);
                acc[0] += wi * v.x, acc[1] += wi * v.y;
                acc[E - 2] += wi * v.z, acc[E - 1] += wi * v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(p);
                acc[0] += wi * v.x, acc[1] += wi * v.y;
            }
        }
    }
    uint32_t w2[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) w2[e / 2] = pack_bf16x2(acc[e], acc[e + 1]);
    __nv_bfloat16 *dst = o + out * D + lane * E;
    if (E == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w2[0], w2[E / 2 - 1]);
    else *reinterpret_cast<uint32_t *>(dst) = w2[0];
    if (lse && lane == 0) lse[out] = z == 0.f ? -INFINITY : (m + log2f(z)) * LN2;
}

}  // namespace

cudaError_t launch_paged_join(const PagedArgs &a, int rows, int pieces, cudaStream_t s) {
    if (pieces < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pieces - 1), (unsigned)(rows / (THREADS / 32)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const uint8_t *ws = static_cast<const uint8_t *>(a.workspace);
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o);
    const int G = a.H / a.Hkv, null_sink = a.sink_mode == 2;
    return a.d == 64 ? cudaLaunchKernelEx(&cfg, join_kernel<64>, ws, rows, pieces, a.H, G, a.sinks,
                                          null_sink, o, a.lse)
                     : cudaLaunchKernelEx(&cfg, join_kernel<128>, ws, rows, pieces, a.H, G,
                                          a.sinks, null_sink, o, a.lse);
}

}  // namespace sattn
