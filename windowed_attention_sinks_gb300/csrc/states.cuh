// Encoder states: which queries and which rows of keys and values a sequence has.
#pragma once

#include "common.cuh"

namespace sattn {

// Sequence b: its queries are rows [t0, t0 + n) of q, its states rows [s0, s0 + len) of k and v.
struct StateSeq {
    int t0, n, s0, len;
};

// Loads sequence b and checks it: cu_seqlens starts at 0 and never falls, its rows lie in
// [0, T); its states lie in [0, S). Returns false for a sequence that does not, which is skipped.
__device__ __forceinline__ bool load_states(const int32_t *cu, const int32_t *starts,
                                            const int32_t *lens, int b, int T, int S, StateSeq &s) {
    s.t0 = __ldg(cu + b);
    const int t1 = __ldg(cu + b + 1);
    s.s0 = __ldg(starts + b);
    s.len = __ldg(lens + b);
    s.n = t1 - s.t0;
    return __ldg(cu) == 0 && s.t0 >= 0 && t1 >= s.t0 && t1 <= T && s.s0 >= 0 && s.len >= 0 &&
           (long long)s.s0 + s.len <= S;
}

// A sink in log2 units. The largest finite values stay finite, at a number that
// fp32's factors ln 2 and log2 e take to an lse and back to itself: a row that a sink decides has
// this lse, and its one key the weight 2^0. (So do all smaller sinks that decide a row: checked
// for every mantissa.)
__device__ __forceinline__ float state_sink(float s) {
    return isinf(s) ? s : fminf(fmaxf(s * LOG2E, -2.9999998e38f), 2.9999998e38f);
}

}  // namespace sattn
