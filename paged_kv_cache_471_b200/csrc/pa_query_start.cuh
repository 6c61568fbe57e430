// Which sequence owns a row of a ragged batch.
#pragma once

#include "pa_decode_kernels.cuh"

namespace pa {

// Whether sequence s owns no legal range of the num_tokens rows.
__device__ __forceinline__ bool bad_rows(const int32_t* query_start, int s, int num_tokens) {
    const int a = __ldg(query_start + s), b = __ldg(query_start + s + 1);
    return a < 0 || b < a || b > num_tokens;
}

// The sequence of a row or unit of work: the largest s in [0, S) with first(s)
// <= x, or -1, by a 32-way search of the whole warp.  Should `first` decrease
// somewhere, it is some s in [0, S), and first(s) may be above x.
template <class First>
__device__ __forceinline__ int find_sequence(int S, int lane, First first, int x) {
    int lo = 0, hi = S;
    for (;;) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const unsigned before = __ballot_sync(kFull, i < hi && first(i) <= x);
        if (before == 0) return -1;
        lo += (__popc(before) - 1) * step;
        hi = min(hi, lo + step);
        if (step == 1) return lo;
    }
}

}  // namespace pa
