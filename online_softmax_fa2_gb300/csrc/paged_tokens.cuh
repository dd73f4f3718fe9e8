// paged_tokens.cuh -- where a packed token of a ragged batch belongs, shared by the kernels that take a
// warp a token.
#pragma once

#include <cuda_runtime.h>

#include "attn_more.h"

namespace attn {

// The sequence of packed token t: the number of entries of cu[1 .. B] that are <= t (cu does not
// decrease), two rounds of 32 probes a warp for up to 1024 sequences.  B when t lies behind the
// last sequence.
__device__ __forceinline__ int find_sequence(const int *cu, int B, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;  // the answer is lo + (entries <= t among cu[lo + 1 .. lo + n])
    while (n > 32) {
        const int step = (n + 31) / 32, at = min((lane + 1) * step, n);
        const int hits = __popc(__ballot_sync(0xffffffffu, __ldg(cu + lo + at) <= t));
        // probes are ordered: the first `hits` of them hold
        const int skip = min(hits * step, n);
        lo += skip;
        n = min(step, n - skip);
        if (hits == 32) return lo;
    }
    const bool le = lane < n && __ldg(cu + lo + 1 + lane) <= t;
    return lo + __popc(__ballot_sync(0xffffffffu, le));
}

// Reports entries of cu that are out of [0, T] or decrease, whatever tokens they belong to: warp `task` of the
// grid looks at 32 entries for every `step` warps, of B in `groups` groups of 32.
__device__ __forceinline__ void report_bad_entries(const int *cu, int B, int T, unsigned task, unsigned groups, unsigned step,
                                                   uint32_t *flags) {
    for (unsigned e = task; e < groups; e += step) {
        const int at = min((int)e * 32 + (int)(threadIdx.x & 31), B - 1);
        const int r0 = __ldg(cu + at), r1 = __ldg(cu + at + 1);
        if (r0 < 0 || r1 < r0 || r1 > T) atomicOr(flags, kFlagBadIndex);
    }
}

// Sequence b of packed token t, its tokens and its place among them; false for a token of no sequence.  The
// sequence's tokens as the attention takes them (seq_info of paged_sched.cuh).  Whole warp.
__device__ __forceinline__ bool find_token(const int *cu, int B, int T, int t, int &b, int &i, int &nq) {
    if (!cu) {
        nq = T / B;
        b = t / nq;
        i = t - b * nq;
        return true;
    }
    b = find_sequence(cu, B, t);
    if (b >= B) return false;  // behind the last sequence
    const int c0 = min(max(__ldg(cu + b), 0), T);
    nq = min(max(__ldg(cu + b + 1), c0), T) - c0;
    i = t - c0;
    return i >= 0 && i < nq;  // else before the first sequence, or cu decreases
}

}  // namespace attn
