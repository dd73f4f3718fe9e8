// paged_merge.cuh -- the end of an item whose key tiles fell into several shares.
//
// Every share's 128 threads write their rows' states (m, l, u) to the share's slot and count them;
// whoever completes the count merges ("How Does FlashAttention Preserve Global Softmax Across
// Tiles?", section 3: all parts to the common maximum, then add).  With more than kGroup parts the merge
// goes in two levels, so that no one walks hundreds of parts: the last of every kGroup shares
// merges those into the first one's slot, and the last group merges the groups.  The order of the sums is that
// of the shares in either case.  The parts come from L2, written by other SMs a moment
// ago: the time is latency, so a warp keeps U rows x 4 parts of loads in flight.
#pragma once

#include "paged_sched.cuh"

namespace attn {
namespace paged {

constexpr int kGroup = 24;  // kGroup^2 shares at most

// Counter words of one row tile: a group's is at its first state's slot, an item's at 2 C + c0.
__host__ __device__ constexpr int counter_words(int shares) { return 3 * shares; }

// Merges the states at slots of shares first, first + step, ... (n of them, n <= kGroup), rows
// [row0, row0 + rows) of a slot, rows <= 128.  Four warps, tid 0 .. 127.  To the slot `to`, or, with
// to < 0, to the rows that out(r, &orow, &lse) names.
template <int D, int U, class Out>
__device__ __forceinline__ void merge_parts(const Args &a, int row0, int rows, int c0, int first, int step, int n, int to,
                                            int tid, Out out) {
    constexpr int LR = D / 4, RW = 32 / LR;  // lanes a row (four columns each), rows a warp load
    const int warp = tid >> 5, lane = tid & 31, sub = lane / LR, col = (lane % LR) * 4;
    const int per = (rows + 3) / 4, lo = warp * per, hi = min(rows, lo + per);
    // lane i holds the weights of row lo + i
    float f[kGroup], M = -INFINITY, sum = 0.f;
    {
        const int r = lo + lane;
        float l[kGroup];
#pragma unroll
        for (int p = 0; p < kGroup; ++p) {
            f[p] = -INFINITY;
            l[p] = 0.f;
            if (p < n && r < hi) {
                const long long at = (long long)state_slot(first + p * step, c0) * a.R + row0 + r;
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.ml + at * 2));
                f[p] = ml.x;
                l[p] = ml.y;
            }
        }
#pragma unroll
        for (int p = 0; p < kGroup; ++p) M = fmaxf(M, f[p]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int p = 0; p < kGroup; ++p) {
            f[p] = ptx::ex2(f[p] - ref);
            sum = fmaf(f[p], l[p], sum);
        }
    }
    for (int r0 = lo; r0 < hi; r0 += RW * U) {
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p0 = 0; p0 < kGroup; p0 += 4) {
            if (p0 >= n) break;
            float4 x[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int r = r0 + u * RW + sub;
                    x[u][p] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (r < hi && p0 + p < n) {
                        const long long at = (long long)state_slot(first + (p0 + p) * step, c0) * a.R + row0 + r;
                        x[u][p] = __ldcg(reinterpret_cast<const float4 *>(a.u + at * D + col));
                    }
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float w = __shfl_sync(0xffffffffu, f[p0 + p], (r0 - lo + u * RW + sub) & 31);
                    v[u].x = fmaf(w, x[u][p].x, v[u].x);
                    v[u].y = fmaf(w, x[u][p].y, v[u].y);
                    v[u].z = fmaf(w, x[u][p].z, v[u].z);
                    v[u].w = fmaf(w, x[u][p].w, v[u].w);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * RW + sub, src = (r - lo) & 31;
            const float s = __shfl_sync(0xffffffffu, sum, src), m = __shfl_sync(0xffffffffu, M, src);
            if (r >= hi) continue;
            if (to >= 0) {
                const long long at = (long long)to * a.R + row0 + r;
                *reinterpret_cast<float4 *>(a.u + at * D + col) = v[u];
                if (col == 0) *reinterpret_cast<float2 *>(a.ml + at * 2) = make_float2(m, s);
            } else {
                __nv_bfloat16 *orow;
                float *lse;
                out(r, orow, lse);
                const float inv = s > 0.f ? 1.f / s : 0.f;
                *reinterpret_cast<uint2 *>(orow + col) =
                    s > 0.f ? make_uint2(ptx::pack_bf16x2(v[u].x * inv, v[u].y * inv), ptx::pack_bf16x2(v[u].z * inv, v[u].w * inv))
                            : make_uint2(0u, 0u);
                if (lse && col == 0) *lse = s > 0.f ? (m + log2f(s)) * kLn2 : -INFINITY;
            }
        }
    }
}

// This share's state is written (by these 128 threads): count it, and merge what is complete.
// cnt: the row tile's counter words; sync(): the 128 threads meet (false: gave up).
template <int D, int U, class Sync, class Out>
__device__ __forceinline__ bool finish_cut(const Args &a, unsigned long long *cnt, int shares, int row0, int rows, int share,
                                           int c0, int n, int tid, volatile int *flag, Sync sync, Out out) {
    if (!sync()) return false;
    int step = 1, parts = n;
    if (n > kGroup) {
        const int g = (share - c0) / kGroup, first = c0 + g * kGroup, slot = state_slot(first, c0);
        const int gn = min(kGroup, n - g * kGroup);
        if (tid == 0) *flag = count_state(a, cnt + slot, gn);
        if (!sync()) return false;
        if (!*flag) return true;
        merge_parts<D, U>(a, row0, rows, c0, first, 1, gn, slot, tid, out);
        if (!sync()) return false;
        step = kGroup;
        parts = (n + kGroup - 1) / kGroup;
    }
    if (tid == 0) *flag = count_state(a, cnt + 2 * shares + c0, parts);
    if (!sync()) return false;
    if (*flag) merge_parts<D, U>(a, row0, rows, c0, c0, step, parts, -1, tid, out);
    return true;
}

}  // namespace paged
}  // namespace attn
