// paged_merge.cuh -- the end of an item whose key tiles fell into several shares.
//
// Every share's 128 threads write their rows' states (m, l, u) to the share's slot, mark the slot as
// written and look whether all marks of the item are there; who sees them all merges ("How Does
// FlashAttention Preserve Global Softmax Across Tiles?", section 3: all parts to the common
// maximum, then add), in share order, whoever it is.  A mark is a word of its own (a counter of the
// item made the shares, which end together, queue up: 17 us for 24 of them); between writing its
// mark and reading the others' a thread fences, so the last to write sees all.  Marks hold the
// call's tag; any other value is no mark, and they are taken away before the merge: the workspace
// may hold anything on entry, and a captured call, whose tag is the same at every replay,
// finds none.
//
// With more than kGroup parts the merge goes in two levels, so that no one walks hundreds of
// parts: every kGroup shares are merged into a slot of the group's own, then the groups.  The parts come
// from L2, written by other SMs a moment ago: the time is latency, so a warp keeps
// many of them in flight.
#pragma once

#include <type_traits>

#include "paged_sched.cuh"

namespace attn {
namespace paged {

constexpr int kGroup = 64;  // parts one merge takes (two a lane); kGroup^2 shares at most

// A group of an item with more than kGroup parts begins at share c0 + kGroup g.  Its slot and mark:
// of the groups that begin in one window of kGroup shares, one at most is its item's first, and
// one at most is not (two items of more than kGroup parts do not begin that near to each other).
__host__ __device__ constexpr int group_slots(int shares) { return 2 * (shares / kGroup + 1); }
__device__ __forceinline__ int group_slot(int first, int g) { return 2 * (first / kGroup) + (g == 0 ? 1 : 0); }
// Slots of states, and marks of one row tile: the shares', then the groups'.
__host__ __device__ constexpr int all_slots(int shares) { return 2 * shares + group_slots(shares); }

// Marks word `mine` as written (the 128 threads have met since the writes) and looks whether words
// word(0) .. word(n - 1), n <= kGroup, are all marked; takes them away if so.  True, for all 128
// threads (through *flag), in one share only.
template <class Sync, class Word>
__device__ __forceinline__ bool all_marked(const Args &a, unsigned long long *marks, int mine, int n, int tid, volatile int *flag,
                                           Sync sync, Word word, bool &ok) {
    if (tid < 32) {
        if (tid == 0) {
            __threadfence();  // the states before the mark
            *reinterpret_cast<volatile unsigned long long *>(marks + mine) = a.tag;
        }
        __syncwarp();
        __threadfence();  // this mark before the others are read
        volatile unsigned long long *w0 = marks + word(tid < n ? tid : 0), *w1 = marks + word(tid + 32 < n ? tid + 32 : 0);
        const unsigned long long x0 = *w0, x1 = *w1;
        bool all = __all_sync(0xffffffffu, x0 == a.tag && x1 == a.tag);
        if (all) {
            __threadfence();  // the marks before the states
            // several may see them all: the one that takes the first mark away merges
            if (tid == 0) all = atomicExch(marks + word(0), 0ull) == a.tag;
            else if (tid < n) *w0 = 0ull;
            if (tid + 32 < n) *w1 = 0ull;
        }
        if (tid == 0) *flag = all;
    }
    ok = sync();
    return ok && *flag;
}

// The merge for few rows: the states at slots slot(0) .. slot(n - 1), n <= kGroup, u as [slot][R][D],
// to the slot `to`, or, with to < 0, to the rows that out(r, orow, lse) names.  Four warps, tid 0 ..
// 127, a row a warp at a time (U of them in flight); of a row's states, lane p holds the weights
// of p and p + 32.
template <int D, int U, int P, class Slot, class Out>
__device__ __forceinline__ void merge_parts(const Args &a, int rows, int n, int to, int tid, Slot slot, Out out) {
    constexpr int C = D / 32;  // columns a lane: C lane .. C lane + C - 1
    using Vec = typename std::conditional<C == 4, float4, float2>::type;
    const int warp = tid >> 5, lane = tid & 31;
    const int per = (rows + 3) / 4, lo = warp * per, hi = min(rows, lo + per);
    const int s0 = lane < n ? slot(lane) : 0, s1 = lane + 32 < n ? slot(lane + 32) : 0;
#pragma unroll 1
    for (int r0 = lo; r0 < hi; r0 += U) {
        float2 w0[U], w1[U];
        float v[U][C];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = min(r0 + u, hi - 1);  // a row past the warp's last is read again
            w0[u] = w1[u] = make_float2(-INFINITY, 0.f);
            if (lane < n) w0[u] = __ldcg(reinterpret_cast<const float2 *>(a.ml + (s0 * (long long)a.R + r) * 2));
            if (lane + 32 < n) w1[u] = __ldcg(reinterpret_cast<const float2 *>(a.ml + (s1 * (long long)a.R + r) * 2));
#pragma unroll
            for (int e = 0; e < C; ++e) v[u][e] = 0.f;
        }
        float M[U], sum[U];
#pragma unroll 1
        for (int p0 = 0; p0 < n; p0 += P) {
            Vec x[U][P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int q = min(p0 + p, n - 1), sl = __shfl_sync(0xffffffffu, q < 32 ? s0 : s1, q & 31);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    x[u][p] = __ldcg(reinterpret_cast<const Vec *>(
                        a.u + (sl * (long long)a.R + min(r0 + u, hi - 1)) * D + C * lane));
            }
            if (p0 == 0) {  // the weights, under the first states' loads
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float m = fmaxf(w0[u].x, w1[u].x);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                    M[u] = m;
                    const float ref = m == -INFINITY ? 0.f : m;
                    w0[u].x = ptx::ex2(w0[u].x - ref);
                    w1[u].x = ptx::ex2(w1[u].x - ref);
                    float s = fmaf(w0[u].x, w0[u].y, w1[u].x * w1[u].y);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                    sum[u] = s;
                }
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int q = p0 + p;
                if (q >= n) break;  // the whole warp
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float w = __shfl_sync(0xffffffffu, q < 32 ? w0[u].x : w1[u].x, q & 31);
                    const float *xs = reinterpret_cast<const float *>(&x[u][p]);
#pragma unroll
                    for (int e = 0; e < C; ++e) v[u][e] = fmaf(w, xs[e], v[u][e]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u;
            if (r >= hi) break;  // the whole warp
            if (to >= 0) {
                const long long at = (long long)to * a.R + r;
                Vec y;
#pragma unroll
                for (int e = 0; e < C; ++e) reinterpret_cast<float *>(&y)[e] = v[u][e];
                *reinterpret_cast<Vec *>(a.u + at * D + C * lane) = y;
                if (lane == 0) *reinterpret_cast<float2 *>(a.ml + at * 2) = make_float2(M[u], sum[u]);
            } else {
                __nv_bfloat16 *orow;
                float *lse;
                out(r, orow, lse);
                const bool empty = sum[u] == 0.f;  // (a part whose sum is NaN makes it NaN, whatever its weight)
                const float inv = empty ? 0.f : 1.f / sum[u];
                uint32_t *o32 = reinterpret_cast<uint32_t *>(orow + C * lane);
#pragma unroll
                for (int e = 0; e < C; e += 2) o32[e / 2] = empty ? 0u : ptx::pack_bf16x2(v[u][e] * inv, v[u][e + 1] * inv);
                if (lse && lane == 0) *lse = empty ? -INFINITY : (M[u] + log2f(sum[u])) * kLn2;
            }
        }
    }
}

// This share's state is written (by these 128 threads): mark it, and merge what is complete, by
// merge(n, to, slot).  marks: the row tile's; sync(): the 128 threads meet (false: gave up).
template <class Sync, class Merge>
__device__ __forceinline__ bool finish_cut(const Args &a, unsigned long long *marks, int shares, int share, int c0, int n,
                                           int tid, volatile int *flag, Sync sync, Merge merge) {
    const int g = (share - c0) / kGroup, base = 2 * shares;
    bool groups = n > kGroup;  // first the shares of a group, then the groups
    int mine = state_slot(share, c0);
    auto slot = [&](int p) {
        return n <= kGroup ? state_slot(c0 + p, c0)
               : groups    ? state_slot(c0 + g * kGroup + p, c0)
                           : base + group_slot(c0 + p * kGroup, p);
    };
#pragma unroll 1
    for (;;) {
        const int parts = n <= kGroup ? n : groups ? min(kGroup, n - g * kGroup) : (n + kGroup - 1) / kGroup;
        bool ok = sync();
        if (!ok) return false;
        const bool all = all_marked(a, marks, mine, parts, tid, flag, sync, slot, ok);
        if (!all) return ok;
        const int to = groups ? base + group_slot(c0 + g * kGroup, g) : -1;
        merge(parts, to, slot);
        if (!groups) return true;
        groups = false;
        mine = to;
    }
}

}  // namespace paged
}  // namespace attn
