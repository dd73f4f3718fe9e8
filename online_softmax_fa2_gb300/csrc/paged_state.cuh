// paged_state.cuh -- the states (m, l, u) of packed tokens' rows that go from the attention over a shared
// prefix to the attention over the sequences' own keys ("How Does FlashAttention Preserve Global Softmax Across
// Tiles?", section 3: over disjoint key sets, all to the common maximum, then add).
#pragma once

#include "paged_sched.cuh"

namespace attn {
namespace paged {

// Row `row` (token * G + head of the group) of key head hk.
struct StateAt {
    long long ml, u, n;  // its index in ml; of its first four columns in u (in float4); rows of a key head
};
__device__ __forceinline__ StateAt state_at(const Args &a, int D, int hk, long long row) {
    const long long n = (long long)a.T * a.G;
    return StateAt{hk * n + row, hk * (D / 4) * n + row, n};
}
__device__ __forceinline__ void write_state_ml(const Args &a, const StateAt &at, float m, float sum) {
    a.state.ml[at.ml] = make_float2(sum == 0.f ? -INFINITY : m, sum);
}
// Columns col .. col + C - 1 of u (C even, col a multiple of C or of 4).
template <int C>
__device__ __forceinline__ void write_state(const Args &a, const StateAt &at, int col, const float (&v)[C], float sum) {
    const bool empty = sum == 0.f;  // its u is 0, whatever 0 times a value was
    float4 *u = reinterpret_cast<float4 *>(a.state.u) + at.u;
    if constexpr (C % 4 == 0) {
#pragma unroll
        for (int c = 0; c < C; c += 4)
            u[(col + c) / 4 * at.n] = empty ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
    } else {
        reinterpret_cast<float2 *>(u + col / 4 * at.n)[col / 2 % 2] = empty ? make_float2(0.f, 0.f) : make_float2(v[0], v[1]);
    }
}

// The weights of a row's own state and of its earlier one, to their common maximum; m and sum become the row's.
struct Weights {
    float own, before;
    bool on;  // there is an earlier one
};
__device__ __forceinline__ Weights join_ml(const Args &a, const StateAt &at, int tok, float &m, float &sum) {
    int c0 = 0, c1 = a.T;
    if (a.state.cu) {
        c0 = min(max(__ldg(a.state.cu), 0), a.T);
        c1 = min(max(__ldg(a.state.cu + a.state.P), 0), a.T);
    }
    Weights w{1.f, 0.f, tok >= c0 && tok < c1};
    if (!w.on) return w;
    const float2 s = __ldcg(a.state.ml + at.ml);
    const float M = fmaxf(m, s.x), ref = M == -INFINITY ? 0.f : M;
    w.own = sum == 0.f ? 0.f : ptx::ex2(m - ref);
    w.before = ptx::ex2(s.x - ref);
    sum = fmaf(w.before, s.y, sum == 0.f ? 0.f : w.own * sum);
    m = M;
    return w;
}
template <int C>
__device__ __forceinline__ void join_u(const Args &a, const StateAt &at, int col, const Weights &w, float (&v)[C]) {
    if (!w.on) return;
    const float4 *u = reinterpret_cast<const float4 *>(a.state.u) + at.u;
    float y[C];
    if constexpr (C % 4 == 0) {
#pragma unroll
        for (int c = 0; c < C; c += 4) *reinterpret_cast<float4 *>(y + c) = __ldcg(u + (col + c) / 4 * at.n);
    } else {
        *reinterpret_cast<float2 *>(y) = __ldcg(reinterpret_cast<const float2 *>(u + col / 4 * at.n) + col / 2 % 2);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = fmaf(w.before, y[c], w.own == 0.f ? 0.f : w.own * v[c]);
}
// Both, for C columns of a row.
template <int C>
__device__ __forceinline__ void join(const Args &a, const StateAt &at, int tok, int col, float (&v)[C], float &m, float &sum) {
    const Weights w = join_ml(a, at, tok, m, sum);
    join_u<C>(a, at, col, w, v);
}

// A kernel that merges states reads what the call before it writes at its very end, and begins while that one still
// runs: it waits for it here, in every CTA (a grid behind this one takes this one's end for that one's), and its
// workspace is another.  What else it reads was there before that call began: its kernels let this one start after their
// own wait.
__device__ __forceinline__ void begin_after_earlier_grids(const Args &a, bool state) {
    if (!state || a.state.mode != kMerged) ptx::grid_dep_wait();
}
__device__ __forceinline__ void wait_for_states(const Args &a) {
    if (a.state.mode == kMerged) ptx::grid_dep_wait();
}

}  // namespace paged
}  // namespace attn
