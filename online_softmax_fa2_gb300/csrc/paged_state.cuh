// paged_state.cuh -- the states (m, l, u) of packed tokens' rows that go from the attention over a shared
// prefix to the attention over the sequences' own keys ("How Does FlashAttention Preserve Global Softmax Across
// Tiles?", section 3: over disjoint key sets, all to the common maximum, then add).
#pragma once

#include "paged_sched.cuh"

namespace attn {
namespace paged {

__device__ __forceinline__ long long state_row(const Args &a, int tok, int h) { return (long long)tok * a.Hq + h; }

__device__ __forceinline__ void write_state_ml(const Args &a, int tok, int h, float m, float sum) {
    a.state.ml[state_row(a, tok, h)] = make_float2(sum == 0.f ? -INFINITY : m, sum);
}
// Columns col .. col + C - 1 of u (C even, 8-byte aligned).
template <int C>
__device__ __forceinline__ void write_state(const Args &a, int tok, int h, int D, int col, const float (&v)[C], float sum) {
    float *to = a.state.u + state_row(a, tok, h) * D + col;
    const bool empty = sum == 0.f;  // its u is 0, whatever 0 times a value was
#pragma unroll
    for (int c = 0; c < C; c += 2) *reinterpret_cast<float2 *>(to + c) = empty ? make_float2(0.f, 0.f) : make_float2(v[c], v[c + 1]);
}

// The weights of a row's own state and of its earlier one, to their common maximum; m and sum become the row's.
struct Weights {
    float own, before;
};
__device__ __forceinline__ Weights join_ml(const Args &a, int tok, int h, float &m, float &sum) {
    int c0 = 0, c1 = a.T;
    if (a.state.cu) {
        c0 = min(max(__ldg(a.state.cu), 0), a.T);
        c1 = min(max(__ldg(a.state.cu + a.state.P), 0), a.T);
    }
    Weights w{1.f, 0.f};
    if (tok < c0 || tok >= c1) return w;
    const float2 s = a.state.ml[state_row(a, tok, h)];
    const float M = fmaxf(m, s.x), ref = M == -INFINITY ? 0.f : M;
    w.own = sum == 0.f ? 0.f : ptx::ex2(m - ref);
    w.before = ptx::ex2(s.x - ref);
    sum = fmaf(w.before, s.y, w.own == 0.f && sum == 0.f ? 0.f : w.own * sum);
    m = M;
    return w;
}
template <int C>
__device__ __forceinline__ void join_u(const Args &a, int tok, int h, int D, int col, const Weights &w, float (&v)[C]) {
    const float *u = a.state.u + state_row(a, tok, h) * D + col;
#pragma unroll
    for (int c = 0; c < C; c += 2) {
        float2 y = make_float2(0.f, 0.f);
        if (w.before != 0.f) y = *reinterpret_cast<const float2 *>(u + c);  // (a NaN weight reads on)
        v[c] = fmaf(w.before, y.x, w.own == 0.f ? 0.f : w.own * v[c]);
        v[c + 1] = fmaf(w.before, y.y, w.own == 0.f ? 0.f : w.own * v[c + 1]);
    }
}
// Both, for C columns of a row.
template <int C>
__device__ __forceinline__ void join(const Args &a, int tok, int h, int D, int col, float (&v)[C], float &m, float &sum) {
    const Weights w = join_ml(a, tok, h, m, sum);
    join_u<C>(a, tok, h, D, col, w, v);
}

}  // namespace paged
}  // namespace attn
