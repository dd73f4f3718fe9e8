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
// A row's end: its state is written (to ml and u), or the earlier one is merged with these weights, to their common
// maximum.
struct Ending {
    float own, before;
    bool written, on;  // on: there is an earlier one
    float2 *ml;
    float *u;
};
__device__ __forceinline__ bool has_state(const Args &a, int tok) {
    if (!a.state.cu) return true;
    const int c0 = __ldg(a.state.cu), c1 = __ldg(a.state.cu + a.state.P);
    return tok >= c0 && tok < c1;
}
// m and sum become the row's where the earlier state is merged.
__device__ __forceinline__ Ending ending(const Args &a, const StateAt &at, int tok, float &m, float &sum) {
    Ending e{1.f, 0.f, a.state.mode == kWritten, false, a.state.ml, a.state.u};
    if (a.state.mode < kMerged || !has_state(a, tok)) return e;
    if (a.state.mode == kLeft) {
        e.written = true;
        e.ml = a.state.ml2;
        e.u = a.state.u2;
        return e;
    }
    e.on = true;
    const float2 s = __ldcg(a.state.ml + at.ml);
    const float M = fmaxf(m, s.x), ref = M == -INFINITY ? 0.f : M;
    e.own = sum == 0.f ? 0.f : ptx::ex2(m - ref);
    e.before = ptx::ex2(s.x - ref);
    sum = fmaf(e.before, s.y, sum == 0.f ? 0.f : e.own * sum);
    m = M;
    return e;
}
__device__ __forceinline__ void write_ml(const Ending &e, const StateAt &at, float m, float sum) {
    e.ml[at.ml] = make_float2(sum == 0.f ? -INFINITY : m, sum);
}
// Columns col .. col + C - 1 of u (C even, col a multiple of C or of 4): written, or v becomes the row's.
template <int C>
__device__ __forceinline__ void end_u(const Ending &e, const StateAt &at, int col, float (&v)[C], float sum) {
    if (e.written) {
        const bool empty = sum == 0.f;  // its u is 0, whatever 0 times a value was
        float4 *u = reinterpret_cast<float4 *>(e.u) + at.u;
        if constexpr (C % 4 == 0) {
#pragma unroll
            for (int c = 0; c < C; c += 4)
                u[(col + c) / 4 * at.n] = empty ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        } else {
            reinterpret_cast<float2 *>(u + col / 4 * at.n)[col / 2 % 2] = empty ? make_float2(0.f, 0.f) : make_float2(v[0], v[1]);
        }
        return;
    }
    if (!e.on) return;
    const float4 *u = reinterpret_cast<const float4 *>(e.u) + at.u;
    float y[C];
    if constexpr (C % 4 == 0) {
#pragma unroll
        for (int c = 0; c < C; c += 4) *reinterpret_cast<float4 *>(y + c) = __ldcg(u + (col + c) / 4 * at.n);
    } else {
        *reinterpret_cast<float2 *>(y) = __ldcg(reinterpret_cast<const float2 *>(u + col / 4 * at.n) + col / 2 % 2);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = fmaf(e.before, y[c], e.own == 0.f ? 0.f : e.own * v[c]);
}

// The earlier state of C columns of a row, asked for before it is needed: (m, l) first, then u.
template <int C>
struct Earlier {
    bool on;
    float2 s;
    float4 y[C / 4];
    __device__ __forceinline__ void ask_ml(const Args &a, const StateAt &at, int tok, bool row) {
        on = row && a.state.mode == kMerged && has_state(a, tok);
        s = on ? __ldcg(a.state.ml + at.ml) : make_float2(-INFINITY, 0.f);
    }
    __device__ __forceinline__ void ask_u(const Args &a, const StateAt &at, int col) {
        const float4 *u = reinterpret_cast<const float4 *>(a.state.u) + at.u + col / 4 * at.n;
#pragma unroll
        for (int c = 0; c < C / 4; ++c) y[c] = on ? __ldcg(u + c * at.n) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // As ending() and end_u().
    __device__ __forceinline__ void merge(float (&v)[C], float &m, float &sum) const {
        if (!on) return;
        const float M = fmaxf(m, s.x), ref = M == -INFINITY ? 0.f : M;
        const float own = sum == 0.f ? 0.f : ptx::ex2(m - ref), before = ptx::ex2(s.x - ref);
        sum = fmaf(before, s.y, own == 0.f ? 0.f : own * sum);
        m = M;
        const float *x = reinterpret_cast<const float *>(y);
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = fmaf(before, x[c], own == 0.f ? 0.f : own * v[c]);
    }
};

// Whether a merged row's outputs are the call's to write.
__device__ __forceinline__ bool is_wanted(const Args &a, int tok) {
    if (!a.state.only) return true;
    return tok >= __ldg(a.state.only) && tok < __ldg(a.state.only + a.state.B);
}

// A kernel that merges states reads what the grids before it write at its very end, and begins while those still run: it
// waits for them where it needs them, in every CTA.  One that leaves its states needs nothing of them; its first CTA waits
// at its end, since a grid behind this one takes this one's end for theirs.  Their workspaces are different ones.  What
// else such a kernel reads was there before those grids began: they let it start after their own wait.
__device__ __forceinline__ void begin_after_earlier_grids(const Args &a, bool state) {
    if (!state || a.state.mode < kMerged) ptx::grid_dep_wait();
}
__device__ __forceinline__ void wait_for_states(const Args &a) {
    if (a.state.mode == kMerged) ptx::grid_dep_wait();
}
__device__ __forceinline__ void end_after_earlier_grids(const Args &a) {
    if (a.state.mode == kMerged || (a.state.mode == kLeft && blockIdx.x == 0)) ptx::grid_dep_wait();
}

}  // namespace paged
}  // namespace attn
