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
// The entry of a cut row: its item's first share (of two an SM at most: 10 bits), its tile of the item (0, 1), its row of the
// 128, and its parts.
__device__ __forceinline__ float cut_row(int share, int tile, int row, int parts) {
    return __uint_as_float(((uint32_t)share << 22) | ((uint32_t)tile << 21) | ((uint32_t)row << 14) | (uint32_t)parts);
}
// And where its parts are (state_ml and state_u of paged_tc_sm103.cu).
struct CutRow {
    int share, tile, row, n;
    __device__ __forceinline__ void set(const Args &a, float entry) {
        const uint32_t e = __float_as_uint(entry);
        share = (int)(e >> 22);
        tile = (int)(e >> 21) & 1;
        row = (int)(e >> 14) & 127;
        n = (int)e & 0x3fff;
        // (an entry that no call over these prefixes has written, where cu decreases)
        if (share + n > a.state.shares || tile >= a.state.tiles) n = 0;
    }
    __device__ __forceinline__ long long place(const Args &a, int p) const {
        return (long long)state_slot(share + p, share) * a.state.tiles + tile;
    }
    __device__ __forceinline__ float2 ml(const Args &a, int p) const {
        return __ldcg(reinterpret_cast<const float2 *>(a.state.part_ml) + place(a, p) * 128 + row);
    }
    // its first columns, in float4; the next four 128 further
    template <int D>
    __device__ __forceinline__ const float4 *u(const Args &a, int p) const {
        return reinterpret_cast<const float4 *>(a.state.part_u) + place(a, p) * (128 * D / 4) + row;
    }
    // (m, l) of all parts
    __device__ __forceinline__ float2 joined(const Args &a) const {
        float m = -INFINITY, l = 0.f;
        for (int p = 0; p < n; ++p) m = fmaxf(m, ml(a, p).x);
        const float ref = m == -INFINITY ? 0.f : m;
        for (int p = 0; p < n; ++p) {
            const float2 s = ml(a, p);
            l = fmaf(ptx::ex2(s.x - ref), s.y, l);
        }
        return make_float2(m, l);
    }
    // y = their u of C columns from col on, relative to the maximum m
    template <int D, int C>
    __device__ __forceinline__ void join(const Args &a, int col, float m, float (&y)[C]) const {
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int c = 0; c < C; ++c) y[c] = 0.f;
#pragma unroll 2
        for (int p = 0; p < n; ++p) {
            const float f = ptx::ex2(ml(a, p).x - ref);
            const float4 *src = u<D>(a, p) + col / 4 * 128;
#pragma unroll
            for (int c = 0; c < C / 4; ++c) {
                const float4 x = __ldcg(src + c * 128);
                y[4 * c] = fmaf(f, x.x, y[4 * c]);
                y[4 * c + 1] = fmaf(f, x.y, y[4 * c + 1]);
                y[4 * c + 2] = fmaf(f, x.z, y[4 * c + 2]);
                y[4 * c + 3] = fmaf(f, x.w, y[4 * c + 3]);
            }
        }
    }
};

// A row's end: its state is written (to ml and u), or the earlier one is merged with these weights, to their common
// maximum.
struct Ending {
    float own, before;
    bool written, on;  // on: there is an earlier one
    float2 *ml;
    float *u;
    bool cut;  // it is in parts
    CutRow parts;
    float m;   // its maximum
    bool none; // the row has seen no key here (a weight of 0 is not none: it keeps a NaN)
};
__device__ __forceinline__ bool has_state(const Args &a, int tok) {
    if (!a.state.cu) return true;
    const int c0 = __ldg(a.state.cu), c1 = __ldg(a.state.cu + a.state.P);
    return tok >= c0 && tok < c1;
}
// m and sum become the row's where the earlier state is merged.  kCut: it may be in parts.
template <bool kCut = false>
__device__ __forceinline__ Ending ending(const Args &a, const StateAt &at, int tok, float &m, float &sum) {
    Ending e{1.f, 0.f, a.state.mode == kWritten, false, a.state.ml, a.state.u, false};
    if (a.state.mode < kMerged || !has_state(a, tok)) return e;
    if (a.state.mode == kLeft) {
        e.written = true;
        e.ml = a.state.ml2;
        e.u = a.state.u2;
        return e;
    }
    e.on = true;
    float2 s = __ldcg(a.state.ml + at.ml);
    if (kCut && s.y == kCutRow) {
        e.cut = true;
        e.parts.set(a, s.x);
        s = e.parts.joined(a);
        e.m = s.x;
    }
    const float M = fmaxf(m, s.x), ref = M == -INFINITY ? 0.f : M;
    e.none = sum == 0.f;
    e.own = e.none ? 0.f : ptx::ex2(m - ref);
    e.before = ptx::ex2(s.x - ref);
    sum = fmaf(e.before, s.y, e.none ? 0.f : e.own * sum);
    m = M;
    return e;
}
__device__ __forceinline__ void write_ml(const Ending &e, const StateAt &at, float m, float sum) {
    e.ml[at.ml] = make_float2(sum == 0.f ? -INFINITY : m, sum);
}
// Columns col .. col + C - 1 of u (C even, col a multiple of C or of 4): written, or v becomes the row's.  D > 0: ending<true>.
template <int C, int D = 0>
__device__ __forceinline__ void end_u(const Args &a, const Ending &e, const StateAt &at, int col, float (&v)[C], float sum) {
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
    if (D > 0 && e.cut) {
        if constexpr (D > 0) e.parts.join<D>(a, col, e.m, y);
    } else if constexpr (C % 4 == 0) {
#pragma unroll
        for (int c = 0; c < C; c += 4) *reinterpret_cast<float4 *>(y + c) = __ldcg(u + (col + c) / 4 * at.n);
    } else {
        *reinterpret_cast<float2 *>(y) = __ldcg(reinterpret_cast<const float2 *>(u + col / 4 * at.n) + col / 2 % 2);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = fmaf(e.before, y[c], e.none ? 0.f : e.own * v[c]);
}

// The earlier state of C columns of a row, asked for before it is needed: (m, l) first, then u.  D > 0: it may be in parts.
template <int C, int D = 0>
struct Earlier {
    bool on;
    float2 s;
    float y[C];
    __device__ __forceinline__ void ask_ml(const Args &a, const StateAt &at, int tok, bool row) {
        on = row && has_state(a, tok);
        s = on ? __ldcg(a.state.ml + at.ml) : make_float2(-INFINITY, 0.f);
    }
    __device__ __forceinline__ bool cut() const { return D > 0 && s.y == kCutRow; }
    __device__ __forceinline__ void ask_u(const Args &a, const StateAt &at, int col) {
        const float4 *u = reinterpret_cast<const float4 *>(a.state.u) + at.u + col / 4 * at.n;
#pragma unroll
        for (int c = 0; c < C / 4; ++c)
            *reinterpret_cast<float4 *>(y + 4 * c) = on && !cut() ? __ldcg(u + c * at.n) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // before merge(), for a row in parts
    __device__ __forceinline__ void join_parts(const Args &a, int col) {
        if constexpr (D > 0)
            if (on && cut()) {
                CutRow r;
                r.set(a, s.x);
                s = r.joined(a);
                r.join<D>(a, col, s.x, y);
            }
    }
    // As ending() and end_u().
    __device__ __forceinline__ void merge(float (&v)[C], float &m, float &sum) const {
        if (!on) return;
        const float M = fmaxf(m, s.x), ref = M == -INFINITY ? 0.f : M;
        const bool none = sum == 0.f;  // (a weight of 0 is not none: it keeps a NaN)
        const float own = none ? 0.f : ptx::ex2(m - ref), before = ptx::ex2(s.x - ref);
        sum = fmaf(before, s.y, none ? 0.f : own * sum);
        m = M;
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = fmaf(before, y[c], none ? 0.f : own * v[c]);
    }
};

// Whether a merged row's outputs are the call's to write.
__device__ __forceinline__ bool is_wanted(const Args &a, int tok) {
    if (!a.state.only) return true;
    return tok >= __ldg(a.state.only) && tok < __ldg(a.state.only + a.state.B);
}

// A kernel that merges states reads what the grid before it, the call's first, writes at its very end, and begins while that
// still runs: it waits for it where it needs it, in every CTA.  One that leaves its states needs nothing of it; its first CTA
// waits at its end, since a grid behind this one takes this one's end for that one's.  Their workspaces are different ones.
//
// What else such a kernel reads (lengths, tables, queries, pages) was written by grids before the call's first, whose end only
// that one has waited for: a grid's wait covers the grid right before it.  So the first grid releases the call's tag
// after its wait, and a thread here that acquires the tag has those writes in its past as the first grid has; one that finds
// another value waits for the first grid's end.  Nobody spins.  The tag is taken away at this grid's end: a captured call finds
// none at its next replay.  (64 sequences behind 8192 keys, over boxes, 55 to 57 us, 52 to 55 without.)
__device__ __forceinline__ void begin_after_earlier_grids(const Args &a, bool state) {
    if (!state || a.state.mode < kMerged) {
        ptx::grid_dep_wait();
        if (state && a.state.mode == kWritten && blockIdx.x == 0 && threadIdx.x == 0) ptx::store_release(a.state.begun, a.state.tag);
        return;
    }
    if (ptx::load_acquire(a.state.begun) != a.state.tag) ptx::grid_dep_wait();
    ptx::fence_proxy_async_global();  // pages and queries come by TMA
}
__device__ __forceinline__ void wait_for_states(const Args &a) {
    if (a.state.mode == kMerged) ptx::grid_dep_wait();
}
__device__ __forceinline__ void end_after_earlier_grids(const Args &a) {
    if (a.state.mode == kMerged || (a.state.mode == kLeft && blockIdx.x == 0)) ptx::grid_dep_wait();
    if (a.state.mode >= kMerged && blockIdx.x == 0 && threadIdx.x == 0) *a.state.begun = 0;
}

}  // namespace paged
}  // namespace attn
