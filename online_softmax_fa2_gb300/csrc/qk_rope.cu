// qk_rope.cu -- RMS norm of every query and key head with the position rotation in one pass,
// its gradients, and the same pass writing keys and values to their slots of a paged cache.
//
//   r = 1 / sqrt(mean_c x_c^2 + eps),   n_c = x_c r,   t_c = w_c n_c
//   y_a = t_a cos - t_b sin,  y_b = t_a sin + t_b cos   for the pairs (a, b) of the first rot
//   dimensions; the others pass through.  The rotation is orthogonal, so going back
//   dt = R^T dy;  dw_c = sum over rows dt_c n_c;  g_c = w_c dt_c;  dx_c = r (g_c - n_c mean_j g_j n_j).
//
// The bound is memory: a row is read once and written once (backward: two reads, one write), so
// everything between happens in registers.  A row belongs to a group of L lanes, each holding two
// 8-element chunks: chunk p and chunk p + rot/16 for p < rot/16 (the two halves of the rotated
// part, so that both members of every pair lie in one lane in either pairing), and two
// neighbouring chunks of the part that is not rotated otherwise.  The row's sum of squares takes
// log2 L shuffles.  A warp stays with one token, whose angles it holds in registers while it
// walks the heads.  Sums, norms and angles are fp32; an output is rounded once.
#include <cuda_bf16.h>

#include "attn_internal.h"
#include "qk_rope.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// 16 bytes past L1 (each is read once); not .nc, since an output may be the input itself.
__device__ __forceinline__ uint4 ld16_rw(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// Eight elements as they lie in memory.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = ld16_rw(p); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float *f) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f[2 * t] = __uint_as_float(w[t] << 16);
            f[2 * t + 1] = __uint_as_float(w[t] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float *f) {
        v = make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                       ptx::pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Chunk<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = ld16_rw(p);
        b = ld16_rw(p + 4);
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<uint4 *>(p)[0] = a;
        reinterpret_cast<uint4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float *f) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = __uint_as_float(w[t]);
    }
    __device__ __forceinline__ void set(const float *f) {
        a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    }
};

template <typename T>
struct Row2 {  // a lane's two chunks of a row
    Chunk<T> c[2];
    __device__ __forceinline__ void load(const T *row, int e0, int e1, bool on) {
        if (on) {
            c[0].load(row + e0);
            c[1].load(row + e1);
        } else {
            c[0].zero();
            c[1].zero();
        }
    }
    __device__ __forceinline__ void store(T *row, int e0, int e1) const {
        c[0].store(row + e0);
        c[1].store(row + e1);
    }
    __device__ __forceinline__ void get(float (&f)[16]) const {
        c[0].get(f);
        c[1].get(f + 8);
    }
    __device__ __forceinline__ void set(const float (&f)[16]) {
        c[0].set(f);
        c[1].set(f + 8);
    }
};

// Where a lane's two chunks lie, and the angles that turn them.
struct Lane {
    int e0, e1;     // first elements of the two chunks
    bool on, turn;  // has chunks (the group may be wider than the row); they are rotated
    float co[8], si[8];
};

template <int L>
__device__ __forceinline__ Lane make_lane(int d, int rot) {
    Lane ln;
    const int p = (threadIdx.x & (L - 1)), rp = rot / 16;
    ln.on = p < d / 16;
    ln.turn = p < rp;
    ln.e0 = ln.turn ? 8 * p : 8 * (2 * rp + 2 * (p - rp));
    ln.e1 = ln.turn ? 8 * (p + rp) : ln.e0 + 8;
    return ln;
}

// The angles of one position: eight pairs a lane.  half split: pair c is (c, c + rot/2), so the
// lane's pairs are 8p .. 8p + 7; adjacent: pair c is (2c, 2c + 1), so they are 4p .. 4p + 3
// (first chunk) and 4 (p + rot/16) .. + 3 (second).
__device__ __forceinline__ void load_angles(Lane &ln, const float *row, int rot, bool inter) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        ln.co[t] = 1.f;
        ln.si[t] = 0.f;
    }
    if (!ln.turn) return;
    const int a = inter ? ln.e0 / 2 : ln.e0, b = inter ? ln.e1 / 2 : ln.e0 + 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int at = s ? b : a;
        const float4 c = __ldg(reinterpret_cast<const float4 *>(row + at));
        const float4 n = __ldg(reinterpret_cast<const float4 *>(row + rot / 2 + at));
        ln.co[4 * s] = c.x; ln.co[4 * s + 1] = c.y; ln.co[4 * s + 2] = c.z; ln.co[4 * s + 3] = c.w;
        ln.si[4 * s] = n.x; ln.si[4 * s + 1] = n.y; ln.si[4 * s + 2] = n.z; ln.si[4 * s + 3] = n.w;
    }
}

// y <- R y (sign 1) or R^T y (sign -1) for the lane's 16 elements.
__device__ __forceinline__ void turn(float (&y)[16], const Lane &ln, bool inter, float sign) {
    if (!inter) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float a = y[t], b = y[8 + t], s = sign * ln.si[t];
            y[t] = fmaf(a, ln.co[t], -b * s);
            y[8 + t] = fmaf(a, s, b * ln.co[t]);
        }
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float a = y[2 * t], b = y[2 * t + 1], s = sign * ln.si[t];
            y[2 * t] = fmaf(a, ln.co[t], -b * s);
            y[2 * t + 1] = fmaf(a, s, b * ln.co[t]);
        }
    }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float sum16(const float (&f)[16]) {
    float s[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t] = (f[t] + f[4 + t]) + (f[8 + t] + f[12 + t]);
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// One kind of head of one token: rows h = first, first + step, ... below hi of a warp's group,
// U of them in flight.  The loop runs alike for all groups (the shuffles need the whole warp).
template <typename T, int L, int U>
__device__ __forceinline__ void norm_rows(const T *in, long long in_h, T *out, long long out_h, const T *w, int lo,
                                          int hi, const Lane &ln, bool inter, int d, float eps) {
    constexpr int GW = 32 / L;
    const int grp = (threadIdx.x & 31) / L;
    float wf[16];
    if (w && ln.on) {
        Row2<T> r;
        r.load(w, ln.e0, ln.e1, true);
        r.get(wf);
    }
    for (int h0 = lo; h0 < hi; h0 += GW * U) {
        Row2<T> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * GW + grp;
            x[u].load(in + h * in_h, ln.e0, ln.e1, ln.on && h < hi);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * GW + grp;
            float f[16];
            x[u].get(f);
            if (w) {
                float q[16];
#pragma unroll
                for (int t = 0; t < 16; ++t) q[t] = f[t] * f[t];
                const float r = rsqrtf(group_sum<L>(sum16(q)) / (float)d + eps);
#pragma unroll
                for (int t = 0; t < 16; ++t) f[t] *= r * wf[t];
            }
            turn(f, ln, inter, 1.f);
            if (ln.on && h < hi) {
                x[u].set(f);
                x[u].store(out + h * out_h, ln.e0, ln.e1);
            }
        }
    }
}

template <typename T, int L, int U>
__device__ __forceinline__ void copy_rows(const T *in, long long in_h, T *out, long long out_h, int lo, int hi,
                                          const Lane &ln) {
    constexpr int GW = 32 / L;
    const int grp = (threadIdx.x & 31) / L;
    for (int h0 = lo; h0 < hi; h0 += GW * U) {
        Row2<T> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * GW + grp;
            x[u].load(in + h * in_h, ln.e0, ln.e1, ln.on && h < hi);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * GW + grp;
            if (ln.on && h < hi) x[u].store(out + h * out_h, ln.e0, ln.e1);
        }
    }
}

// A position clamped into the angle table; one outside is reported.
__device__ __forceinline__ int table_row(long long pos, int P, uint32_t *flags, bool report) {
    if (pos >= 0 && pos < P) return (int)pos;
    if (report && (threadIdx.x & 31) == 0) atomicOr(flags, kFlagBadIndex);
    return pos < 0 ? 0 : P - 1;
}

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

struct RopeArgs {
    int B, N, Hq, Hk, d, rot, inter, P, parts;
    long long tasks;
    float eps;
    const void *q, *k, *wq, *wk;
    void *qo, *ko;
    long long qs[3], ks[3], qos[3], kos[3];
    const float *cs;
    long long cs_row;
    const int *pos;
    long long pos_s[2];
    uint32_t *flags;
};

// Task (token, part): part i of `parts` of the token's query heads and of its key heads.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (task >= a.tasks) return;
    const long long tok = task / a.parts;
    const int part = (int)(task % a.parts);
    const int b = (int)(tok / a.N), n = (int)(tok % a.N);
    Lane ln = make_lane<L>(a.d, a.rot);
    long long pos = n;
    if (a.pos) pos = __ldg(a.pos + b * a.pos_s[0] + n * a.pos_s[1]);
    if (a.rot) load_angles(ln, a.cs + table_row(pos, a.P, a.flags, part == 0) * a.cs_row, a.rot, a.inter);
    else load_angles(ln, nullptr, 0, false);
    // heads [lo, hi) of this part, q and k alike
    const int ql = (int)((long long)a.Hq * part / a.parts), qh = (int)((long long)a.Hq * (part + 1) / a.parts);
    const int kl = (int)((long long)a.Hk * part / a.parts), kh = (int)((long long)a.Hk * (part + 1) / a.parts);
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    norm_rows<T, L, U>(static_cast<const T *>(a.q) + b * a.qs[0] + n * a.qs[1], a.qs[2],
                       static_cast<T *>(a.qo) + b * a.qos[0] + n * a.qos[1], a.qos[2], static_cast<const T *>(a.wq), ql,
                       qh, ln, a.inter, a.d, a.eps);
    norm_rows<T, L, U>(static_cast<const T *>(a.k) + b * a.ks[0] + n * a.ks[1], a.ks[2],
                       static_cast<T *>(a.ko) + b * a.kos[0] + n * a.kos[1], a.kos[2], static_cast<const T *>(a.wk), kl,
                       kh, ln, a.inter, a.d, a.eps);
}

struct AppendArgs {
    int B, T, Hq, Hk, d, rot, inter, P, parts;
    long long tasks;
    float eps;
    const void *q, *k, *v, *wq, *wk;
    void *qo, *kp, *vp;
    long long qs[2], ks[2], vs[2], qos[2], kps[3], vps[3];
    const float *cs;
    long long cs_row;
    const int *pos, *bt, *lens, *cu;
    long long bt_s, pages, page_size, width;
    uint32_t *flags;
};

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a) {
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (task >= a.tasks) return;
    const int t = (int)(task / a.parts), part = (int)(task % a.parts);
    const bool report = part == 0 && (threadIdx.x & 31) == 0;
    int b, i, nq;
    if (a.cu) {
        b = find_sequence(a.cu, a.B, t);
        if (b >= a.B) return;  // behind the last sequence: left as it was
        const int c0 = __ldg(a.cu + b);
        nq = __ldg(a.cu + b + 1) - c0;
        i = t - c0;
        if (i < 0) return;  // before the first sequence: left as it was
        if (i >= nq) {      // cu_q decreases somewhere
            if (report) atomicOr(a.flags, kFlagBadIndex);
            return;
        }
    } else {
        nq = a.T / a.B;
        b = t / nq;
        i = t - b * nq;
    }
    const long long room = a.width * a.page_size;
    const int raw = __ldg(a.lens + b);
    const long long len = raw < 0 ? 0 : raw > room ? room : raw;
    if (report && len != raw) atomicOr(a.flags, kFlagKvLenClamped);
    const long long at = len - nq + i;  // the token's place in its sequence; < 0: it has none
    Lane ln = make_lane<L>(a.d, a.rot);
    if (a.rot) {
        const long long pos = a.pos ? (long long)__ldg(a.pos + t) : max(at, 0ll);
        load_angles(ln, a.cs + table_row(pos, a.P, a.flags, part == 0) * a.cs_row, a.rot, a.inter);
    } else {
        load_angles(ln, nullptr, 0, false);
    }
    const int ql = (int)((long long)a.Hq * part / a.parts), qh = (int)((long long)a.Hq * (part + 1) / a.parts);
    const int kl = (int)((long long)a.Hk * part / a.parts), kh = (int)((long long)a.Hk * (part + 1) / a.parts);
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    norm_rows<T, L, U>(static_cast<const T *>(a.q) + t * a.qs[0], a.qs[1], static_cast<T *>(a.qo) + t * a.qos[0],
                       a.qos[1], static_cast<const T *>(a.wq), ql, qh, ln, a.inter, a.d, a.eps);
    if (at < 0) return;
    const int page = __ldg(a.bt + b * a.bt_s + at / a.page_size);
    if (page < 0 || page >= a.pages) {
        if (report) atomicOr(a.flags, kFlagBadIndex);
        return;
    }
    const long long slot = at % a.page_size;
    norm_rows<T, L, U>(static_cast<const T *>(a.k) + t * a.ks[0], a.ks[1],
                       static_cast<T *>(a.kp) + page * a.kps[0] + slot * a.kps[1], a.kps[2],
                       static_cast<const T *>(a.wk), kl, kh, ln, a.inter, a.d, a.eps);
    copy_rows<T, L, U>(static_cast<const T *>(a.v) + t * a.vs[0], a.vs[1],
                       static_cast<T *>(a.vp) + page * a.vps[0] + slot * a.vps[1], a.vps[2], kl, kh, ln);
}

// ------------------------------------------------------------------------------- backward
//
// Blocks [0, nbq) take the queries' rows and blocks [nbq, nbq + nbk) the keys', so that a thread
// holds the weight gradient of one tensor only.  A block walks tokens; at its end its rows'
// sums go to its own partial, and bwd_weight_kernel adds the partials in a fixed order: the
// weight gradients are the same from run to run.

struct RopeBwdArgs {
    int B, N, d, rot, inter, P, parts, nb[2], H[2];
    float eps;
    const void *x[2], *dy[2], *w[2];
    void *dx[2];
    long long xs[2][3], dys[2][3], dxs[2][3];
    const float *cs;
    long long cs_row;
    const int *pos;
    long long pos_s[2];
    float *part;  // [nb[0] + nb[1], d]
    uint32_t *flags;
};

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_bwd_kernel(const RopeBwdArgs a) {
    constexpr int GW = 32 / L, U = sizeof(T) == 2 ? 2 : 1;
    __shared__ float red[kWarps][L * 16];
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const int s = (int)blockIdx.x >= a.nb[0];
    const int blk = (int)blockIdx.x - (s ? a.nb[0] : 0);
    const int warp = threadIdx.x >> 5, grp = (threadIdx.x & 31) / L;
    const T *w = static_cast<const T *>(a.w[s]);
    Lane ln = make_lane<L>(a.d, a.rot);
    float wf[16], dw[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) wf[t] = dw[t] = 0.f;
    if (w && ln.on) {
        Row2<T> r;
        r.load(w, ln.e0, ln.e1, true);
        r.get(wf);
    }
    const long long tasks = (long long)a.B * a.N * a.parts;
    for (long long task = (long long)blk * kWarps + warp; task < tasks; task += (long long)a.nb[s] * kWarps) {
        const long long tok = task / a.parts;
        const int part = (int)(task % a.parts);
        const int b = (int)(tok / a.N), n = (int)(tok % a.N);
        long long pos = n;
        if (a.pos) pos = __ldg(a.pos + b * a.pos_s[0] + n * a.pos_s[1]);
        if (a.rot) load_angles(ln, a.cs + table_row(pos, a.P, a.flags, part == 0) * a.cs_row, a.rot, a.inter);
        else load_angles(ln, nullptr, 0, false);
        const int lo = (int)((long long)a.H[s] * part / a.parts), hi = (int)((long long)a.H[s] * (part + 1) / a.parts);
        const T *x = static_cast<const T *>(a.x[s]) + b * a.xs[s][0] + n * a.xs[s][1];
        const T *dy = static_cast<const T *>(a.dy[s]) + b * a.dys[s][0] + n * a.dys[s][1];
        T *dx = static_cast<T *>(a.dx[s]) + b * a.dxs[s][0] + n * a.dxs[s][1];
        for (int h0 = lo; h0 < hi; h0 += GW * U) {
            Row2<T> rx[U], rg[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * GW + grp;
                const bool in = ln.on && h < hi;
                if (w) rx[u].load(x + h * a.xs[s][2], ln.e0, ln.e1, in);
                rg[u].load(dy + h * a.dys[s][2], ln.e0, ln.e1, in);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * GW + grp;
                float g[16];
                rg[u].get(g);
                turn(g, ln, a.inter, -1.f);
                if (w) {
                    float f[16], q[16];
                    rx[u].get(f);
#pragma unroll
                    for (int t = 0; t < 16; ++t) q[t] = f[t] * f[t];
                    const float r = rsqrtf(group_sum<L>(sum16(q)) / (float)a.d + a.eps);
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        f[t] *= r;                  // n
                        dw[t] = fmaf(g[t], f[t], dw[t]);
                        g[t] *= wf[t];
                        q[t] = g[t] * f[t];
                    }
                    const float m = group_sum<L>(sum16(q)) / (float)a.d;
#pragma unroll
                    for (int t = 0; t < 16; ++t) g[t] = r * fmaf(-m, f[t], g[t]);
                }
                if (ln.on && h < hi) {
                    rg[u].set(g);
                    rg[u].store(dx + h * a.dxs[s][2], ln.e0, ln.e1);
                }
            }
        }
    }
    if (!w) return;
    // the groups of a warp, then the warps of the block
#pragma unroll
    for (int t = 0; t < 16; ++t) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1) dw[t] += __shfl_xor_sync(0xffffffffu, dw[t], o);
    }
    if (grp == 0 && ln.on) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            red[warp][ln.e0 + t] = dw[t];
            red[warp][ln.e1 + t] = dw[8 + t];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) t += red[k][c];
        a.part[(long long)blockIdx.x * a.d + c] = t;
    }
}

// dw[s][c] = the sum of the partials of tensor s: a block takes 32 columns of one tensor, its 8
// warps every eighth partial.
__global__ void __launch_bounds__(256) bwd_weight_kernel(const float *part, int nb0, int nb1, int d, float *dwq,
                                                         float *dwk) {
    __shared__ float red[8][33];
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const int s = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float *dst = s ? dwk : dwq;
    if (!dst) return;
    const int lo = s ? nb0 : 0, hi = s ? nb0 + nb1 : nb0;
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < d) {
        int i = lo + w;
        for (; i + 24 < hi; i += 32)
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] += part[(long long)(i + 8 * k) * d + c];
        for (; i < hi; i += 8) t[0] += part[(long long)i * d + c];
    }
    red[w][threadIdx.x & 31] = (t[0] + t[1]) + (t[2] + t[3]);
    __syncthreads();
    if (w == 0 && c < d) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v += red[k][threadIdx.x];
        dst[c] = v;
    }
}

void copy3(long long (&d)[3], const int64_t s[3]) {
    for (int i = 0; i < 3; ++i) d[i] = s[i];
}
void copy2(long long (&d)[2], const int64_t s[2]) {
    for (int i = 0; i < 2; ++i) d[i] = s[i];
}

// How many warps share a token: enough for about four warps a scheduler on the whole GPU when
// there are few tokens, but no more than the heads (of the tensor with most) fill a group each.
int token_parts(int64_t tokens, int64_t heads, int L) {
    const int64_t want = 16LL * sm_count(), most = (heads + 32 / L - 1) / (32 / L);
    int64_t p = tokens ? (want + tokens - 1) / tokens : 1;
    p = p < 1 ? 1 : p > most ? most : p;
    return (int)(p < 1 ? 1 : p);
}

int lanes_of(int64_t d) { return d <= 64 ? 4 : d <= 128 ? 8 : 16; }

attn_status_t launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace

int rope_bwd_blocks(int64_t Hq, int64_t Hkv, int64_t tokens, int nb[2]) {
    // both tensors' blocks together fill the GPU several times over (2 x 152 x 4), each tensor's
    // share by its heads; never more blocks than warps of work
    const int64_t most = 8LL * (sm_count() ? sm_count() : 152), H[2] = {Hq, Hkv};
    for (int s = 0; s < 2; ++s) {
        int64_t n = (most * H[s] + (Hq + Hkv) - 1) / (Hq + Hkv);
        const int64_t cap = (tokens * H[s] + kWarps - 1) / kWarps;
        n = n > cap ? cap : n;
        nb[s] = (int)(n < 1 ? 1 : n);
    }
    return nb[0] + nb[1];
}

attn_status_t launch_qk_norm_rope(const attn_qk_norm_rope_params_t &p, cudaStream_t st) {
    RopeArgs a;
    a.B = (int)p.B; a.N = (int)p.N; a.Hq = (int)p.Hq; a.Hk = (int)p.Hkv; a.d = (int)p.d;
    a.rot = p.cos_sin ? (int)p.rot : 0;
    a.inter = p.interleaved; a.P = (int)p.cos_sin_rows; a.eps = p.eps;
    a.q = p.q; a.k = p.k; a.wq = p.wq; a.wk = p.wk; a.qo = p.q_out; a.ko = p.k_out;
    copy3(a.qs, p.q_stride); copy3(a.ks, p.k_stride); copy3(a.qos, p.q_out_stride); copy3(a.kos, p.k_out_stride);
    a.cs = p.cos_sin; a.cs_row = p.cos_sin_stride; a.pos = p.positions; copy2(a.pos_s, p.positions_stride);
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    const int L = lanes_of(p.d);
    const int64_t tokens = p.B * p.N;
    a.parts = token_parts(tokens, p.Hq > p.Hkv ? p.Hq : p.Hkv, L);
    a.tasks = tokens * a.parts;
    const dim3 grid((unsigned)((a.tasks + kWarps - 1) / kWarps));
    const bool h = p.dtype == ATTN_DTYPE_BF16;
    void (*kern)(const RopeArgs) =
        L == 4   ? (h ? qk_norm_rope_kernel<__nv_bfloat16, 4> : qk_norm_rope_kernel<float, 4>)
        : L == 8 ? (h ? qk_norm_rope_kernel<__nv_bfloat16, 8> : qk_norm_rope_kernel<float, 8>)
                 : (h ? qk_norm_rope_kernel<__nv_bfloat16, 16> : qk_norm_rope_kernel<float, 16>);
    return launched(launch_pdl(kern, grid, dim3(kThreads), 0, st, a), "qk_norm_rope");
}

attn_status_t launch_qk_norm_rope_bwd(const attn_qk_norm_rope_bwd_params_t &bp, float *part, cudaStream_t st) {
    const attn_qk_norm_rope_params_t &p = bp.fwd;
    RopeBwdArgs a;
    a.B = (int)p.B; a.N = (int)p.N; a.H[0] = (int)p.Hq; a.H[1] = (int)p.Hkv; a.d = (int)p.d;
    a.rot = p.cos_sin ? (int)p.rot : 0;
    a.inter = p.interleaved; a.P = (int)p.cos_sin_rows; a.eps = p.eps;
    a.x[0] = p.q; a.x[1] = p.k; a.w[0] = p.wq; a.w[1] = p.wk;
    a.dy[0] = bp.dq_out; a.dy[1] = bp.dk_out; a.dx[0] = bp.dq; a.dx[1] = bp.dk;
    copy3(a.xs[0], p.q_stride); copy3(a.xs[1], p.k_stride);
    copy3(a.dys[0], bp.dq_out_stride); copy3(a.dys[1], bp.dk_out_stride);
    copy3(a.dxs[0], bp.dq_stride); copy3(a.dxs[1], bp.dk_stride);
    a.cs = p.cos_sin; a.cs_row = p.cos_sin_stride; a.pos = p.positions; copy2(a.pos_s, p.positions_stride);
    a.part = part;
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    const int L = lanes_of(p.d);
    const int64_t tokens = p.B * p.N;
    const int blocks = rope_bwd_blocks(p.Hq, p.Hkv, tokens, a.nb);
    a.parts = token_parts(tokens, p.Hq > p.Hkv ? p.Hq : p.Hkv, L);
    const bool h = p.dtype == ATTN_DTYPE_BF16;
    void (*kern)(const RopeBwdArgs) =
        L == 4   ? (h ? qk_norm_rope_bwd_kernel<__nv_bfloat16, 4> : qk_norm_rope_bwd_kernel<float, 4>)
        : L == 8 ? (h ? qk_norm_rope_bwd_kernel<__nv_bfloat16, 8> : qk_norm_rope_bwd_kernel<float, 8>)
                 : (h ? qk_norm_rope_bwd_kernel<__nv_bfloat16, 16> : qk_norm_rope_bwd_kernel<float, 16>);
    attn_status_t r = launched(launch_pdl(kern, dim3(blocks), dim3(kThreads), 0, st, a), "qk_norm_rope_bwd");
    if (r || (!bp.dwq && !bp.dwk)) return r;
    return launched(launch_pdl(bwd_weight_kernel, dim3((unsigned)((p.d + 31) / 32), 2), dim3(256), 0, st,
                               (const float *)part, a.nb[0], a.nb[1], (int)p.d, bp.dwq, bp.dwk),
                    "qk_norm_rope_bwd weights");
}

attn_status_t launch_paged_append(const attn_paged_append_params_t &p, cudaStream_t st) {
    AppendArgs a;
    const attn_paged_cache_t &c = p.cache;
    a.B = (int)c.B; a.T = (int)c.T; a.Hq = (int)p.Hq; a.Hk = (int)c.Hkv; a.d = (int)c.d;
    a.rot = p.cos_sin ? (int)p.rot : 0;
    a.inter = p.interleaved; a.P = (int)p.cos_sin_rows; a.eps = p.eps;
    a.q = p.q; a.k = p.k; a.v = p.v; a.wq = p.wq; a.wk = p.wk; a.qo = p.q_out; a.kp = c.k_pages; a.vp = c.v_pages;
    copy2(a.qs, p.q_stride); copy2(a.ks, p.k_stride); copy2(a.vs, p.v_stride); copy2(a.qos, p.q_out_stride);
    copy3(a.kps, c.k_stride); copy3(a.vps, c.v_stride);
    a.cs = p.cos_sin; a.cs_row = p.cos_sin_stride; a.pos = p.positions;
    a.bt = c.block_table; a.bt_s = c.table_stride; a.lens = c.kv_lens; a.cu = c.cu_q;
    a.pages = c.num_pages; a.page_size = c.page_size; a.width = c.table_width;
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    const int L = lanes_of(c.d);
    a.parts = token_parts(c.T, p.Hq > c.Hkv ? p.Hq : c.Hkv, L);
    a.tasks = c.T * a.parts;
    const dim3 grid((unsigned)((a.tasks + kWarps - 1) / kWarps));
    const bool h = c.dtype == ATTN_DTYPE_BF16;
    void (*kern)(const AppendArgs) =
        L == 4   ? (h ? paged_append_kernel<__nv_bfloat16, 4> : paged_append_kernel<float, 4>)
        : L == 8 ? (h ? paged_append_kernel<__nv_bfloat16, 8> : paged_append_kernel<float, 8>)
                 : (h ? paged_append_kernel<__nv_bfloat16, 16> : paged_append_kernel<float, 16>);
    return launched(launch_pdl(kern, grid, dim3(kThreads), 0, st, a), "paged_append");
}

}  // namespace attn
