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
// part, so that both members of every pair lie in one lane in either pairing), and likewise one of
// each half of the part that is not rotated otherwise (neighbouring lanes always hold neighbouring
// chunks: with two neighbours a lane there, each load used half of its sectors, and the backward with
// half the head rotated took 49 us for 40).  The row's sum of squares takes
// log2 L shuffles.  Sums, norms and angles are fp32; an output is rounded once.
#include <cuda_bf16.h>

#include "fwd_bf16_common.cuh"
#include "paged_tokens.cuh"
#include "q8.cuh"
#include "qk_rope.h"
#include "sm100_ptx.cuh"
#include "warp_mma.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// (d0, d1) = (a0 * b0, a1 * b1) in one packed instruction
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// 16 bytes; not .nc, since an output may be the input itself.  (Past L1, with L1::no_allocate, a load
// that takes half a line costs the whole line: half the head rotated took 33 us for 27.)
__device__ __forceinline__ uint4 ld16_rw(const void *p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
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

// Where a lane's two chunks lie.
struct Lane {
    int e0, e1;     // first elements of the two chunks
    bool on, turn;  // has chunks (the group may be wider than the row); they are rotated
};

template <int L>
__device__ __forceinline__ Lane make_lane(int d, int rot) {
    Lane ln;
    const int p = (threadIdx.x & (L - 1)), rp = rot / 16;
    ln.on = p < d / 16;
    ln.turn = p < rp;
    ln.e0 = ln.turn ? 8 * p : 8 * (p + rp);
    ln.e1 = ln.turn ? 8 * (p + rp) : 8 * (p + d / 16);
    return ln;
}

// The angles of one position: eight pairs a lane (cos 1 and sin 0 where nothing is rotated).  half
// split: pair c is (c, c + rot/2), so the lane's pairs are 8p .. 8p + 7; adjacent: pair c is
// (2c, 2c + 1), so they are 4p .. 4p + 3 (first chunk) and 4 (p + rot/16) .. + 3 (second).
struct Angles {
    float co[8], si[8];
};
__device__ __forceinline__ Angles load_angles(const Lane &ln, const float *row, int rot, bool inter) {
    Angles an;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        an.co[t] = 1.f;
        an.si[t] = 0.f;
    }
    if (!ln.turn) return an;
    const int a = inter ? ln.e0 / 2 : ln.e0, b = inter ? ln.e1 / 2 : ln.e0 + 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int at = s ? b : a;
        const float4 c = __ldg(reinterpret_cast<const float4 *>(row + at));
        const float4 n = __ldg(reinterpret_cast<const float4 *>(row + rot / 2 + at));
        an.co[4 * s] = c.x; an.co[4 * s + 1] = c.y; an.co[4 * s + 2] = c.z; an.co[4 * s + 3] = c.w;
        an.si[4 * s] = n.x; an.si[4 * s + 1] = n.y; an.si[4 * s + 2] = n.z; an.si[4 * s + 3] = n.w;
    }
    return an;
}

// Of the lane's 16 elements, pair t's are A(t) and B(t): in order (half split: t and 8 + t), or
// neighbours (adjacent: 2t and 2t + 1).  apart() and together() bring the adjacent ones into the
// half split's places and back, so that the arithmetic is the same two-element instructions.
template <bool kInter>
__device__ __forceinline__ void apart(const float (&f)[16], float (&y)[16]) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        y[t] = f[kInter ? 2 * t : t];
        y[8 + t] = f[kInter ? 2 * t + 1 : 8 + t];
    }
}
template <bool kInter>
__device__ __forceinline__ void together(const float (&y)[16], float (&f)[16]) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        f[kInter ? 2 * t : t] = y[t];
        f[kInter ? 2 * t + 1 : 8 + t] = y[8 + t];
    }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// sum of x y over the lane's 16 elements
__device__ __forceinline__ float dot16(const float (&x)[16], const float (&y)[16]) {
    float s[4];
    mul2(s[0], s[1], x[0], x[1], y[0], y[1]);
    mul2(s[2], s[3], x[2], x[3], y[2], y[3]);
#pragma unroll
    for (int t = 4; t < 16; t += 4) {
        ptx::fma2(s[0], s[1], x[t], x[t + 1], y[t], y[t + 1], s[0], s[1]);
        ptx::fma2(s[2], s[3], x[t + 2], x[t + 3], y[t + 2], y[t + 3], s[2], s[3]);
    }
    return (s[0] + s[2]) + (s[1] + s[3]);
}

// d = x y + z, d = x y, d = x c for 8 elements
__device__ __forceinline__ void mul8(float *d, const float *x, const float *y) {
#pragma unroll
    for (int t = 0; t < 8; t += 2) mul2(d[t], d[t + 1], x[t], x[t + 1], y[t], y[t + 1]);
}
__device__ __forceinline__ void fma8(float *d, const float *x, const float *y, const float *z) {
#pragma unroll
    for (int t = 0; t < 8; t += 2) ptx::fma2(d[t], d[t + 1], x[t], x[t + 1], y[t], y[t + 1], z[t], z[t + 1]);
}
__device__ __forceinline__ void scale8(float *d, const float *x, float c) {
#pragma unroll
    for (int t = 0; t < 8; t += 2) mul2(d[t], d[t + 1], x[t], x[t + 1], c, c);
}

// Where a row goes: as T, or as codes and a scale byte.  Called by the whole warp, f the lane's 16 elements
// (zeros without a row), on where it has some to store.
template <typename T>
struct ToRows {
    T *out;
    long long out_h;
    __device__ __forceinline__ void operator()(int u, float (&f)[16], const Lane &ln, bool on) const {
        if (!on) return;
        Row2<T> y;
        y.set(f);
        y.store(out + u * out_h, ln.e0, ln.e1);
    }
};
template <int L>
struct ToCodes {
    uint8_t *out, *scale;
    long long out_h, scale_h;
    __device__ __forceinline__ static float largest(const float (&f)[16]) {  // of the group; a NaN is passed over
        float m = 0.f;
#pragma unroll
        for (int t = 0; t < 16; ++t) m = fmaxf(m, fabsf(f[t]));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    }
    __device__ __forceinline__ void operator()(int u, float (&f)[16], const Lane &ln, bool on) const {
        float m = largest(f);
        if (__any_sync(0xffffffffu, isinf(m))) {  // e4m3 has no infinity: it becomes a NaN
#pragma unroll
            for (int t = 0; t < 16; ++t)
                if (isinf(f[t])) f[t] = NAN;
            m = largest(f);
        }
        const uint32_t e = q8::scale_byte(m);
        const float s = q8::inverse(e);
        scale8(f, f, s);
        scale8(f + 8, f + 8, s);
        if (!on) return;
        uint8_t *row = out + u * out_h;
        *reinterpret_cast<uint2 *>(row + ln.e0) = make_uint2(q8::encode4(f[0], f[1], f[2], f[3]), q8::encode4(f[4], f[5], f[6], f[7]));
        *reinterpret_cast<uint2 *>(row + ln.e1) =
            make_uint2(q8::encode4(f[8], f[9], f[10], f[11]), q8::encode4(f[12], f[13], f[14], f[15]));
        if ((threadIdx.x & (L - 1)) == 0) scale[u * scale_h] = (uint8_t)e;
    }
};

// `count` (0 to U) consecutive heads of one tensor at one token, the group's own.  The norm's weight
// goes into the angles once for all of them: with (a, b) = r (x_a w_a, x_b w_b),
//   y_a = r (x_a (w_a cos) - x_b (w_b sin)),  y_b = r (x_a (w_a sin) + x_b (w_b cos)).
// (The shuffles need the whole warp: rows past count are zeros.)
template <typename T, int U>
__device__ __forceinline__ void load_rows(Row2<T> (&x)[U], const T *in, long long in_h, int count, const Lane &ln) {
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].load(in + u * in_h, ln.e0, ln.e1, ln.on && u < count);
}
template <typename T, int L, int U, bool kInter, class Store>
__device__ __forceinline__ void norm_rows(Row2<T> (&x)[U], const Store &store, const T *w, const float *angle_row, int count,
                                          const Lane &ln, int rot, float inv_d, float eps) {
    Row2<T> wr;
    wr.load(w, ln.e0, ln.e1, w != nullptr && ln.on);
    const Angles an = load_angles(ln, angle_row, rot, kInter);
    float ac[8], as[8], bc[8], bs[8];  // w_a cos, w_a sin, w_b cos, -w_b sin
    {
        float wf[16], y[16];
        wr.get(wf);
        apart<kInter>(wf, y);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            ac[t] = an.co[t];
            as[t] = an.si[t];
            bc[t] = an.co[t];
            bs[t] = -an.si[t];
        }
        if (w) {
            mul8(ac, ac, y);
            mul8(as, as, y);
            mul8(bc, bc, y + 8);
            mul8(bs, bs, y + 8);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[16], y[16], z[16];
        x[u].get(f);
        float r = 1.f;
        if (w) r = rsqrtf(fmaf(group_sum<L>(dot16(f, f)), inv_d, eps));
        apart<kInter>(f, y);
        if (w) {
            scale8(y, y, r);
            scale8(y + 8, y + 8, r);
        }
        // (times sine 0 an infinite element would make a NaN of the one that it is held beside)
        mul8(z, y + 8, bs);
#pragma unroll
        for (int t = 0; t < 8; ++t) z[t] = ln.turn ? z[t] : -0.f;
        fma8(z, y, ac, z);
        mul8(z + 8, y + 8, bc);
        if (ln.turn) fma8(z + 8, y, as, z + 8);
        together<kInter>(z, f);
        store(u, f, ln, ln.on && u < count);
    }
}

// Division by a number that the host knows (fast_div_params of fwd_bf16_common.cuh).
struct Div {
    uint32_t m;
    int s;
    __device__ __forceinline__ unsigned operator()(unsigned x) const { return bf16fwd::div_fast(x, m, s); }
};
Div div_by(uint32_t d) {
    Div r;
    bf16fwd::fast_div_params(d, r.m, r.s);
    return r;
}

// A position clamped into the angle table; one outside is reported.
__device__ __forceinline__ int table_row(long long pos, int P, uint32_t *flags, bool report) {
    if (pos >= 0 && pos < P) return (int)pos;
    if (report) atomicOr(flags, kFlagBadIndex);
    return pos < 0 ? 0 : P - 1;
}

// A group takes a unit: U consecutive heads of one tensor at one token.  The units of all tokens form
// one row, the groups of a warp neighbours in it (a warp that kept to one token left most of its
// lanes idle when there are few heads: 32768 tokens of one query and one key head took 37 us, so 15);
// first the warps of q, then those of k.  Measured: 24 us for 33.5 M elements in bf16 (B4 N2048 H16
// d128), 5.7 TB/s, with half of the issue slots used; 30 us before the two-element instructions and the
// folded weight.
struct RopeArgs {
    unsigned tokens, warps_q;
    int N, H[2], d, rot, P, per[2];  // units a token
    Div by_n, by_per[2];
    float inv_d, eps;
    const void *x[2], *w[2];
    void *o[2];
    long long xs[2][3], os[2][3];
    const float *cs;
    long long cs_row;
    const int *pos;
    long long pos_s[2];
    uint32_t *flags;
};

template <typename T, int L, int U, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int GW = 32 / L;
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    unsigned warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int s = warp >= a.warps_q;
    if (s) warp -= a.warps_q;
    const unsigned unit = warp * GW + (threadIdx.x & 31) / L;
    unsigned tok = a.by_per[s](unit);
    const int h0 = (int)(unit - tok * a.per[s]) * U;
    const int count = tok < a.tokens ? min(U, a.H[s] - h0) : 0;
    if (count == 0) tok = 0;  // the last warps' spare groups
    const int b = (int)a.by_n(tok), n = (int)(tok - (unsigned)b * a.N);
    const Lane ln = make_lane<L>(a.d, a.rot);
    const float *row = nullptr;
    if (a.rot) {
        long long pos = n;
        if (a.pos) pos = __ldg(a.pos + b * a.pos_s[0] + n * a.pos_s[1]);
        row = a.cs + table_row(pos, a.P, a.flags, count > 0 && h0 == 0 && (threadIdx.x & (L - 1)) == 0) * a.cs_row;
    }
    const ToRows<T> store{static_cast<T *>(a.o[s]) + b * a.os[s][0] + n * a.os[s][1] + h0 * a.os[s][2], a.os[s][2]};
    Row2<T> x[U];
    load_rows(x, static_cast<const T *>(a.x[s]) + b * a.xs[s][0] + n * a.xs[s][1] + h0 * a.xs[s][2], a.xs[s][2], count, ln);
    norm_rows<T, L, U, kInter>(x, store, static_cast<const T *>(a.w[s]), row, count, ln, a.rot, a.inv_d, a.eps);
}

// Blocks an SM, at least.  What a warp waits for (its rows, its token's place, the angles) is hidden by other warps: into
// codes eight blocks of 64 registers a thread take 46 us for the tokens below, six of 74 49; twice the heads a warp, at 111
// registers, 50 to 57, half 59.
template <typename T>
constexpr int append_blocks(bool q8) { return q8 && sizeof(T) == 2 ? 8 : 0; }  // (0: as the compiler likes)

// A warp takes one token, a tensor (q, k, v) and the part of its heads that its groups hold at once
// (the token's sequence is looked up by the whole warp).  Measured: 44 us for 10148 tokens of 32 query and
// 8 key heads of 128 in bf16, 5.8 TB/s; into codes 46 us, 5.0 TB/s.  Tasks of a token: cq parts of q, then ck of k,
// then ck of v.
struct AppendArgs {
    int B, T, Hq, Hk, d, rot, P, cq, ck;
    long long tasks;
    float inv_d, eps;
    const void *q, *k, *v, *wq, *wk;
    void *qo, *kp, *vp;
    long long qs[2], ks[2], vs[2], qos[2], kps[3], vps[3];
    const float *cs;
    long long cs_row;
    const int *pos, *bt, *lens, *cu;
    long long bt_s;
    uint8_t *scales[2];  // of a cache in 8 bits: k, v
    long long scale_s[2][2];
    unsigned cu_groups, cu_step;  // groups of 32 sequences, and the warps that look at their entries of cu
    int pages, page_size, width;
    uint32_t *flags;
};

template <typename T, int L, int U, bool kInter, bool kQ8>
__global__ void __launch_bounds__(kThreads, append_blocks<T>(kQ8)) paged_append_kernel(const AppendArgs a) {
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const unsigned task = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (task >= a.tasks) return;
    const unsigned per = a.cq + 2 * a.ck;
    const int t = (int)(task / per), part = (int)(task - (unsigned)t * per);
    const bool report = part == 0 && (threadIdx.x & 31) == 0;
    // the group's heads of the part's tensor; their rows are asked for before the token's place is looked up
    const int s = part < a.cq ? 0 : part < a.cq + a.ck ? 1 : 2, H = s == 0 ? a.Hq : a.Hk;
    const int h0 = ((part - (s == 0 ? 0 : s == 1 ? a.cq : a.cq + a.ck)) * (32 / L) + (threadIdx.x & 31) / L) * U;
    const int count = min(max(H - h0, 0), U), h = count > 0 ? h0 : 0;
    const Lane ln = make_lane<L>(a.d, a.rot);
    const long long *in_s = s == 0 ? a.qs : s == 1 ? a.ks : a.vs;
    Row2<T> x[U];
    load_rows(x, static_cast<const T *>(s == 0 ? a.q : s == 1 ? a.k : a.v) + t * in_s[0] + h * in_s[1], in_s[1], count, ln);
    int b, i, nq;
    if (a.cu) report_bad_entries(a.cu, a.B, a.T, task, a.cu_groups, a.cu_step, a.flags);
    if (!find_token(a.cu, a.B, a.T, t, b, i, nq)) return;  // left as it was
    const int room = a.width * a.page_size, raw = __ldg(a.lens + b), len = min(max(raw, 0), room);
    if (report && len != raw) atomicOr(a.flags, kFlagKvLenClamped);
    const int at = len - nq + i;  // the token's place in its sequence; < 0: it has none
    const float *row = nullptr;
    if (a.rot && part < a.cq + a.ck)
        row = a.cs + table_row(a.pos ? __ldg(a.pos + t) : max(at, 0), a.P, a.flags, report) * a.cs_row;
    if (s == 0) {
        const ToRows<T> store{static_cast<T *>(a.qo) + t * a.qos[0] + h * a.qos[1], a.qos[1]};
        norm_rows<T, L, U, kInter>(x, store, static_cast<const T *>(a.wq), row, count, ln, a.rot, a.inv_d, a.eps);
        return;
    }
    if (at < 0) return;
    const int page = __ldg(a.bt + b * a.bt_s + at / a.page_size);
    if (page < 0 || page >= a.pages) {
        if (part == a.cq && (threadIdx.x & 31) == 0) atomicOr(a.flags, kFlagBadIndex);
        return;
    }
    const long long slot = at % a.page_size;
    const long long *ps = s == 1 ? a.kps : a.vps;
    void *pages = s == 1 ? a.kp : a.vp;
    if constexpr (kQ8) {
        const ToCodes<L> store{static_cast<uint8_t *>(pages) + page * ps[0] + slot * ps[1] + h * ps[2],
                               a.scales[s - 1] + page * a.scale_s[s - 1][0] + h * a.scale_s[s - 1][1] + slot, ps[2], a.scale_s[s - 1][1]};
        if (s == 1) {
            norm_rows<T, L, U, kInter>(x, store, static_cast<const T *>(a.wk), row, count, ln, a.rot, a.inv_d, a.eps);
            return;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[16];
            x[u].get(f);
            store(u, f, ln, ln.on && u < count);
        }
    } else {
        T *to = static_cast<T *>(pages) + page * ps[0] + slot * ps[1] + h * ps[2];
        if (s == 1) {
            norm_rows<T, L, U, kInter>(x, ToRows<T>{to, ps[2]}, static_cast<const T *>(a.wk), row, count, ln, a.rot, a.inv_d, a.eps);
            return;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ln.on && u < count) x[u].store(to + u * ps[2], ln.e0, ln.e1);
    }
}

// ------------------------------------------------------------------------------- backward
//
// Blocks [0, nbq) take the queries' rows and blocks [nbq, nbq + nbk) the keys', so that a thread
// holds the weight gradient of one tensor only.  A block walks tokens; at its end its rows'
// sums go to its own partial, and bwd_weight_kernel adds the partials in a fixed order: the
// weight gradients are the same from run to run.

struct RopeBwdArgs {
    unsigned tokens, units[2];  // U heads of a token each, as in the forward
    int N, d, rot, P, nb[2], H[2], per[2];
    Div by_n, by_per[2];
    float inv_d, eps;
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

// The rows and angles of a group's next unit are on their way into shared memory while it works on one: each lane copies the chunks that it will read itself, and waits for nothing but them.
// (Angles copied once for the groups of a warp that share a token: no faster.)
// With S1 = sum x^2 and S2 = sum w dt x (one run of shuffles for both),
//   dw += (r dt) x,   dx = w (r dt) - (r^3 S2 / d) x.
// What bounds it is the issue of instructions as much as memory: with loads into registers it took
// 49 us at B4 N2048 H16 d128 in bf16, with eight elements a lane (each row's addresses and shuffles
// spread over twice the warps) 46, so 36, 34.8 with the sums below (5.8 TB/s).  Two units in shared memory and four blocks an SM:
// four units and two blocks, as many bytes on their way, took 37.5 with half as many warps to issue from,
// three and three 36.0.
constexpr int kDepth = 2, kBwdBlocks = 4;

template <int U, int C>
struct BwdStage {
    uint4 rows[U][2][2][kThreads];       // [head][x, dy][chunk][thread]: a chunk is 16 bytes, C elements
    float4 angles[2][C / 4][kThreads];   // cos, sin of the lane's C pairs
};

__device__ __forceinline__ void unpack(const uint4 &v, float *f, __nv_bfloat16) {
    Chunk<__nv_bfloat16> c;
    c.v = v;
    c.get(f);
}
__device__ __forceinline__ void unpack(const uint4 &v, float *f, float) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 repack(const float *f, __nv_bfloat16) {
    Chunk<__nv_bfloat16> c;
    c.set(f);
    return c.v;
}
__device__ __forceinline__ uint4 repack(const float *f, float) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
// Angles on their way, through L1 (the groups of a token want the same ones).
__device__ __forceinline__ void fetch_16(void *dst, const float *p) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(p) : "memory");
}
__device__ __forceinline__ void fetch_8(void *dst, const float *p) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(dst)), "l"(p) : "memory");
}
// Of a lane's 2 C elements, the pairs' first members and then the second ones, and back.
template <bool kInter, int C>
__device__ __forceinline__ void apart_c(const float (&f)[2 * C], float (&y)[2 * C]) {
#pragma unroll
    for (int t = 0; t < C; ++t) {
        y[t] = f[kInter ? 2 * t : t];
        y[C + t] = f[kInter ? 2 * t + 1 : C + t];
    }
}
template <bool kInter, int C>
__device__ __forceinline__ void together_c(const float (&y)[2 * C], float (&f)[2 * C]) {
#pragma unroll
    for (int t = 0; t < C; ++t) {
        f[kInter ? 2 * t : t] = y[t];
        f[kInter ? 2 * t + 1 : C + t] = y[C + t];
    }
}
template <int E>
__device__ __forceinline__ float dot_c(const float (&x)[E], const float (&y)[E]) {
    float s[4];
    mul2(s[0], s[1], x[0], x[1], y[0], y[1]);
    mul2(s[2], s[3], x[2], x[3], y[2], y[3]);
#pragma unroll
    for (int t = 4; t < E; t += 4) {
        ptx::fma2(s[0], s[1], x[t], x[t + 1], y[t], y[t + 1], s[0], s[1]);
        ptx::fma2(s[2], s[3], x[t + 2], x[t + 3], y[t + 2], y[t + 3], s[2], s[3]);
    }
    return (s[0] + s[2]) + (s[1] + s[3]);
}

// L lanes a row, each with two 16-byte chunks (C elements): of the rotated part chunk p and the one rot/2
// further, of the rest one of each half.
template <typename T, int L, int U, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_bwd_kernel(const RopeBwdArgs a) {
    constexpr int GW = 32 / L, C = 16 / sizeof(T), E = 2 * C;
    extern __shared__ __align__(16) uint8_t dsm[];
    BwdStage<U, C> *stage = reinterpret_cast<BwdStage<U, C> *>(dsm);
    __shared__ float red[kWarps][L * E];
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const int s = (int)blockIdx.x >= a.nb[0];
    const int blk = (int)blockIdx.x - (s ? a.nb[0] : 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane / L;
    const T *w = static_cast<const T *>(a.w[s]);
    const int p = lane & (L - 1), rp = a.rot / E;
    const bool on = p < a.d / E, turn = p < rp;
    const int e0 = turn ? C * p : C * (p + rp), e1 = turn ? C * (p + rp) : C * (p + a.d / E);
    float wf[E], dw[E];  // the pairs' first members, then the second ones
    {
        float f[E];
        unpack(w && on ? *reinterpret_cast<const uint4 *>(w + e0) : make_uint4(0u, 0u, 0u, 0u), f, T{});
        unpack(w && on ? *reinterpret_cast<const uint4 *>(w + e1) : make_uint4(0u, 0u, 0u, 0u), f + C, T{});
        apart_c<kInter, C>(f, wf);
    }
#pragma unroll
    for (int t = 0; t < E; ++t) dw[t] = 0.f;
    const unsigned step = (unsigned)a.nb[s] * kWarps * GW, units = a.units[s];
    const T *x0 = static_cast<const T *>(w ? a.x[s] : a.dy[s]), *dy0 = static_cast<const T *>(a.dy[s]);
    const int c0 = on ? e0 : 0, c1 = on ? e1 : 0;
    struct At {
        int b, n, h, count;
    };
    auto place = [&](unsigned unit) -> At {
        const unsigned tok = a.by_per[s](unit);
        At at;
        at.h = (int)(unit - tok * a.per[s]) * U;
        at.b = (int)a.by_n(tok);
        at.n = (int)(tok - (unsigned)at.b * a.N);
        at.count = min(U, a.H[s] - at.h);
        return at;
    };
    // asks for a unit; past the last one for zeros, while other groups of the warp go on
    auto fetch = [&](unsigned unit, BwdStage<U, C> &st) {
        if (unit - grp < units) {
            const At at = unit < units ? place(unit) : At{0, 0, 0, 0};
            const T *x = x0 + at.b * a.xs[s][0] + at.n * a.xs[s][1] + at.h * a.xs[s][2];
            const T *dy = dy0 + at.b * a.dys[s][0] + at.n * a.dys[s][1] + at.h * a.dys[s][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = on && u < at.count;
                if (w) {
                    wmma16::cp_async16(ptx::smem_u32(&st.rows[u][0][0][threadIdx.x]), x + c0, in ? 16u : 0u);
                    wmma16::cp_async16(ptx::smem_u32(&st.rows[u][0][1][threadIdx.x]), x + c1, in ? 16u : 0u);
                }
                wmma16::cp_async16(ptx::smem_u32(&st.rows[u][1][0][threadIdx.x]), dy + c0, in ? 16u : 0u);
                wmma16::cp_async16(ptx::smem_u32(&st.rows[u][1][1][threadIdx.x]), dy + c1, in ? 16u : 0u);
                if (u + 1 < at.count) {
                    x += a.xs[s][2];
                    dy += a.dys[s][2];
                }
            }
            if (turn && at.count > 0) {  // pairs C p .. C p + C - 1; adjacent ones C/2 from each chunk
                long long pos = at.n;
                if (a.pos) pos = __ldg(a.pos + at.b * a.pos_s[0] + at.n * a.pos_s[1]);
                const float *row = a.cs + table_row(pos, a.P, a.flags, p == 0 && at.h == 0) * a.cs_row;
#pragma unroll
                for (int i = 0; i < C / 4; ++i) {
                    float4 *c = &st.angles[0][i][threadIdx.x], *n = &st.angles[1][i][threadIdx.x];
                    if (kInter && C == 4) {
                        fetch_8(c, row + e0 / 2);
                        fetch_8(reinterpret_cast<float2 *>(c) + 1, row + e1 / 2);
                        fetch_8(n, row + a.rot / 2 + e0 / 2);
                        fetch_8(reinterpret_cast<float2 *>(n) + 1, row + a.rot / 2 + e1 / 2);
                    } else {
                        const int at4 = kInter ? (i ? e1 : e0) / 2 : e0 + 4 * i;
                        fetch_16(c, row + at4);
                        fetch_16(n, row + a.rot / 2 + at4);
                    }
                }
            }
        }
        wmma16::cp_async_commit();
    };
    unsigned unit = (unsigned)(blk * kWarps + warp) * GW + grp;
#pragma unroll 1
    for (int i = 0; i < kDepth - 1; ++i) fetch(unit + i * step, stage[i]);
    int cur = 0;
    // the groups of a warp go on together (their shuffles meet) until the first of them is past the end
#pragma unroll 1
    for (; unit - grp < units; unit += step) {
        wmma16::cp_async_wait<kDepth - 2>();
        fetch(unit + (kDepth - 1) * step, stage[cur == 0 ? kDepth - 1 : cur - 1]);
        const BwdStage<U, C> &st = stage[cur];
        if (++cur == kDepth) cur = 0;
        float co[C], si[C];
#pragma unroll
        for (int t = 0; t < C / 4; ++t) {
            float4 c = make_float4(1.f, 1.f, 1.f, 1.f), n = make_float4(0.f, 0.f, 0.f, 0.f);
            if (turn && unit < units) {
                c = st.angles[0][t][threadIdx.x];
                n = st.angles[1][t][threadIdx.x];
            }
            co[4 * t] = c.x; co[4 * t + 1] = c.y; co[4 * t + 2] = c.z; co[4 * t + 3] = c.w;
            si[4 * t] = n.x; si[4 * t + 1] = n.y; si[4 * t + 2] = n.z; si[4 * t + 3] = n.w;
        }
        const At now = unit < units ? place(unit) : At{0, 0, 0, 0};
        T *dx = static_cast<T *>(a.dx[s]) + now.b * a.dxs[s][0] + now.n * a.dxs[s][1] + now.h * a.dxs[s][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[E], y[E], g[E];
            unpack(st.rows[u][1][0][threadIdx.x], f, T{});
            unpack(st.rows[u][1][1][threadIdx.x], f + C, T{});
            apart_c<kInter, C>(f, y);
            // g = R^T dy: g_a = dy_a cos + dy_b sin, g_b = dy_b cos - dy_a sin
            if (turn) {
#pragma unroll
                for (int t = 0; t < C; t += 2) {
                    float q0, q1;
                    mul2(g[t], g[t + 1], y[C + t], y[C + 1 + t], si[t], si[t + 1]);
                    ptx::fma2(g[t], g[t + 1], y[t], y[t + 1], co[t], co[t + 1], g[t], g[t + 1]);
                    mul2(q0, q1, y[t], y[t + 1], -si[t], -si[t + 1]);
                    ptx::fma2(g[C + t], g[C + 1 + t], y[C + t], y[C + 1 + t], co[t], co[t + 1], q0, q1);
                }
            } else {  // (no products with sine 0: an infinite element would reach the one that it is held beside)
#pragma unroll
                for (int t = 0; t < E; ++t) g[t] = y[t];
            }
            if (w) {
                unpack(st.rows[u][0][0][threadIdx.x], f, T{});
                unpack(st.rows[u][0][1][threadIdx.x], f + C, T{});
                apart_c<kInter, C>(f, y);
                float wx[E];
#pragma unroll
                for (int t = 0; t < E; t += 2) mul2(wx[t], wx[t + 1], wf[t], wf[t + 1], y[t], y[t + 1]);
                float s1 = dot_c(y, y), s2 = dot_c(g, wx);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) {
                    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                    s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                }
                const float r = rsqrtf(fmaf(s1, a.inv_d, a.eps)), c = -(r * r) * (r * s2) * a.inv_d;
#pragma unroll
                for (int t = 0; t < E; t += 2) {
                    float q0, q1;
                    mul2(g[t], g[t + 1], g[t], g[t + 1], r, r);
                    ptx::fma2(dw[t], dw[t + 1], g[t], g[t + 1], y[t], y[t + 1], dw[t], dw[t + 1]);
                    mul2(q0, q1, y[t], y[t + 1], c, c);
                    ptx::fma2(g[t], g[t + 1], g[t], g[t + 1], wf[t], wf[t + 1], q0, q1);
                }
            }
            if (on && u < now.count) {
                together_c<kInter, C>(g, f);
                *reinterpret_cast<uint4 *>(dx + e0) = repack(f, T{});
                *reinterpret_cast<uint4 *>(dx + e1) = repack(f + C, T{});
            }
            if (u + 1 < now.count) dx += a.dxs[s][2];
        }
    }
    wmma16::cp_async_wait<0>();
    if (!w) return;
    // the groups of a warp, then the warps of the block
#pragma unroll
    for (int t = 0; t < E; ++t) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1) dw[t] += __shfl_xor_sync(0xffffffffu, dw[t], o);
    }
    if (grp == 0 && on) {
        float f[E];
        together_c<kInter, C>(dw, f);
#pragma unroll
        for (int t = 0; t < C; ++t) {
            red[warp][e0 + t] = f[t];
            red[warp][e1 + t] = f[C + t];
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

// dw[s][c] = the sum of the partials of tensor s: a block takes 32 columns of one tensor, its 32
// warps every 32nd partial, eight loads in flight (its time is their latency).
constexpr int kWeightWarps = 32, kWeightLoads = 8;
__global__ void __launch_bounds__(32 * kWeightWarps) bwd_weight_kernel(const float *part, int nb0, int nb1, int d, float *dwq,
                                                         float *dwk) {
    __shared__ float red[kWeightWarps][33];
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const int s = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float *dst = s ? dwk : dwq;
    if (!dst) return;
    const int lo = s ? nb0 : 0, hi = s ? nb0 + nb1 : nb0;
    float sum = 0.f;
    if (c < d) {
        for (int i = lo + w; i < hi; i += kWeightWarps * kWeightLoads) {
            float t[kWeightLoads];
#pragma unroll
            for (int k = 0; k < kWeightLoads; ++k) {
                const int at = i + kWeightWarps * k;
                t[k] = at < hi ? part[(long long)at * d + c] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kWeightLoads; ++k) sum += t[k];
        }
    }
    red[w][threadIdx.x & 31] = sum;
    __syncthreads();
    if (w == 0 && c < d) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWeightWarps; ++k) v += red[k][threadIdx.x];
        dst[c] = v;
    }
}

void copy3(long long (&d)[3], const int64_t s[3]) {
    for (int i = 0; i < 3; ++i) d[i] = s[i];
}
void copy2(long long (&d)[2], const int64_t s[2]) {
    for (int i = 0; i < 2; ++i) d[i] = s[i];
}

int lanes_of(int64_t d) { return d <= 64 ? 4 : d <= 128 ? 8 : 16; }

attn_status_t launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace

int rope_bwd_blocks() { return kBwdBlocks * (sm_count() ? sm_count() : 152); }

namespace {

// Heads a group takes at once: two (four leave more lanes idle and fewer warps: 24 and 8 heads 31 us
// for 27), or one where two would leave less than 16 warps an SM, as in a decode step.
int heads_at_once(int64_t rows, int L) { return rows * L / 64 >= 16LL * sm_count() ? 2 : 1; }

template <typename T, bool kInter>
auto rope_kernel(int L, int U) -> void (*)(const RopeArgs) {
    if (L == 4) return U == 2 ? qk_norm_rope_kernel<T, 4, 2, kInter> : qk_norm_rope_kernel<T, 4, 1, kInter>;
    if (L == 8) return U == 2 ? qk_norm_rope_kernel<T, 8, 2, kInter> : qk_norm_rope_kernel<T, 8, 1, kInter>;
    return U == 2 ? qk_norm_rope_kernel<T, 16, 2, kInter> : qk_norm_rope_kernel<T, 16, 1, kInter>;
}
template <typename T, bool kInter, bool kQ8>
auto append_kernel(int L, int U) -> void (*)(const AppendArgs) {
    if (L == 4) return U == 2 ? paged_append_kernel<T, 4, 2, kInter, kQ8> : paged_append_kernel<T, 4, 1, kInter, kQ8>;
    if (L == 8) return U == 2 ? paged_append_kernel<T, 8, 2, kInter, kQ8> : paged_append_kernel<T, 8, 1, kInter, kQ8>;
    return U == 2 ? paged_append_kernel<T, 16, 2, kInter, kQ8> : paged_append_kernel<T, 16, 1, kInter, kQ8>;
}
template <bool kQ8>
auto append_kernel(bool half, bool inter, int L, int U) -> void (*)(const AppendArgs) {
    return inter ? (half ? append_kernel<__nv_bfloat16, true, kQ8>(L, U) : append_kernel<float, true, kQ8>(L, U))
                 : (half ? append_kernel<__nv_bfloat16, false, kQ8>(L, U) : append_kernel<float, false, kQ8>(L, U));
}
// The backward's kernel, the heads a group takes at once, the groups of a warp, and its shared memory.
struct BwdPick {
    void (*kern)(const RopeBwdArgs);
    int U, groups, smem;
};
template <typename T, bool kInter>
BwdPick bwd_pick(int64_t d) {
    constexpr int U = 2, L0 = sizeof(T) == 2 ? 4 : 8;  // lanes a row of up to 64
    return {d <= 64    ? qk_norm_rope_bwd_kernel<T, L0, U, kInter>
            : d <= 128 ? qk_norm_rope_bwd_kernel<T, 2 * L0, U, kInter>
                       : qk_norm_rope_bwd_kernel<T, 4 * L0, U, kInter>,
            U, 32 / (d <= 64 ? L0 : d <= 128 ? 2 * L0 : 4 * L0), kDepth * (int)sizeof(BwdStage<U, 16 / sizeof(T)>)};
}

}  // namespace

attn_status_t launch_qk_norm_rope(const attn_qk_norm_rope_params_t &p, cudaStream_t st) {
    RopeArgs a;
    a.N = (int)p.N; a.H[0] = (int)p.Hq; a.H[1] = (int)p.Hkv; a.d = (int)p.d;
    a.rot = p.cos_sin ? (int)p.rot : 0;
    a.P = (int)p.cos_sin_rows; a.inv_d = 1.f / (float)p.d; a.eps = p.eps;
    a.x[0] = p.q; a.x[1] = p.k; a.w[0] = p.wq; a.w[1] = p.wk; a.o[0] = p.q_out; a.o[1] = p.k_out;
    copy3(a.xs[0], p.q_stride); copy3(a.xs[1], p.k_stride); copy3(a.os[0], p.q_out_stride); copy3(a.os[1], p.k_out_stride);
    a.cs = p.cos_sin; a.cs_row = p.cos_sin_stride; a.pos = p.positions; copy2(a.pos_s, p.positions_stride);
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    const int L = lanes_of(p.d), GW = 32 / L;
    const bool h = p.dtype == ATTN_DTYPE_BF16;
    a.tokens = (unsigned)(p.B * p.N);
    a.by_n = div_by((uint32_t)p.N);
    const int U = heads_at_once((long long)a.tokens * (p.Hq + p.Hkv), L);
    long long warps[2];
    for (int s = 0; s < 2; ++s) {
        a.per[s] = (a.H[s] + U - 1) / U;
        a.by_per[s] = div_by((uint32_t)a.per[s]);
        warps[s] = ((long long)a.tokens * a.per[s] + GW - 1) / GW;
        if ((warps[s] + kWarps) * GW > 0xffffffffLL) return fail(ATTN_ERR_UNSUPPORTED, "B * N * (Hq + Hkv) is too large");
    }
    a.warps_q = (unsigned)warps[0];
    const dim3 grid((unsigned)((warps[0] + warps[1] + kWarps - 1) / kWarps));
    auto kern = p.interleaved ? (h ? rope_kernel<__nv_bfloat16, true>(L, U) : rope_kernel<float, true>(L, U))
                              : (h ? rope_kernel<__nv_bfloat16, false>(L, U) : rope_kernel<float, false>(L, U));
    return launched(launch_pdl(kern, grid, dim3(kThreads), 0, st, a), "qk_norm_rope");
}

attn_status_t launch_qk_norm_rope_bwd(const attn_qk_norm_rope_bwd_params_t &bp, float *part, cudaStream_t st) {
    const attn_qk_norm_rope_params_t &p = bp.fwd;
    RopeBwdArgs a;
    a.N = (int)p.N; a.H[0] = (int)p.Hq; a.H[1] = (int)p.Hkv; a.d = (int)p.d;
    a.rot = p.cos_sin ? (int)p.rot : 0;
    a.P = (int)p.cos_sin_rows; a.inv_d = 1.f / (float)p.d; a.eps = p.eps;
    a.x[0] = p.q; a.x[1] = p.k; a.w[0] = p.wq; a.w[1] = p.wk;
    a.dy[0] = bp.dq_out; a.dy[1] = bp.dk_out; a.dx[0] = bp.dq; a.dx[1] = bp.dk;
    copy3(a.xs[0], p.q_stride); copy3(a.xs[1], p.k_stride);
    copy3(a.dys[0], bp.dq_out_stride); copy3(a.dys[1], bp.dk_out_stride);
    copy3(a.dxs[0], bp.dq_stride); copy3(a.dxs[1], bp.dk_stride);
    a.cs = p.cos_sin; a.cs_row = p.cos_sin_stride; a.pos = p.positions; copy2(a.pos_s, p.positions_stride);
    a.part = part;
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    const bool h = p.dtype == ATTN_DTYPE_BF16;
    const BwdPick pick = p.interleaved ? (h ? bwd_pick<__nv_bfloat16, true>(p.d) : bwd_pick<float, true>(p.d))
                                       : (h ? bwd_pick<__nv_bfloat16, false>(p.d) : bwd_pick<float, false>(p.d));
    a.tokens = (unsigned)(p.B * p.N);
    a.by_n = div_by((uint32_t)p.N);
    for (int s = 0; s < 2; ++s) {
        a.per[s] = (a.H[s] + pick.U - 1) / pick.U;
        a.by_per[s] = div_by((uint32_t)a.per[s]);
        const long long units = (long long)a.tokens * a.per[s];
        if (units > 0x70000000LL) return fail(ATTN_ERR_UNSUPPORTED, "B * N * (Hq + Hkv) is too large");
        a.units[s] = (unsigned)units;
    }
    // what an SM's shared memory holds of blocks, each tensor's share by its units; never more blocks
    // than warps of work
    const int most = rope_bwd_blocks();
    a.nb[0] = (int)((long long)most * a.per[0] / (a.per[0] + a.per[1]));
    a.nb[0] = a.nb[0] < 1 ? 1 : a.nb[0];
    a.nb[1] = most - a.nb[0];
    for (int s = 0; s < 2; ++s) {
        const int cap = (int)((a.units[s] + kWarps * pick.groups - 1) / (kWarps * pick.groups));
        a.nb[s] = a.nb[s] < cap ? a.nb[s] : cap;
    }
    const int blocks = a.nb[0] + a.nb[1];
    cudaError_t e = cudaFuncSetAttribute(pick.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, pick.smem);
    if (e == cudaSuccess) e = launch_pdl(pick.kern, dim3(blocks), dim3(kThreads), pick.smem, st, a);
    const attn_status_t r = launched(e, "qk_norm_rope_bwd");
    if (r || (!bp.dwq && !bp.dwk)) return r;
    return launched(launch_pdl(bwd_weight_kernel, dim3((unsigned)((p.d + 31) / 32), 2), dim3(32 * kWeightWarps), 0, st,
                               (const float *)part, a.nb[0], a.nb[1], (int)p.d, bp.dwq, bp.dwk),
                    "qk_norm_rope_bwd weights");
}

attn_status_t launch_paged_append(const attn_paged_append_params_t &p, const attn_paged_scales_t *scales, cudaStream_t st) {
    AppendArgs a{};
    const attn_paged_cache_t &c = p.cache;
    a.B = (int)c.B; a.T = (int)c.T; a.Hq = (int)p.Hq; a.Hk = (int)c.Hkv; a.d = (int)c.d;
    a.rot = p.cos_sin ? (int)p.rot : 0;
    a.P = (int)p.cos_sin_rows; a.inv_d = 1.f / (float)c.d; a.eps = p.eps;
    a.q = p.q; a.k = p.k; a.v = p.v; a.wq = p.wq; a.wk = p.wk; a.qo = p.q_out; a.kp = c.k_pages; a.vp = c.v_pages;
    copy2(a.qs, p.q_stride); copy2(a.ks, p.k_stride); copy2(a.vs, p.v_stride); copy2(a.qos, p.q_out_stride);
    copy3(a.kps, c.k_stride); copy3(a.vps, c.v_stride);
    a.cs = p.cos_sin; a.cs_row = p.cos_sin_stride; a.pos = p.positions;
    a.bt = c.block_table; a.bt_s = c.table_stride; a.lens = c.kv_lens; a.cu = c.cu_q;
    if (scales) {
        a.scales[0] = static_cast<uint8_t *>(scales->k);
        a.scales[1] = static_cast<uint8_t *>(scales->v);
        copy2(a.scale_s[0], scales->k_stride); copy2(a.scale_s[1], scales->v_stride);
    }
    a.pages = (int)c.num_pages; a.page_size = c.page_size; a.width = (int)c.table_width;
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    const int L = lanes_of(c.d);
    const bool h = c.dtype == ATTN_DTYPE_BF16;
    const int U = heads_at_once(c.T * (p.Hq + 2 * c.Hkv), L), n = 32 / L * U;
    a.cq = (int)((p.Hq + n - 1) / n);
    a.ck = (int)((c.Hkv + n - 1) / n);
    a.tasks = c.T * (a.cq + 2 * a.ck);
    if (a.tasks > 0xfffffff0LL) return fail(ATTN_ERR_UNSUPPORTED, "T * (Hq + 2 Hkv) is too large");
    a.cu_groups = (unsigned)((a.B + 31) / 32);
    a.cu_step = a.tasks < a.cu_groups ? (unsigned)a.tasks : a.cu_groups;
    const dim3 grid((unsigned)((a.tasks + kWarps - 1) / kWarps));
    auto kern = scales ? append_kernel<true>(h, p.interleaved, L, U) : append_kernel<false>(h, p.interleaved, L, U);
    return launched(launch_pdl(kern, grid, dim3(kThreads), 0, st, a), "paged_append");
}

}  // namespace attn
