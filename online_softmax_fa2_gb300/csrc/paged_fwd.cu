// paged_fwd.cu -- attention of the new tokens of a ragged batch over a paged key/value cache.
//
// One warp per (token, query head): the warp walks the visible keys, D / 32 dimensions a lane,
// with the online update of (m, l, u) ("How Does FlashAttention Preserve Global Softmax Across
// Tiles?", sections 3 and 5).
#include <cuda_bf16.h>

#include "paged.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct PagedArgs {
    int B, T, Hq, G, causal, page_size, table_width, num_pages;
    float scale_log2;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *o;
    float *lse;
    long long qs[2], os[2], ks[3], vs[3], bt_s;
    const int *bt, *lens, *cu;
    uint32_t *flags;
};

template <int D>
__global__ void __launch_bounds__(kThreads) paged_simple_kernel(const PagedArgs a) {
    constexpr int E = D / 32;
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= (long long)a.T * a.Hq) return;
    const int t = (int)(row / a.Hq), h = (int)(row % a.Hq), hk = h / a.G;
    int b, i, nq;
    if (a.cu) {
        b = 0;
        while (b < a.B && __ldg(a.cu + b + 1) <= t) ++b;
        if (b >= a.B) return;
        nq = __ldg(a.cu + b + 1) - __ldg(a.cu + b);
        i = t - __ldg(a.cu + b);
        if (i < 0 || i >= nq) return;
    } else {
        nq = a.T / a.B;
        b = t / nq;
        i = t - b * nq;
    }
    const long long room = (long long)a.table_width * a.page_size;
    const int raw = __ldg(a.lens + b);
    const int n = (int)(raw < 0 ? 0 : raw > room ? room : raw);
    if (n != raw && lane == 0) atomicOr(a.flags, kFlagKvLenClamped);
    const int end = a.causal ? max(0, min(n, i + n - nq + 1)) : n;
    float q[E], u[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(a.q[t * a.qs[0] + h * a.qs[1] + lane * E + e]) * a.scale_log2;
        u[e] = 0.f;
    }
    for (int j = 0; j < end; ++j) {
        const int page = __ldg(a.bt + b * a.bt_s + j / a.page_size), slot = j % a.page_size;
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(a.flags, kFlagBadIndex);
            continue;
        }
        const __nv_bfloat16 *kr = a.k + page * a.ks[0] + slot * a.ks[1] + hk * a.ks[2] + lane * E;
        const __nv_bfloat16 *vr = a.v + page * a.vs[0] + slot * a.vs[1] + hk * a.vs[2] + lane * E;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(q[e], __bfloat162float(kr[e]), x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        const float mn = fmaxf(m, x), al = m == -INFINITY ? 0.f : ptx::ex2(m - mn), p = ptx::ex2(x - mn);
        l = fmaf(al, l, p);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] = fmaf(al, u[e], p * __bfloat162float(vr[e]));
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        a.o[t * a.os[0] + h * a.os[1] + lane * E + e] = __float2bfloat16(l > 0.f ? u[e] / l : 0.f);
    if (a.lse && lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t paged_fwd_workspace(const attn_paged_fwd_params_t &) { return 0; }

attn_status_t launch_paged_fwd(const attn_paged_fwd_params_t &p, void *, cudaStream_t st) {
    const attn_paged_cache_t &c = p.cache;
    PagedArgs a;
    a.B = (int)c.B; a.T = (int)c.T; a.Hq = (int)p.Hq; a.G = (int)(p.Hq / c.Hkv); a.causal = p.causal;
    a.page_size = c.page_size; a.table_width = (int)c.table_width; a.num_pages = (int)c.num_pages;
    a.scale_log2 = p.scale * kLog2e;
    a.q = static_cast<const __nv_bfloat16 *>(p.q);
    a.k = static_cast<const __nv_bfloat16 *>(c.k_pages);
    a.v = static_cast<const __nv_bfloat16 *>(c.v_pages);
    a.o = static_cast<__nv_bfloat16 *>(p.o);
    a.lse = p.lse;
    for (int i = 0; i < 2; ++i) { a.qs[i] = p.q_stride[i]; a.os[i] = p.o_stride[i]; }
    for (int i = 0; i < 3; ++i) { a.ks[i] = c.k_stride[i]; a.vs[i] = c.v_stride[i]; }
    a.bt = c.block_table; a.bt_s = c.table_stride; a.lens = c.kv_lens; a.cu = c.cu_q;
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    const long long rows = (long long)c.T * p.Hq;
    const cudaError_t e = launch_pdl(c.d == 64 ? paged_simple_kernel<64> : paged_simple_kernel<128>,
                                     dim3((unsigned)((rows + 3) / 4)), dim3(kThreads), 0, st, a);
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "paged_fwd launch: %s", cudaGetErrorString(e));
}

}  // namespace attn
