// paged_read_q8.cu -- rows of a paged cache in 8 bits read back as packed bf16 or fp32.
//
// x = code * 2^(e - 127): d + 1 bytes in and 2 d or 4 d out a row, so the bound is memory.  A warp takes one
// packed row (its sequence is looked up by the whole warp) and 32 kParts chunks of 16 bytes of output
// of its heads' keys and values, all loads before the first store.
#include <cuda_bf16.h>

#include "fwd_bf16_common.cuh"
#include "paged.h"
#include "paged_tokens.cuh"
#include "q8.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kParts = 8;

struct ReadArgs {
    int B, T, H, d, width, page_size, pages;
    unsigned chunks, parts, cu_groups, cu_step;  // chunks of one packed row, and the warps that share them
    uint32_t row_m;  // division by the chunks of a head
    int row_s;
    long long tasks;
    const int *bt, *lens, *cu;
    long long bt_s;
    const uint8_t *pages_of[2], *scales[2];
    long long ps[2][3], ss[2][2], os[2][2];
    void *out[2];
    uint32_t *flags;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) paged_read_q8_kernel(const ReadArgs a) {
    constexpr int E = 16 / sizeof(T);  // elements of a chunk
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const unsigned task = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (task >= a.tasks) return;
    const int t = (int)(task / a.parts), part = (int)(task - (unsigned)t * a.parts), lane = threadIdx.x & 31;
    if (a.cu) report_bad_entries(a.cu, a.B, a.T, task, a.cu_groups, a.cu_step, a.flags);
    int b, i, n;
    if (!find_token(a.cu, a.B, a.T, t, b, i, n)) return;
    const int room = a.width * a.page_size, raw = __ldg(a.lens + b), len = min(max(raw, 0), room);
    if (lane == 0 && len != raw) atomicOr(a.flags, kFlagKvLenClamped);
    const int at = len - n + i;
    if (at < 0) return;
    const int page = __ldg(a.bt + b * a.bt_s + at / a.page_size);
    if (page < 0 || page >= a.pages) {
        if (lane == 0) atomicOr(a.flags, kFlagBadIndex);
        return;
    }
    const int slot = at % a.page_size;
    uint2 code[kParts];
    uint32_t scale[kParts];
    T *to[kParts];
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
        const unsigned c = (unsigned)(part * kParts + u) * 32 + lane;
        unsigned row = bf16fwd::div_fast(c, a.row_m, a.row_s);
        const int e0 = (int)(c - row * (unsigned)(a.d / E)) * E, x = row >= (unsigned)a.H;
        if (x) row -= a.H;
        to[u] = nullptr;
        if (c < a.chunks && a.out[x]) {
            const uint8_t *p = a.pages_of[x] + page * a.ps[x][0] + slot * a.ps[x][1] + row * a.ps[x][2] + e0;
            if (E == 8) code[u] = __ldg(reinterpret_cast<const uint2 *>(p));
            else code[u].x = __ldg(reinterpret_cast<const uint32_t *>(p));
            scale[u] = __ldg(a.scales[x] + page * a.ss[x][0] + row * a.ss[x][1] + slot);
            to[u] = static_cast<T *>(a.out[x]) + t * a.os[x][0] + row * a.os[x][1] + e0;
        }
    }
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
        if (!to[u]) continue;
        const float s = q8::pow2(scale[u]);
        float f[E];
#pragma unroll
        for (int w = 0; w < E / 4; ++w) {
            uint32_t h[2];
            q8::decode4(w ? code[u].y : code[u].x, h[0], h[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
                f[4 * w + 2 * k] = v.x * s;
                f[4 * w + 2 * k + 1] = v.y * s;
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = E == 8 ? ptx::pack_bf16x2(f[(2 * k) % E], f[(2 * k + 1) % E]) : __float_as_uint(f[k]);
        *reinterpret_cast<uint4 *>(to[u]) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

attn_status_t launch_paged_read_q8(const attn_paged_read_q8_params_t &p, cudaStream_t st) {
    const attn_paged_cache_t &c = p.cache;
    const bool half = c.dtype == ATTN_DTYPE_BF16;
    const int E = half ? 8 : 4;
    ReadArgs a{};
    a.B = (int)c.B; a.T = (int)c.T; a.H = (int)c.Hkv; a.d = (int)c.d;
    a.width = (int)c.table_width; a.page_size = c.page_size; a.pages = (int)c.num_pages;
    bf16fwd::fast_div_params((uint32_t)(c.d / E), a.row_m, a.row_s);
    const int64_t chunks = 2 * c.Hkv * (c.d / E);
    a.chunks = (unsigned)chunks;
    a.parts = (unsigned)((chunks + 32 * kParts - 1) / (32 * kParts));
    a.tasks = c.T * a.parts;
    if (a.tasks > 0xfffffff0LL) return fail(ATTN_ERR_UNSUPPORTED, "T * Hkv is too large");
    a.cu_groups = (unsigned)((a.B + 31) / 32);
    a.cu_step = a.tasks < a.cu_groups ? (unsigned)a.tasks : a.cu_groups;
    a.bt = c.block_table; a.bt_s = c.table_stride; a.lens = c.kv_lens; a.cu = c.cu_q;
    for (int x = 0; x < 2; ++x) {
        a.pages_of[x] = static_cast<const uint8_t *>(x ? c.v_pages : c.k_pages);
        a.scales[x] = static_cast<const uint8_t *>(x ? p.scales.v : p.scales.k);
        a.out[x] = x ? p.v : p.k;
        for (int i = 0; i < 3; ++i) a.ps[x][i] = x ? c.v_stride[i] : c.k_stride[i];
        for (int i = 0; i < 2; ++i) {
            a.ss[x][i] = x ? p.scales.v_stride[i] : p.scales.k_stride[i];
            a.os[x][i] = x ? p.v_stride[i] : p.k_stride[i];
        }
    }
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    const dim3 grid((unsigned)((a.tasks + kWarps - 1) / kWarps));
    const cudaError_t e = half ? launch_pdl(paged_read_q8_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a)
                               : launch_pdl(paged_read_q8_kernel<float>, grid, dim3(kThreads), 0, st, a);
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "paged_read_q8 launch: %s", cudaGetErrorString(e));
}

}  // namespace attn
