// paged_read_q8.cu -- rows of a paged cache in 8 bits read back as packed bf16 or fp32.
//
// x = code * 2^(e - 127): d + 1 bytes in and 2 d or 4 d out a row, so the bound is memory.  A group of lanes takes a row of
// a head, eight codes a lane; a warp takes kRows such rows a group of keys or of values, for a run of packed rows whose
// places its lanes look up at once (sequence, length, page: three loads that wait for one another).  What it has to
// spare is instructions: with 32 chunks of any rows a warp, whose rows and addresses each lane formed for each chunk, 700 a
// packed row of 8 heads of 128, 24 ragged sequences to 8192 keys took 89 us, with or without the stores.
#include <cuda_bf16.h>

#include "paged.h"
#include "paged_tokens.cuh"
#include "q8.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kRows = 4;

struct ReadArgs {
    int B, T, H, d, width, page_size, pages;
    int run, lanes_log2;                   // packed rows a warp; lanes a row
    unsigned parts, cu_groups, cu_step;    // warps that share a packed row: K's, then V's
    long long tasks;
    const int *bt, *lens, *cu;
    long long bt_s;
    const uint8_t *pages_of[2], *scales[2];
    long long ps[2][3], ss[2][2], os[2][2];
    void *out[2];
    uint32_t *flags;
};

// A lane's rows: head h and every `step` further, of those below H.
template <typename T>
struct Rows {
    static constexpr int E = 8;               // elements a lane
    const uint8_t *codes, *scales;            // of head h at page 0, slot 0
    T *out;                                   // of head h at packed row 0
    int h, step, H;

    uint2 code[kRows];
    uint32_t scale[kRows];
    __device__ __forceinline__ void load(const ReadArgs &a, int x, int page, int slot) {
        const uint8_t *c = codes + page * a.ps[x][0] + slot * a.ps[x][1], *e = scales + page * a.ss[x][0] + slot;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (h + u * step < H) {
                code[u] = __ldg(reinterpret_cast<const uint2 *>(c + u * (step * a.ps[x][2])));
                scale[u] = __ldg(e + u * (step * a.ss[x][1]));
            }
    }
    __device__ __forceinline__ void store(const ReadArgs &a, int x, int t) const {
        T *o = out + t * a.os[x][0];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (h + u * step < H) {
                const float s = q8::pow2(scale[u]);
                float f[E];
#pragma unroll
                for (int w = 0; w < E / 4; ++w) {
                    uint32_t p[2];
                    q8::decode4(w ? code[u].y : code[u].x, p[0], p[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&p[k]));
                        f[4 * w + 2 * k] = v.x * s;
                        f[4 * w + 2 * k + 1] = v.y * s;
                    }
                }
                uint4 *to = reinterpret_cast<uint4 *>(o + u * (step * a.os[x][1]));
                if constexpr (sizeof(T) == 2) {
                    to[0] = make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                                       ptx::pack_bf16x2(f[6], f[7]));
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        to[k] = make_uint4(__float_as_uint(f[4 * k]), __float_as_uint(f[4 * k + 1]), __float_as_uint(f[4 * k + 2]),
                                           __float_as_uint(f[4 * k + 3]));
                }
            }
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) paged_read_q8_kernel(const ReadArgs a) {
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const unsigned task = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (task >= a.tasks) return;
    const int lane = threadIdx.x & 31, first = (int)(task / a.parts) * a.run, part = (int)(task % a.parts);
    if (a.cu) report_bad_entries(a.cu, a.B, a.T, task, a.cu_groups, a.cu_step, a.flags);
    // lane l: where row first + l lies (-1: nowhere)
    int page = -1, slot = 0;
    {
        int b = 0, i = 0, n = a.cu ? 0 : a.T / a.B;
        const int t = first + lane;
        bool on = lane < a.run && t < a.T;
        if (a.cu) {
            b = find_sequence(a.cu, a.B, first);
            if (on && b < a.B && __ldg(a.cu + b + 1) <= t) {  // a later sequence's, behind empty ones perhaps: find it by halves
                int end = a.B;
                for (++b; b < end;) {
                    const int mid = (b + end) / 2;
                    if (__ldg(a.cu + mid + 1) <= t) b = mid + 1;
                    else end = mid;
                }
            }
            on = on && b < a.B;
            if (on) {  // the sequence's rows as find_token takes them
                const int c0 = min(max(__ldg(a.cu + b), 0), a.T);
                n = min(max(__ldg(a.cu + b + 1), c0), a.T) - c0;
                i = t - c0;
                on = i >= 0 && i < n;
            }
        } else if (on) {
            b = t / n;
            i = t - b * n;
        }
        if (on) {
            const int room = a.width * a.page_size, raw = __ldg(a.lens + b), len = min(max(raw, 0), room), at = len - n + i;
            if (len != raw) atomicOr(a.flags, kFlagKvLenClamped);
            if (at >= 0) {
                page = __ldg(a.bt + b * a.bt_s + at / a.page_size);
                slot = at % a.page_size;
                if (page < 0 || page >= a.pages) {
                    atomicOr(a.flags, kFlagBadIndex);
                    page = -1;
                }
            }
        }
    }
    const int x = part >= (int)a.parts / 2, e0 = (lane & ((1 << a.lanes_log2) - 1)) * Rows<T>::E;
    Rows<T> r[2];
    r[0].step = 32 >> a.lanes_log2;
    r[0].H = e0 < a.d && a.out[x] ? a.H : 0;
    r[0].h = (part - x * (int)a.parts / 2) * kRows * r[0].step + (lane >> a.lanes_log2);
    r[0].codes = a.pages_of[x] + r[0].h * a.ps[x][2] + e0;
    r[0].scales = a.scales[x] + r[0].h * a.ss[x][1];
    r[0].out = static_cast<T *>(a.out[x]) + r[0].h * a.os[x][1] + e0;
    r[1] = r[0];
    // two packed rows in flight
#pragma unroll 1
    for (int j = 0; j < a.run; j += 2) {
        int p[2], s[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            p[k] = __shfl_sync(0xffffffffu, page, j + k);
            s[k] = __shfl_sync(0xffffffffu, slot, j + k);
            if (p[k] >= 0) r[k].load(a, x, p[k], s[k]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (p[k] >= 0) r[k].store(a, x, first + j + k);
    }
}

}  // namespace

attn_status_t launch_paged_read_q8(const attn_paged_read_q8_params_t &p, cudaStream_t st) {
    const attn_paged_cache_t &c = p.cache;
    const bool half = c.dtype == ATTN_DTYPE_BF16;
    ReadArgs a{};
    a.B = (int)c.B; a.T = (int)c.T; a.H = (int)c.Hkv; a.d = (int)c.d;
    a.width = (int)c.table_width; a.page_size = c.page_size; a.pages = (int)c.num_pages;
    while ((8 << a.lanes_log2) < c.d) ++a.lanes_log2;
    const int64_t group = (int64_t)kRows * (32 >> a.lanes_log2);
    a.parts = (unsigned)(2 * ((c.Hkv + group - 1) / group));
    // runs of four where that leaves 16 warps an SM or more (that case 73 us, 75 with eight, 81 with 16)
    a.run = c.T * a.parts >= (int64_t)4 * 16 * (sm_count() ? sm_count() : 152) ? 4 : 2;
    a.tasks = (c.T + a.run - 1) / a.run * a.parts;
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
