// paged_api.cu -- the C entry points of the head norms with rotation, the append to a paged cache
// and the attention over it: argument checks on the host, then the launchers.
#include <cmath>

#include "paged.h"
#include "qk_rope.h"

namespace attn {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

attn_status_t check_dtype(int32_t dtype) {
    if (dtype != ATTN_DTYPE_F32 && dtype != ATTN_DTYPE_BF16)
        return fail(ATTN_ERR_INVALID_ARG, "dtype %d is not ATTN_DTYPE_F32 or ATTN_DTYPE_BF16", dtype);
    return ATTN_OK;
}

// A tensor's base and its n strides: present, not negative, 16-byte steps.
attn_status_t check_tensor(const char *name, const void *p, const int64_t *s, int n, int32_t dtype) {
    const int64_t m = dtype == ATTN_DTYPE_BF16 ? 8 : 4;
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "%s is NULL", name);
    for (int i = 0; i < n; ++i)
        if (s[i] < 0) return fail(ATTN_ERR_INVALID_ARG, "%s_stride[%d] = %lld is negative", name, i, (long long)s[i]);
    if (!aligned16(p)) return fail(ATTN_ERR_MISALIGNED, "%s must be 16-byte aligned", name);
    for (int i = 0; i < n; ++i)
        if (s[i] % m) return fail(ATTN_ERR_MISALIGNED, "%s strides must be multiples of 16 bytes", name);
    return ATTN_OK;
}

// Every element of a tensor that is written has a place of its own: a stride of zero along a
// dimension longer than one would make rows write over one another.
attn_status_t check_written(const char *name, const int64_t *s, const int64_t *sizes, int n) {
    for (int i = 0; i < n; ++i)
        if (sizes[i] > 1 && s[i] == 0)
            return fail(ATTN_ERR_INVALID_ARG, "%s_stride[%d] is 0: an output cannot be broadcast", name, i);
    return ATTN_OK;
}

attn_status_t check_rope(int64_t d, int64_t rot, int32_t interleaved, float eps, const void *wq, const void *wk,
                         const float *cs, int64_t rows, int64_t stride) {
    if (d < 1) return fail(ATTN_ERR_INVALID_ARG, "d must be >= 1 (got %lld)", (long long)d);
    if (d > 256 || d % 16) return fail(ATTN_ERR_UNSUPPORTED, "d must be a multiple of 16 up to 256 (got %lld)", (long long)d);
    if (interleaved != 0 && interleaved != 1)
        return fail(ATTN_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %d)", interleaved);
    if ((wq || wk) && !(eps > 0.f && std::isfinite(eps)))
        return fail(ATTN_ERR_INVALID_ARG, "eps must be positive and finite (got %g)", eps);
    if (!aligned16(wq) || !aligned16(wk)) return fail(ATTN_ERR_MISALIGNED, "wq and wk must be 16-byte aligned");
    if (cs) {
        if (rot < 0 || rot > d) return fail(ATTN_ERR_INVALID_ARG, "rot = %lld is not in [0, d = %lld]", (long long)rot, (long long)d);
        if (rot % 16) return fail(ATTN_ERR_UNSUPPORTED, "rot must be a multiple of 16 (got %lld)", (long long)rot);
        if (rows < 1 || rows > INT32_MAX) return fail(ATTN_ERR_INVALID_ARG, "cos_sin_rows = %lld", (long long)rows);
        if (stride < rot && rows > 1) return fail(ATTN_ERR_INVALID_ARG, "cos_sin_stride = %lld < rot", (long long)stride);
        if (!aligned16(cs) || (rows > 1 && stride % 4))
            return fail(ATTN_ERR_MISALIGNED, "cos_sin rows must be 16-byte aligned");
    }
    return ATTN_OK;
}

// The checks shared by the forward and the backward, up to the tensors themselves.
attn_status_t check_norm_rope_sizes(const attn_qk_norm_rope_params_t *p) {
    attn_status_t st = check_dtype(p->dtype);
    if (st) return st;
    if (p->B < 0 || p->N < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%lld N=%lld)", (long long)p->B, (long long)p->N);
    if (p->Hq < 1 || p->Hkv < 1)
        return fail(ATTN_ERR_INVALID_ARG, "Hq and Hkv must be >= 1 (got %lld, %lld)", (long long)p->Hq, (long long)p->Hkv);
    if (p->Hq > 65535 || p->Hkv > 65535) return fail(ATTN_ERR_UNSUPPORTED, "Hq and Hkv must be <= 65535");
    if (p->B > INT32_MAX || p->N > INT32_MAX || (p->N && p->B > INT32_MAX / p->N))
        return fail(ATTN_ERR_UNSUPPORTED, "B * N must be below 2^31");
    if ((st = check_rope(p->d, p->rot, p->interleaved, p->eps, p->wq, p->wk, p->cos_sin, p->cos_sin_rows, p->cos_sin_stride)))
        return st;
    if (p->positions && (p->positions_stride[0] < 0 || p->positions_stride[1] < 0))
        return fail(ATTN_ERR_INVALID_ARG, "positions_stride is negative");
    return ATTN_OK;
}

// The sizes of a cache and its batch.
attn_status_t check_cache_sizes(const attn_paged_cache_t &c) {
    attn_status_t st = check_dtype(c.dtype);
    if (st) return st;
    if (c.B < 0 || c.T < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%lld T=%lld)", (long long)c.B, (long long)c.T);
    if (c.B > 65535 || c.T > INT32_MAX) return fail(ATTN_ERR_UNSUPPORTED, "B must be <= 65535 and T below 2^31");
    if (c.Hkv < 1 || c.Hkv > 65535) return fail(ATTN_ERR_INVALID_ARG, "Hkv = %lld", (long long)c.Hkv);
    if (c.page_size < 1) return fail(ATTN_ERR_INVALID_ARG, "page_size must be >= 1 (got %d)", c.page_size);
    if (c.num_pages < 0 || c.num_pages > INT32_MAX || c.table_width < 0 || c.table_width > INT32_MAX ||
        c.table_stride < 0)
        return fail(ATTN_ERR_INVALID_ARG, "num_pages, table_width or table_stride is out of range");
    if (c.T == 0) return ATTN_OK;
    if (c.B < 1) return fail(ATTN_ERR_INVALID_ARG, "B must be >= 1 when there are tokens");
    if (c.table_width * c.page_size > INT32_MAX)
        return fail(ATTN_ERR_UNSUPPORTED, "table_width * page_size must be below 2^31");
    if (!c.cu_q && c.T % c.B)
        return fail(ATTN_ERR_INVALID_ARG, "without cu_q, T = %lld must be a multiple of B = %lld", (long long)c.T, (long long)c.B);
    return ATTN_OK;
}

// Pages of codes or scale bytes: the base, and the n strides of dimensions longer than one, are present, positive, and
// multiples of `step` bytes.
attn_status_t check_bytes(const char *name, const void *p, const int64_t *s, const int64_t *sizes, int n, int64_t step) {
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "%s is NULL", name);
    for (int i = 0; i < n; ++i) {
        if (sizes[i] <= 1) continue;
        if (s[i] < 1) return fail(ATTN_ERR_INVALID_ARG, "%s_stride[%d] = %lld is not positive", name, i, (long long)s[i]);
        if (s[i] % step) return fail(ATTN_ERR_MISALIGNED, "%s strides must be multiples of %lld bytes", name, (long long)step);
    }
    if (reinterpret_cast<uintptr_t>(p) % (uintptr_t)step) return fail(ATTN_ERR_MISALIGNED, "%s must be %lld-byte aligned", name, (long long)step);
    return ATTN_OK;
}

// A cache in 8 bits: codes in steps of 16 bytes, scale bytes in steps of `step`.
attn_status_t check_q8(const attn_paged_cache_t &c, const attn_paged_scales_t &sc, int64_t step) {
    const int64_t sizes[3] = {c.num_pages, c.page_size, c.Hkv}, rows[2] = {c.num_pages, c.Hkv};
    attn_status_t st = ATTN_OK;
    if (c.num_pages > 0 &&
        ((st = check_bytes("k_pages", c.k_pages, c.k_stride, sizes, 3, 16)) || (st = check_bytes("v_pages", c.v_pages, c.v_stride, sizes, 3, 16)) ||
         (st = check_bytes("k_scales", sc.k, sc.k_stride, rows, 2, step)) || (st = check_bytes("v_scales", sc.v, sc.v_stride, rows, 2, step))))
        return st;
    return ATTN_OK;
}

// scales: of a cache in 8 bits (of any alignment), or null.
attn_status_t check_cache(const attn_paged_cache_t &c, const attn_paged_scales_t *scales) {
    attn_status_t st = check_cache_sizes(c);
    if (st || c.T == 0) return st;
    if (!c.kv_lens || (!c.block_table && c.table_width > 0))
        return fail(ATTN_ERR_INVALID_ARG, "kv_lens or block_table is NULL");
    if (scales) return check_q8(c, *scales, 1);
    const int64_t sizes[3] = {c.num_pages, c.page_size, c.Hkv};
    if (c.num_pages > 0) {
        if ((st = check_tensor("k", c.k_pages, c.k_stride, 3, c.dtype))) return st;
        if ((st = check_tensor("v", c.v_pages, c.v_stride, 3, c.dtype))) return st;
        if ((st = check_written("k", c.k_stride, sizes, 3)) || (st = check_written("v", c.v_stride, sizes, 3))) return st;
    }
    return ATTN_OK;
}

attn_status_t check_paged_fwd(const attn_paged_fwd_params_t *p) {
    const attn_paged_cache_t &c = p->cache;
    attn_status_t st = check_dtype(c.dtype);
    if (st) return st;
    if (p->causal != 0 && p->causal != 1) return fail(ATTN_ERR_INVALID_ARG, "causal must be 0 or 1 (got %d)", p->causal);
    if (!std::isfinite(p->scale)) return fail(ATTN_ERR_INVALID_ARG, "scale is not finite");
    if (c.dtype != ATTN_DTYPE_BF16) return fail(ATTN_ERR_UNSUPPORTED, "paged attention supports bfloat16 only");
    if (c.d != 64 && c.d != 128) return fail(ATTN_ERR_UNSUPPORTED, "paged attention supports d in {64, 128} (got %lld)", (long long)c.d);
    if (!(p->scale > 0.f)) return fail(ATTN_ERR_UNSUPPORTED, "paged attention needs scale > 0 (got %g)", p->scale);
    if (c.page_size < 16 || (c.page_size & (c.page_size - 1)))
        return fail(ATTN_ERR_UNSUPPORTED, "page_size must be a power of two >= 16 (got %d)", c.page_size);
    if (c.Hkv < 1 || p->Hq < 1 || p->Hq % c.Hkv)
        return fail(ATTN_ERR_INVALID_ARG, "Hq = %lld must be a multiple of Hkv = %lld", (long long)p->Hq, (long long)c.Hkv);
    if (p->Hq / c.Hkv > 64) return fail(ATTN_ERR_UNSUPPORTED, "Hq / Hkv must be <= 64 (got %lld)", (long long)(p->Hq / c.Hkv));
    if (c.T > (1 << 30) / (p->Hq / c.Hkv)) return fail(ATTN_ERR_UNSUPPORTED, "T * Hq / Hkv must be at most 2^30");
    if (p->max_q < 0) return fail(ATTN_ERR_INVALID_ARG, "max_q is negative");
    // the last tile's end, past the keys by up to 127, stays an int
    if (c.table_width > 0 && c.table_width > (INT32_MAX - 255) / c.page_size)
        return fail(ATTN_ERR_UNSUPPORTED, "table_width * page_size must be at most 2^31 - 256");
    return ATTN_OK;
}

// The pointers of an attention that has tokens.
attn_status_t check_paged_tensors(const attn_paged_fwd_params_t *p, const attn_paged_scales_t *scales) {
    const attn_paged_cache_t &c = p->cache;
    const int64_t nq[2] = {c.T, p->Hq};
    attn_status_t st;
    if ((st = check_tensor("q", p->q, p->q_stride, 2, c.dtype)) || (st = check_tensor("o", p->o, p->o_stride, 2, c.dtype)) ||
        (st = check_written("q", p->q_stride, nq, 2)) || (st = check_written("o", p->o_stride, nq, 2)))
        return st;
    return scales ? check_q8(c, *scales, 16) : ATTN_OK;
}

attn_status_t check_workspace(const void *workspace, size_t bytes, size_t need) {
    if (need && (!workspace || !aligned16(workspace) || bytes < need))
        return fail(ATTN_ERR_WORKSPACE, "workspace must be 16-byte aligned and hold %zu bytes (got %zu)", need, bytes);
    return ATTN_OK;
}

const attn_paged_scales_t *scales_of(const attn_paged_prefix_params_t &p) { return p.scales.k || p.scales.v ? &p.scales : nullptr; }

// The sizes of both attentions of a call.
attn_status_t check_prefix_sizes(const attn_paged_prefix_params_t *p) {
    attn_status_t st;
    if ((st = check_paged_fwd(&p->fwd)) || (st = check_cache_sizes(p->fwd.cache))) return st;
    if (p->fwd.cache.T == 0) return ATTN_OK;
    if (p->P < 1 || p->P > 65535) return fail(ATTN_ERR_INVALID_ARG, "P must be in [1, 65535] (got %lld)", (long long)p->P);
    if (p->prefix_width < 0 || p->prefix_width > INT32_MAX || p->prefix_stride < 0)
        return fail(ATTN_ERR_INVALID_ARG, "prefix_width or prefix_stride is out of range");
    if (p->prefix_width > 0 && p->prefix_width > (INT32_MAX - 255) / p->fwd.cache.page_size)
        return fail(ATTN_ERR_UNSUPPORTED, "prefix_width * page_size must be at most 2^31 - 256");
    if (!p->cu_prefix && p->fwd.cache.T % p->P)
        return fail(ATTN_ERR_INVALID_ARG, "without cu_prefix, T = %lld must be a multiple of P = %lld", (long long)p->fwd.cache.T, (long long)p->P);
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" attn_status_t attn_qk_norm_rope(const attn_qk_norm_rope_params_t *p, attn_stream_t stream) {
    clear_error();
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "params is NULL");
    attn_status_t st = check_norm_rope_sizes(p);
    if (st) return st;
    if (p->B * p->N == 0) return ATTN_OK;
    const int64_t nq[3] = {p->B, p->N, p->Hq}, nk[3] = {p->B, p->N, p->Hkv};
    if ((st = check_tensor("q", p->q, p->q_stride, 3, p->dtype)) || (st = check_tensor("k", p->k, p->k_stride, 3, p->dtype)) ||
        (st = check_tensor("q_out", p->q_out, p->q_out_stride, 3, p->dtype)) ||
        (st = check_tensor("k_out", p->k_out, p->k_out_stride, 3, p->dtype)) ||
        (st = check_written("q_out", p->q_out_stride, nq, 3)) || (st = check_written("k_out", p->k_out_stride, nk, 3)))
        return st;
    return launch_qk_norm_rope(*p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t attn_qk_norm_rope_bwd_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t Hkv, int64_t d) {
    if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || d < 1 || Hq > 65535 || Hkv > 65535 || B > INT32_MAX / N) return 0;
    return (size_t)rope_bwd_blocks() * (size_t)d * sizeof(float);
}

extern "C" attn_status_t attn_qk_norm_rope_bwd(const attn_qk_norm_rope_bwd_params_t *bp, void *workspace,
                                               size_t workspace_bytes, attn_stream_t stream) {
    clear_error();
    if (!bp) return fail(ATTN_ERR_INVALID_ARG, "params is NULL");
    const attn_qk_norm_rope_params_t *p = &bp->fwd;
    attn_status_t st = check_norm_rope_sizes(p);
    if (st) return st;
    if ((!bp->dwq) != (!p->wq) || (!bp->dwk) != (!p->wk))
        return fail(ATTN_ERR_INVALID_ARG, "dwq and dwk are given exactly where wq and wk are");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (p->B * p->N == 0) {  // no rows: the weight gradients are sums of nothing
        for (float *dw : {bp->dwq, bp->dwk})
            if (dw) {
                const cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)p->d * sizeof(float), s);
                if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
            }
        return ATTN_OK;
    }
    const int64_t nq[3] = {p->B, p->N, p->Hq}, nk[3] = {p->B, p->N, p->Hkv};
    if ((st = check_tensor("q", p->q, p->q_stride, 3, p->dtype)) || (st = check_tensor("k", p->k, p->k_stride, 3, p->dtype)) ||
        (st = check_tensor("dq_out", bp->dq_out, bp->dq_out_stride, 3, p->dtype)) ||
        (st = check_tensor("dk_out", bp->dk_out, bp->dk_out_stride, 3, p->dtype)) ||
        (st = check_tensor("dq", bp->dq, bp->dq_stride, 3, p->dtype)) ||
        (st = check_tensor("dk", bp->dk, bp->dk_stride, 3, p->dtype)) ||
        (st = check_written("dq", bp->dq_stride, nq, 3)) || (st = check_written("dk", bp->dk_stride, nk, 3)))
        return st;
    if (p->wq || p->wk) {
        const size_t need = attn_qk_norm_rope_bwd_workspace_bytes(p->B, p->N, p->Hq, p->Hkv, p->d);
        if (!workspace || !aligned16(workspace) || workspace_bytes < need)
            return fail(ATTN_ERR_WORKSPACE, "workspace must be 16-byte aligned and hold %zu bytes (got %zu)", need,
                        workspace_bytes);
    }
    return launch_qk_norm_rope_bwd(*bp, static_cast<float *>(workspace), s);
}

namespace {

attn_status_t append(const attn_paged_append_params_t *p, const attn_paged_scales_t *scales, attn_stream_t stream) {
    const attn_paged_cache_t &c = p->cache;
    attn_status_t st = check_cache(c, scales);
    if (st) return st;
    if (p->Hq < 1 || p->Hq > 65535) return fail(ATTN_ERR_INVALID_ARG, "Hq = %lld", (long long)p->Hq);
    if ((st = check_rope(c.d, p->rot, p->interleaved, p->eps, p->wq, p->wk, p->cos_sin, p->cos_sin_rows, p->cos_sin_stride)))
        return st;
    if (c.T == 0) return ATTN_OK;
    const int64_t nq[2] = {c.T, p->Hq};
    if ((st = check_tensor("q", p->q, p->q_stride, 2, c.dtype)) || (st = check_tensor("k", p->k, p->k_stride, 2, c.dtype)) ||
        (st = check_tensor("v", p->v, p->v_stride, 2, c.dtype)) ||
        (st = check_tensor("q_out", p->q_out, p->q_out_stride, 2, c.dtype)) ||
        (st = check_written("q_out", p->q_out_stride, nq, 2)))
        return st;
    return launch_paged_append(*p, scales, reinterpret_cast<cudaStream_t>(stream));
}

size_t fwd_workspace(const attn_paged_fwd_params_t *p, const attn_paged_scales_t *scales) {
    if (!p || check_paged_fwd(p) || check_cache_sizes(p->cache) || p->cache.T < 1) {
        clear_error();
        return 0;
    }
    return paged_fwd_workspace(*p, scales);
}

attn_status_t fwd(const attn_paged_fwd_params_t *p, const attn_paged_scales_t *scales, void *workspace, size_t workspace_bytes,
                  attn_stream_t stream) {
    attn_status_t st = check_paged_fwd(p);
    if (st || (st = check_cache(p->cache, scales))) return st;
    if (p->cache.T == 0) return ATTN_OK;
    if ((st = check_paged_tensors(p, scales)) || (st = check_workspace(workspace, workspace_bytes, paged_fwd_workspace(*p, scales))))
        return st;
    return launch_paged_fwd(*p, scales, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" attn_status_t attn_paged_append(const attn_paged_append_params_t *p, attn_stream_t stream) {
    clear_error();
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "params is NULL");
    return append(p, nullptr, stream);
}

extern "C" attn_status_t attn_paged_append_q8(const attn_paged_append_q8_params_t *p, attn_stream_t stream) {
    clear_error();
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "params is NULL");
    return append(&p->append, &p->scales, stream);
}

extern "C" attn_status_t attn_paged_read_q8(const attn_paged_read_q8_params_t *p, attn_stream_t stream) {
    clear_error();
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "params is NULL");
    const attn_paged_cache_t &c = p->cache;
    attn_status_t st = check_cache(c, &p->scales);
    if (st) return st;
    if (c.d < 1) return fail(ATTN_ERR_INVALID_ARG, "d must be >= 1 (got %lld)", (long long)c.d);
    if (c.d > 256 || c.d % 16) return fail(ATTN_ERR_UNSUPPORTED, "d must be a multiple of 16 up to 256 (got %lld)", (long long)c.d);
    if (c.T == 0 || (!p->k && !p->v)) return ATTN_OK;
    const int64_t n[2] = {c.T, c.Hkv};
    if (p->k && ((st = check_tensor("k", p->k, p->k_stride, 2, c.dtype)) || (st = check_written("k", p->k_stride, n, 2)))) return st;
    if (p->v && ((st = check_tensor("v", p->v, p->v_stride, 2, c.dtype)) || (st = check_written("v", p->v_stride, n, 2)))) return st;
    return launch_paged_read_q8(*p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t attn_paged_fwd_workspace_bytes(const attn_paged_fwd_params_t *p) {
    clear_error();
    return fwd_workspace(p, nullptr);
}

extern "C" attn_status_t attn_paged_fwd(const attn_paged_fwd_params_t *p, void *workspace, size_t workspace_bytes,
                                        attn_stream_t stream) {
    clear_error();
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "params is NULL");
    return fwd(p, nullptr, workspace, workspace_bytes, stream);
}

extern "C" size_t attn_paged_fwd_q8_workspace_bytes(const attn_paged_fwd_q8_params_t *p) {
    clear_error();
    return p ? fwd_workspace(&p->fwd, &p->scales) : 0;
}

extern "C" attn_status_t attn_paged_fwd_q8(const attn_paged_fwd_q8_params_t *p, void *workspace, size_t workspace_bytes,
                                           attn_stream_t stream) {
    clear_error();
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "params is NULL");
    return fwd(&p->fwd, &p->scales, workspace, workspace_bytes, stream);
}

extern "C" size_t attn_paged_prefix_fwd_workspace_bytes(const attn_paged_prefix_params_t *p) {
    clear_error();
    if (!p || check_prefix_sizes(p) || p->fwd.cache.T < 1) {
        clear_error();
        return 0;
    }
    return paged_prefix_workspace(*p);
}

extern "C" attn_status_t attn_paged_prefix_fwd(const attn_paged_prefix_params_t *p, void *workspace, size_t workspace_bytes,
                                               attn_stream_t stream) {
    clear_error();
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "params is NULL");
    const attn_paged_scales_t *scales = scales_of(*p);
    attn_status_t st = check_prefix_sizes(p);
    if (st || (st = check_cache(p->fwd.cache, scales))) return st;
    if (p->fwd.cache.T == 0) return ATTN_OK;
    if (!p->prefix_lens || (!p->prefix_table && p->prefix_width > 0))
        return fail(ATTN_ERR_INVALID_ARG, "prefix_lens or prefix_table is NULL");
    if ((st = check_paged_tensors(&p->fwd, scales))) return st;
    const size_t need = paged_prefix_workspace(*p);
    if (!need) return fail(ATTN_ERR_UNSUPPORTED, "Hkv (T Hq / Hkv + B) table_width page_size is too large");
    if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
    return launch_paged_prefix(*p, workspace, reinterpret_cast<cudaStream_t>(stream));
}
