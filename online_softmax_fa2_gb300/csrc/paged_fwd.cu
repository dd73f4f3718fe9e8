// paged_fwd.cu -- attention of the new tokens of a ragged batch over a paged key/value cache: the
// choice of a kernel, the cut of its workspace, the tensor maps.
#include <cudaTypedefs.h>

#include <atomic>
#include <chrono>

#include "paged.h"
#include "paged_merge.cuh"

namespace attn {

PFN_cuTensorMapEncodeTiled_v12000 get_encoder();  // fwd_bf16_sm103.cu

namespace {

using namespace paged;

struct Plan {
    int tc, tile_rows;  // row tiles a block (0: the kernel for few rows), rows of one at most
    int R, kt, grid, box;
    int min_cut;
    bool cuts;  // a block may be cut
    bool fits;  // the line of tiles is shorter than kLongestLine
    size_t off_ml, off_u, bytes;
};

Plan make_plan(const attn_paged_fwd_params_t &p) {
    const attn_paged_cache_t &c = p.cache;
    const int64_t G = p.Hq / c.Hkv;
    // tokens a sequence, or their mean
    const int64_t most = p.max_q > c.T ? c.T : p.max_q > 0 ? p.max_q : (c.T + c.B - 1) / c.B;
    const int64_t rows = most * G;
    Plan pl;
    // Up to 16 rows a key head the warp-level kernel, then the tiles: 64 sequences of 2048 keys, 8 heads of
    // 128: 16 rows take 97 us in blocks of 16 and 104 in tiles, 24 take 178 and 105; d = 64: 16 rows 60
    // and 68, 24 rows 105 and 68.  One tile a block up to its 128 rows (96 rows of 64 dimensions 69 us,
    // 87 with two tiles; 160 rows 111 and 100), of 64 rows where that is enough (512 sequences of 128
    // keys, 64 rows: 75 us, 84 in a tile of 128; 96 rows: 129 and 88).
    pl.tc = rows > (128 / G) * G ? 2 : rows > 16 ? 1 : 0;
    pl.tile_rows = rows > (64 / G) * G ? 128 : 64;
    // (the tiles take whole tokens, so that TMA can bring their queries)
    pl.R = pl.tc ? (int)(pl.tc * (pl.tile_rows / G) * G) : 16;
    pl.kt = pl.tc ? 7 : 6;
    pl.box = pl.tc ? kTcBoxKeys : kRowsBoxKeys;
    const int sms = sm_count() ? sm_count() : 152;
    // no more shares than tiles there can be
    const int64_t keys = c.table_width * c.page_size;
    const double tiles = (double)c.Hkv * ((double)c.T * G / pl.R + c.B) * (double)((keys >> pl.kt) + 5);
    pl.fits = tiles < (double)kLongestLine;
    const int64_t full = (int64_t)sms * (pl.tc ? 3 - pl.tc : rows_blocks(c.d));
    pl.grid = (int)(tiles < (double)full ? (int64_t)tiles + 1 : full);
    if (pl.grid > kGroup * kGroup) pl.grid = kGroup * kGroup;  // as many parts as two levels merge
    const size_t slots = pl.tc ? 2 * (size_t)pl.grid : (size_t)all_slots(pl.grid);
    // Tiles that a boundary has to leave at either side of a cut.  Less cuts more finely and merges more, and
    // the tiles are between the two: with 4, 3 and 2 a mixed batch of chunks takes 76.9, 74.3 and 74.0 us, 512
    // tokens over 2048 keys 33.7, 30.3 and 29.3, 64 sequences of 2048 keys with 8 tokens 89.8, 88.3 and 86.9,
    // but 512 tokens over 512 keys 14.5, 14.5 and 16.9, 256 sequences of 512 keys with 64 tokens 146.3, 146.3
    // and 152.  Few rows, with 6, 4 and 3: one decode over 1024 keys 14.0, 13.0 and 12.9 us, over 8192 keys
    // 18.3, 17.0 and 16.9, 8 over 2048 keys 21.1, 19.7 and 19.8.
    pl.min_cut = pl.tc ? 3 : 4;
    pl.cuts = pl.grid > 1 && keys > (int64_t)((2 * pl.min_cut - 1) << pl.kt);
    if (!pl.cuts) {  // every block is shorter than two such parts: no states
        pl.off_ml = pl.off_u = pl.bytes = 0;
        return pl;
    }
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    pl.off_ml = up(pl.tc ? pl.grid * kCutBytes : slots * sizeof(unsigned long long));
    const size_t srows = pl.tc ? 128 * pl.tc : pl.R;  // rows a slot
    pl.off_u = pl.off_ml + up(slots * srows * 2 * sizeof(float));
    pl.bytes = pl.off_u + slots * srows * (size_t)c.d * sizeof(float);
    return pl;
}

// 4-D map over pages [num_pages, page_size, Hkv, d] with element strides s (page, slot, head); a
// box is 64 dimensions of `box` keys of one head of one page, 128-byte swizzle.  L2 fetches whole
// rows of a head and no more: with 64 dimensions (128 bytes) a 256-byte fetch would bring the next
// head's row too (351 MB read for 278 MB of cache, measured).
attn_status_t encode_pages(CUtensorMap *m, const void *ptr, const attn_paged_cache_t &c, const int64_t s[3], int box,
                           const char *name) {
    auto enc = get_encoder();
    if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    auto bytes = [](int64_t st, int64_t size) -> cuuint64_t { return size <= 1 ? 16u : (cuuint64_t)(st * 2); };
    cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page_size, (cuuint64_t)c.Hkv, (cuuint64_t)c.num_pages};
    cuuint64_t strides[3] = {bytes(s[1], c.page_size), bytes(s[2], c.Hkv), bytes(s[0], c.num_pages)};
    cuuint32_t b[4] = {64, (cuuint32_t)(c.page_size < box ? c.page_size : box), 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, b, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           c.d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ATTN_ERR_INVALID_ARG, "TMA descriptor for %s rejected (CUresult %d)", name, (int)r);
    return ATTN_OK;
}

// 3-D map over the packed queries [T, Hq, d]; a box is 64 dimensions of the G heads that share a
// key head, of `tokens` tokens: 128 rows or nearly.
attn_status_t encode_q(CUtensorMap *m, const attn_paged_fwd_params_t &p, int tokens) {
    auto enc = get_encoder();
    if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const int64_t G = p.Hq / p.cache.Hkv;
    auto bytes = [](int64_t st, int64_t size) -> cuuint64_t { return size <= 1 ? 16u : (cuuint64_t)(st * 2); };
    cuuint64_t dims[3] = {(cuuint64_t)p.cache.d, (cuuint64_t)p.Hq, (cuuint64_t)p.cache.T};
    cuuint64_t strides[2] = {bytes(p.q_stride[1], p.Hq), bytes(p.q_stride[0], p.cache.T)};
    cuuint32_t b[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
    cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p.q), dims, strides, b, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ATTN_ERR_INVALID_ARG, "TMA descriptor for q rejected (CUresult %d)", (int)r);
    return ATTN_OK;
}

// A tag for the marks of one call: never 0, another one every call of the process; the sequence starts
// from the clock, so that it does not repeat an earlier process's.
unsigned long long next_tag() {
    static std::atomic<unsigned long long> next{
        (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() * 2654435761ull};
    for (;;)
        if (const unsigned long long t = next.fetch_add(1)) return t;
}

int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

}  // namespace

size_t paged_fwd_workspace(const attn_paged_fwd_params_t &p) {
    const Plan pl = make_plan(p);
    return pl.fits ? pl.bytes : 0;
}

attn_status_t launch_paged_fwd(const attn_paged_fwd_params_t &p, void *workspace, cudaStream_t st) {
    const attn_paged_cache_t &c = p.cache;
    const Plan pl = make_plan(p);
    if (!pl.fits) return fail(ATTN_ERR_UNSUPPORTED, "Hkv (T Hq / Hkv + B) table_width page_size is too large");
    Args a;
    a.B = (int)c.B; a.T = (int)c.T; a.Hq = (int)p.Hq; a.Hkv = (int)c.Hkv; a.G = (int)(p.Hq / c.Hkv); a.causal = p.causal;
    a.R = pl.R; a.kt = pl.kt;
    bf16fwd::fast_div_params((uint32_t)a.G, a.g_m, a.g_s);
    bf16fwd::fast_div_params((uint32_t)a.R, a.r_m, a.r_s);
    a.page_log2 = log2_of(c.page_size);
    a.width = c.num_pages > 0 ? (int)c.table_width : 0;  // without pages there are no keys
    a.num_pages = (int)c.num_pages;
    // Least tiles a share.  Few rows: a cut costs 4 to 8 tiles (8 decodes over 2048 keys take 29 us with
    // shares of 4 tiles, 27 with 8).  128-row tiles: one sequence of 8192 keys, 8 tokens of 64/8 heads
    // takes 25.6 us with shares of 1, 20.0 of 4, 24.1 of 8; 64 tokens of 32/8 heads over 2048 keys
    // 20.7, 19.9 and 24.8.
    a.min_share = pl.tc ? 4 : 8;
    a.min_cut = pl.min_cut;
    // What a block's beginning and end cost, in tiles.  Batches of many blocks take any value near it (a
    // mixed one of 244 blocks of 3 to 32 tiles 73.5 us as 3, 74.4 as 4, 76.9 as 5; before later steps 134 as 0,
    // 97 as 4 or 6; 64 sequences of 2048 keys with 8 tokens of 64/8 heads 86.4, 88.3, 87.6).  Short items
    // decide: as the least share of the tiles, and half of that of few rows, it puts the cuts of an item of
    // 4 n tiles at whole shares (one sequence, 8 tokens of 64/8 heads over 2048 keys 19.7, 17.0, 19.2 us as
    // 3, 4, 5, over 8192 keys 22.3, 19.9, 22.4; few rows, one token over 1024 keys 14.8, 13.0, 14.9, 8 of
    // them over 2048 keys 20.8, 19.7, 20.9).
    a.cost = 4;
    a.scale_log2 = p.scale * kLog2e;
    a.q = static_cast<const __nv_bfloat16 *>(p.q);
    a.o = static_cast<__nv_bfloat16 *>(p.o);
    a.lse = p.lse;
    a.qs0 = p.q_stride[0]; a.qs1 = p.q_stride[1]; a.os0 = p.o_stride[0]; a.os1 = p.o_stride[1];
    a.bt = c.block_table; a.bt_s = c.table_stride; a.lens = c.kv_lens; a.cu = c.cu_q;
    char *ws = static_cast<char *>(workspace);
    a.marks = pl.cuts ? reinterpret_cast<unsigned long long *>(ws) : nullptr;
    a.ml = reinterpret_cast<float *>(ws + pl.off_ml);
    a.u = reinterpret_cast<float *>(ws + pl.off_u);
    a.tag = next_tag();
    a.flags = device_flags();
    if (!a.flags) return fail(ATTN_ERR_CUDA, "could not resolve the device error word");
    CUtensorMap mk{}, mv{};  // not used when there are no pages
    if (c.num_pages > 0) {
        attn_status_t r;
        if ((r = encode_pages(&mk, c.k_pages, c, c.k_stride, pl.box, "k_pages"))) return r;
        if ((r = encode_pages(&mv, c.v_pages, c, c.v_stride, pl.box, "v_pages"))) return r;
    }
    if (pl.tc) {
        CUtensorMap mq;
        const attn_status_t r = encode_q(&mq, p, pl.tile_rows / a.G);
        if (r) return r;
        return launch_paged_tc(mq, mk, mv, a, (int)c.d, pl.tc, pl.tile_rows, pl.grid, pl.cuts, st);
    }
    return launch_paged_rows(mk, mv, a, (int)c.d, pl.grid, st);
}

}  // namespace attn
