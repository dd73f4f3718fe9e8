// paged_rows.cu -- attention over a paged cache for few rows per key/value head (a decode step,
// a few drafted tokens): R = 16 rows a block.
//
// The bound is the cache, read once for all rows that share a key head.  Warp 4 copies 64-key
// tiles of K and V, page by page, into a ring of shared-memory stages with TMA (128-byte
// swizzle); warps 0-3 compute on them with warp-level tensor-core products (mma.sync m16n8k16):
// 16 rows are far below the 128 of a tcgen05 tile, and the tensor work is small next to the
// copy (64 keys x 16 rows x 128 dimensions take 128 products of the SM's warps against 0.75 us of copy, 32 KB at an
// SM's share of HBM).
//   S = Q K^T   warp w takes keys 16 w .. 16 w + 15 of the tile, all rows;
//   the row maxima of the four warps meet in shared memory, so that the CTA keeps one reference
//   per row; P = exp2(S - m) goes to shared memory in bf16, as the product takes it: half a step of 2^-8
//   of a weight, which averages out over the keys (the outputs lie 1.3 to 1.4 times as far from 64 bits
//   as with fp32 weights), where fp32 weights would want V in 32 bits too and twice the products;
//   O += P V    warp w takes dimensions [w D/4, (w + 1) D/4), all keys and rows.
// So no state is merged across warps, and a row's accumulator takes D/16 registers a thread.
//
// Two CTAs an SM with 96 KB of ring each, three with 64 KB at d = 64.  Measured (d 128, 32/8 heads): 64 ragged
// sequences to 8192 keys (1.32 GB) 205 us, 6.4 TB/s; one of 131072 keys (537 MB) 93 us, of which the
// ends of the call (lengths and pages before the first copy, the merge after the last) are about 12;
// d 64, 16 heads, 32 ragged sequences to 4096 keys x 4 tokens (275 MB) 58 us.  Short sequences pay
// about 1 us a block beside 0.9 us a tile: 1024 of 64 to 128 keys take 96 us for 80 us of whole pages.
#include <cudaTypedefs.h>

#include "paged.h"
#include "paged_merge.cuh"
#include "warp_mma.cuh"

namespace attn {

using namespace paged;
using namespace wmma16;

namespace {

constexpr int kConsumers = 128, kThreads = kConsumers + 32;
constexpr int KT = 64;  // keys a tile
constexpr int R = 16;   // rows a block

template <int D>
struct Rows {
    static constexpr int kPanels = D / 64;
    static constexpr int kPanelBytes = KT * 128;
    static constexpr int kTile = kPanels * kPanelBytes;  // K or V
    static constexpr int kBlocks = rows_blocks(D);
    static constexpr int kStages = (kBlocks == 3 ? 64 : 96) * 1024 / (2 * kTile);
    static constexpr int kQRow = 2 * D + 16, kPRow = 2 * KT + 16;  // padded: ldmatrix without bank conflicts
    static constexpr int kQOff = kStages * 2 * kTile;
    static constexpr int kPOff = kQOff + 2 * R * kQRow;  // this block's queries and the next one's
    static constexpr int kRedOff = kPOff + R * kPRow;    // [4][R] maxima, [4][R] sums
    static constexpr int kCtrlOff = kRedOff + 2 * 4 * R * 4;
};

struct Ctrl {
    uint64_t full[8], empty[8];
    Share share;
    int abort, last;
};

template <int D>
constexpr int smem_bytes() {
    constexpr int n = Rows<D>::kCtrlOff + (int)sizeof(Ctrl) + 1024;
    static_assert((n + 1024) * Rows<D>::kBlocks <= 228 * 1024, "shared memory of the CTAs an SM holds");
    return n;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// kState: with states of the packed tokens' rows (paged_state.cuh).
template <int D, bool kState>
__global__ void __launch_bounds__(kThreads, Rows<D>::kBlocks)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Args a) {
    using L = Rows<D>;
    constexpr int NS = L::kStages, DW = D / 4;  // DW: a warp's dimensions of O
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem + L::kCtrlOff);
    volatile int *abort = &ctrl->abort;
    float *red = reinterpret_cast<float *>(smem + L::kRedOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(&ctrl->full[s], 1);
            ptx::mbar_init(&ctrl->empty[s], 4);
        }
        ctrl->abort = 0;
        ptx::fence_mbar_init();
    }
    begin_after_earlier_grids(a, kState);
    ptx::launch_dependents();
    int *sums_of_32 = reinterpret_cast<int *>(smem);  // where the copies will go
    if (a.B > 32) {
        line_sums(a, sums_of_32);
        __syncthreads();
    }
    if (warp == 4) {
        const Share sh = find_share(a, blockIdx.x, gridDim.x, sums_of_32);
        if (lane == 0) ctrl->share = sh;
    }
    if (a.B > 32) ptx::fence_proxy_async_smem();  // the sums, before a copy takes their place
    __syncthreads();
    Walk w;
    if (!w.begin(a, ctrl->share)) {
        if (kState) end_after_earlier_grids(a);
        return;
    }

    if (warp == 4) {
        // ------------------------------------------------------------ TMA producer
        const int pb_log2 = min(a.page_log2, 6), boxes = KT >> pb_log2;
        const int box = lane / (2 * L::kPanels), part = lane % (2 * L::kPanels), panel = part >> 1;
        const CUtensorMap *tm = (part & 1) ? &tm_v : &tm_k;
        int st = 0, ph = 0, issued = 0;
        bool ok = true, more = true;
        // this lane's page among the 32 table entries from that of tile j on
        auto pages_at = [&](const Walk &p, int j) -> int {
            const int at = ((j * KT) >> a.page_log2) + lane;
            return p.keys > 0 && at <= (p.seq.n - 1) >> a.page_log2 ? __ldg(a.bt + p.b * a.bt_s + at) : 0;
        };
        int ahead = pages_at(w, w.j0);
        while (more && ok) {
            const Walk p = w;
            int pages = ahead, held = (p.j0 * KT) >> a.page_log2;
            // the next piece's pages load under this one's tiles
            more = w.next(a);
            if (more) ahead = pages_at(w, w.j0);
            for (int j = p.j0; p.keys > 0 && j < p.j1; ++j) {
                const int kv0 = j * KT;
                if ((min(kv0 + KT, p.seq.n) - 1) >> a.page_log2 >= held + 32) {
                    held = kv0 >> a.page_log2;
                    pages = pages_at(p, j);
                }
                if (pages < 0 || pages >= a.num_pages) pages = a.num_pages;  // outside the tensor: TMA fills zeros
                if (issued >= NS) ok = ptx::mbar_wait(&ctrl->empty[st], ph ^ 1, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                // boxes that hold a key of the sequence; each is kPanels copies of K and of V
                const int nbox = min(boxes, ((p.seq.n - kv0 - 1) >> pb_log2) + 1);
                if (lane == 0) ptx::mbar_arrive_expect_tx(&ctrl->full[st], (uint32_t)(nbox * 2 * L::kPanels) << (pb_log2 + 7));
                __syncwarp();
                const int key = kv0 + (box << pb_log2);
                const int page = __shfl_sync(0xffffffffu, pages, min(max((key >> a.page_log2) - held, 0), 31));
                if (box < nbox) {
                    uint8_t *dst = smem + st * 2 * L::kTile + (part & 1) * L::kTile + panel * L::kPanelBytes + (box << (pb_log2 + 7));
                    ptx::tma_load_4d(dst, tm, &ctrl->full[st], panel * 64, key & ((1 << a.page_log2) - 1), p.hk, page);
                    if (page == a.num_pages && part == 0) atomicOr(a.flags, kFlagBadIndex);
                }
                ++issued;
                if (++st == NS) { st = 0; ph ^= 1; }
            }
        }
        if (*abort) {  // copies in flight land before the CTA leaves
            const int n = min(issued, NS);
            for (int i = 0; i < n; ++i) {
                if (--st < 0) { st = NS - 1; ph ^= 1; }
                ptx::mbar_wait_quiet(&ctrl->full[st], ph, kWaitLimitNs);
            }
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3, mi = lane >> 3, mr = lane & 7;
    uint8_t *sP = smem + L::kPOff;
    float *sums = red + 4 * R;
    int st = 0, ph = 0, qb = 0;
    // a block's queries into one of the two buffers (rows past the block's end are zero)
    auto bring_q = [&](const Walk &p, int buf) {
        const int left = p.seq.nq * a.G - p.k * R;
        uint8_t *dst = smem + L::kQOff + buf * R * L::kQRow;
#pragma unroll
        for (int i = threadIdx.x; i < R * (D / 8); i += kConsumers) {
            const int r = i / (D / 8), c = i % (D / 8), row = p.k * R + r, tok = div_g(a, row);
            const bool in = r < left;
            const __nv_bfloat16 *src = a.q + (in ? (p.seq.q0 + tok) * a.qs0 + (p.hk * a.G + row - tok * a.G) * a.qs1 + c * 8 : 0);
            cp_async16(smem_addr(dst + r * L::kQRow + c * 16), src, in ? 16u : 0u);
        }
        cp_async_commit();
    };
    bring_q(w, 0);
    bool more = true;
    while (more) {
        const Walk p = w;
        const int rows = min(R, p.seq.nq * a.G - p.k * R), row0 = p.k * R;
        const uint8_t *sQ = smem + L::kQOff + qb * R * L::kQRow;
        int lim[2];  // keys < lim are visible to this lane's rows 8 e + g
        float m[2], l[2], o[DW / 8][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * e + g;
            lim[e] = (a.causal && r < rows) ? min(max(p.seq.n - p.seq.nq + div_g(a, row0 + r) + 1, 0), p.seq.n) : p.seq.n;
            m[e] = -INFINITY;
            l[e] = 0.f;
        }
        const int lim0 = a.causal ? min(max(p.seq.n - p.seq.nq + div_g(a, row0) + 1, 0), p.seq.n) : p.seq.n;
#pragma unroll
        for (int nt = 0; nt < DW / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
        cp_async_wait<0>();
        consumer_sync();  // the queries are there; the last piece is done with the other buffer and with sums
        more = w.next(a);
        qb ^= 1;
        if (more) bring_q(w, qb);

        for (int j = p.j0; p.keys > 0 && j < p.j1; ++j) {
            const int kv0 = j * KT;
            // a wait that gave up is reported; the walk goes on (the four warps keep meeting at the
            // same barriers) and ends, its waits returning at once
            ptx::mbar_wait(&ctrl->full[st], ph, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
            __syncwarp();
            uint8_t *sK = smem + st * 2 * L::kTile, *sV = sK + L::kTile;

            // S of this warp's 16 keys
            float s[2][4], s2[2][4];  // even and odd k steps: two chains of products
#pragma unroll
            for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = s2[0][e] = s2[1][e] = 0.f;
            const int krow = 16 * warp + (mi >> 1) * 8 + mr;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t kf[4];
                const int ch = (kk & 3) * 2 + (mi & 1);
                ldsm_x4(smem_addr(sK + (kk >> 2) * L::kPanelBytes + krow * 128 + ((ch ^ (krow & 7)) << 4)), kf);
                uint32_t qf[4];
                ldsm_x4(smem_addr(sQ + ((mi & 1) * 8 + mr) * L::kQRow + (2 * kk + (mi >> 1)) * 16), qf);
                mma_16816((kk & 1 ? s2 : s)[0], qf[0], qf[1], qf[2], qf[3], kf[0], kf[1]);
                mma_16816((kk & 1 ? s2 : s)[1], qf[0], qf[1], qf[2], qf[3], kf[2], kf[3]);
            }
            // scale, mask, row maxima of this warp's keys
            const bool edge = kv0 + KT > lim0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x[4] = {s[0][2 * e] + s2[0][2 * e], s[0][2 * e + 1] + s2[0][2 * e + 1],
                              s[1][2 * e] + s2[1][2 * e], s[1][2 * e + 1] + s2[1][2 * e + 1]};
                const int key = kv0 + 16 * warp + 2 * t;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] *= a.scale_log2;
                    if (edge && key + (i >> 1) * 8 + (i & 1) >= lim[e]) x[i] = -INFINITY;
                    s[i >> 1][2 * e + (i & 1)] = x[i];
                }
                float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                if (t == 0) red[warp * R + 8 * e + g] = mx;
            }
            // value rows past the sequence may hold anything: zero, so that 0 * v is 0
            const bool ragged = kv0 + KT > p.seq.n;
            if (ragged)
                for (int i = threadIdx.x; i < KT * L::kPanels * 8; i += kConsumers) {
                    const int key = (i >> 3) % KT, panel = (i >> 3) / KT;
                    if (kv0 + key >= p.seq.n)
                        *reinterpret_cast<uint4 *>(sV + panel * L::kPanelBytes + key * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
            consumer_sync();
            float al[2];
            bool moved = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * e + g;
                const float mn = fmaxf(fmaxf(m[e], fmaxf(red[r], red[R + r])), fmaxf(red[2 * R + r], red[3 * R + r]));
                const float ref = mn == -INFINITY ? 0.f : mn;
                al[e] = ptx::ex2(m[e] - ref);
                moved |= mn != m[e];
                m[e] = mn;
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = ptx::ex2(s[i >> 1][2 * e + (i & 1)] - ref);
                l[e] = fmaf(al[e], l[e], (p[0] + p[1]) + (p[2] + p[3]));
                uint8_t *pr = sP + r * L::kPRow + (16 * warp + 2 * t) * 2;
                *reinterpret_cast<uint32_t *>(pr) = pack_bf16(p[0], p[1]);
                *reinterpret_cast<uint32_t *>(pr + 16) = pack_bf16(p[2], p[3]);
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nt = 0; nt < DW / 8; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][e] *= al[e >> 1];
            }
            consumer_sync();
            // O of this warp's dimensions
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
                uint32_t pf[4];
                ldsm_x4(smem_addr(sP + ((mi & 1) * 8 + mr) * L::kPRow + (2 * kk + (mi >> 1)) * 16), pf);
                const int vrow = 16 * kk + (mi & 1) * 8 + mr;
#pragma unroll
                for (int nt = 0; nt < DW / 16; ++nt) {
                    uint32_t vf[4];
                    const int c = (warp * DW + nt * 16) / 8 + (mi >> 1);
                    ldsm_x4_trans(smem_addr(sV + (c >> 3) * L::kPanelBytes + vrow * 128 + (((c & 7) ^ (vrow & 7)) << 4)), vf);
                    mma_16816(o[2 * nt], pf[0], pf[1], pf[2], pf[3], vf[0], vf[1]);
                    mma_16816(o[2 * nt + 1], pf[0], pf[1], pf[2], pf[3], vf[2], vf[3]);
                }
            }
            if (ragged) ptx::fence_proxy_async_smem();  // the zeros above, before the stage's next copy
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->empty[st]);
            if (++st == NS) { st = 0; ph ^= 1; }
        }

        // ------------------------------------------------------------ the piece's rows
        // row sums: over the quad, then over the four warps
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = l[e];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if (t == 0) sums[warp * R + 8 * e + g] = v;
        }
        consumer_sync();
        if (kState) wait_for_states(a);
        const bool whole = p.whole();
        const int c0 = whole ? 0 : p.first_share(a);
        const long long slot = whole ? 0 : state_slot(blockIdx.x, c0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * e + g;
            if (r >= rows) continue;
            float sum = (sums[r] + sums[R + r]) + (sums[2 * R + r] + sums[3 * R + r]);
            if (whole) {
                const int tg = div_g(a, row0 + r), tok = p.seq.q0 + tg, h = p.hk * a.G + row0 + r - tg * a.G;
                if (kState) {
                    const StateAt at = state_at(a, D, p.hk, (long long)p.seq.q0 * a.G + row0 + r);
                    const Ending end = ending(a, at, tok, m[e], sum);
#pragma unroll
                    for (int nt = 0; nt < DW / 8; ++nt) {
                        float v[2] = {o[nt][2 * e], o[nt][2 * e + 1]};
                        end_u<2>(a, end, at, warp * DW + 2 * t + 8 * nt, v, sum);
                        o[nt][2 * e] = v[0];
                        o[nt][2 * e + 1] = v[1];
                    }
                    if (end.written) {
                        if (warp == 0 && t == 0) write_ml(end, at, m[e], sum);
                        continue;
                    }
                }
                const bool empty = sum == 0.f;  // a NaN is no empty row: it goes on into o and lse
                const float inv = empty ? 0.f : 1.f / sum;
                __nv_bfloat16 *orow = a.o + tok * a.os0 + h * a.os1 + warp * DW + 2 * t;
#pragma unroll
                for (int nt = 0; nt < DW / 8; ++nt)
                    *reinterpret_cast<uint32_t *>(orow + 8 * nt) = empty ? 0u : pack_bf16(o[nt][2 * e] * inv, o[nt][2 * e + 1] * inv);
                if (a.lse && warp == 0 && t == 0)
                    a.lse[(long long)tok * a.Hq + h] = empty ? -INFINITY : (m[e] + log2f(sum)) * kLn2;
            } else {
                float *ur = a.u + (slot * R + r) * D + warp * DW + 2 * t;
#pragma unroll
                for (int nt = 0; nt < DW / 8; ++nt)
                    *reinterpret_cast<float2 *>(ur + 8 * nt) = make_float2(o[nt][2 * e], o[nt][2 * e + 1]);
                if (warp == 0 && t == 0)
                    *reinterpret_cast<float2 *>(a.ml + (slot * R + r) * 2) = make_float2(sum == 0.f ? -INFINITY : m[e], sum);
            }
        }
        if (!whole)
            finish_cut(
                a, a.marks, gridDim.x, blockIdx.x, c0, p.parts(a, c0, p.tiles), threadIdx.x, &ctrl->last,
                [] {
                    consumer_sync();
                    return true;
                },
                [&](int n, int to, auto slot) {
                    merge_parts<D, 2, 8>(a, rows, n, to, threadIdx.x, slot, [&](int r, float (&v)[D / 32], float mx, float sum) {
                        end_row<D, kState>(a, p.seq.q0, p.hk, row0 + r, v, mx, sum);
                    });
                });
    }
    if (kState) end_after_earlier_grids(a);
}

template <int D>
attn_status_t launch(const CUtensorMap &mk, const CUtensorMap &mv, const Args &a, int grid, cudaStream_t st) {
    auto kern = a.state.mode == kNone ? paged_rows_kernel<D, false> : paged_rows_kernel<D, true>;
    const int smem = smem_bytes<D>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, mk, mv, a);
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "paged_rows launch: %s", cudaGetErrorString(e));
}

}  // namespace

attn_status_t launch_paged_rows(const CUtensorMap &mk, const CUtensorMap &mv, const Args &a, int d, int grid, cudaStream_t st) {
    return d == 64 ? launch<64>(mk, mv, a, grid, st) : launch<128>(mk, mv, a, grid, st);
}

}  // namespace attn
