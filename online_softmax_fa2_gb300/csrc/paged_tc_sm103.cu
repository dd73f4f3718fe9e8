// paged_tc_sm103.cu -- attention over a paged cache for many rows per key/value head (prompt
// chunks) on the 5th-generation tensor cores.
//
// A block is up to 256 rows of one (sequence, key/value head) -- tokens times the G query heads that
// share the head, so a key or value tile in shared memory serves all of them -- as two tiles A and
// B of floor(128 / G) tokens (128 rows, or 125 and more for G < 8) whose softmax warpgroups take turns
// with the tensor cores, as in the two-tile prefill kernel: while one warpgroup turns its S into P, the
// products of the other run.  One CTA an SM walks its share of the line of key tiles
// (paged_sched.cuh).  Where no sequence has more than one
// tile's rows, a block is one tile, and two CTAs an SM take turns instead: with tile B empty, nothing
// ran under tile A's softmax and between two blocks (1024 sequences of 128 keys, 16 tokens of 32/8
// heads of 128: 227 us with two tiles, 147 with one).
//
// Roles (384 threads, 256 with one tile: no warps 8-11, and half the columns):
//   warp 0       TMA producer: 128-key tiles of K and V into two rings, a box a page (or a part of
//                one), the boxes of a tile issued by as many lanes.
//   warp 1       tensor-core issuer (one thread); owns the 512 TMEM columns:
//                  S_A/P_A [0,128)  S_B/P_B [128,256)  O_A [256,384)  O_B [384,512).
//   warps 4-7    rows of tile A, one thread a row (its TMEM lane);  warps 8-11  rows of tile B.
//                One thread of each also asks for its tile's Q by TMA, for the next block
//                right after the last P of this one, so that its first S runs under this one's
//                epilogue.
//   warp 2       finds the share; warp 3 writes down what the merge has to know.
// A row's state over its part of an item goes to the workspace when the item is cut, and
// paged_tc_merge_kernel merges the parts.
//
// The row's 128 logits take most of a softmax thread's registers, and what is spilled goes to the little
// L1 that shared memory leaves: the accumulator is rescaled 16 columns at a time, and the walk lies in
// shared memory meanwhile (2048 tokens over 18432 keys 429 -> 404 us; 256 sequences of up to 512 keys,
// 64 tokens each, 192 -> 148; 1024 of 128 keys, 16 tokens, 240 -> 156).
//
// What bounds it: a 256 x 128 tile takes 1.5 us an SM (1.35 at the burst peak; the softmax of 128
// logits a thread takes turns with the products), 1.45 PFLOP/s for the chunk above, 0.77 of the burst peak and 0.85 of the
// sustained one; with few rows the cache (64 sequences of 2048 keys, 8 tokens of 64/8 heads: 106 us for
// 537 MB, 5.1 TB/s).  16 ragged sequences to 4096 keys, chunks to 512 tokens, 28/4 heads of 128: 75 us.
#include <cudaTypedefs.h>

#include "fwd_bf16_common.cuh"
#include "paged.h"
#include "paged_sched.cuh"

namespace attn {

using paged::Share;
using paged::Walk;

namespace {

using bf16fwd::BK;
using bf16fwd::BQ;
using bf16fwd::kPanelBytes;
using bf16fwd::kSmemMax;
using paged::kLn2;
using paged::kWaitLimitNs;

// 3-D tiled bulk-tensor load global -> shared, completion counted on `bar` (bytes).
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *m, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// Brings a 3-D box into L2.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *m, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(m)), "r"(c0),
                 "r"(c1), "r"(c2)
                 : "memory");
}

// 16 columns of this lane's TMEM row.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// NT row tiles a CTA.  Registers: launched at 168 a thread (384 x 168 = 64512), split 128 x 56 +
// 256 x 224 = 64512; with one tile at 128 (256 x 128 = 32768, two CTAs an SM), split 128 x 48 + 128 x 208.
constexpr int threads(int NT) { return 128 + 128 * NT; }
constexpr int launch_regs(int NT) { return NT == 2 ? 168 : 128; }
constexpr uint32_t issue_regs(int NT) { return NT == 2 ? 56 : 48; }
constexpr uint32_t softmax_regs(int NT) { return NT == 2 ? 224 : 208; }
static_assert(128 * (issue_regs(2) + 2 * softmax_regs(2)) <= threads(2) * launch_regs(2), "register split");
static_assert(128 * (issue_regs(1) + softmax_regs(1)) <= threads(1) * launch_regs(1), "register split");

struct Ctrl {
    uint64_t q_full[2], s_full[2], p_full[2], o_final[2];
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t final_mma;
    Share share;
    Walk parked[8];  // a softmax warp's walk while it goes through the key tiles of a piece
    uint32_t tmem_base;
    int abort;
};

// D dimensions, NT row tiles of QR rows.  A tile of 64 rows is multiplied as one of 128 whose upper half
// is whatever lies behind it in shared memory (a row's values reach that row alone).  The room that it
// leaves is L1's: 1024 sequences of 128 keys, 64 rows a head of 128, 157 us in tiles of 128, 147 in tiles
// of 64, 160 with a second K tile in its place; long sequences alike (87 to 89 us for 64 of 2048 keys).
template <int D, int NT, int QR>
struct Layout {
    static constexpr uint32_t kTmemCols = 256 * NT, kIssueRegs = issue_regs(NT), kSoftmaxRegs = softmax_regs(NT);
    static constexpr int kQPanel = QR * 128, kQTile = (D / 64) * kQPanel;
    static constexpr int kTile = (D / 64) * kPanelBytes;  // 128 keys of K or V
    static constexpr int kKStages = NT == 2 ? (D == 128 ? 3 : 4) : D == 64 ? 2 : 1;
    static constexpr int kVStages = NT == 2 ? (D == 128 ? 2 : 4) : D == 64 ? 2 : 1;
    static constexpr int kKOff = NT * kQTile, kVOff = kKOff + kKStages * kTile;
    static constexpr int kDataBytes = kVOff + kVStages * kTile;
    static constexpr int kBytes = kDataBytes + (int)sizeof(Ctrl);
    static_assert(NT == 2 ? kBytes <= kSmemMax : 2 * (kBytes + 1024) <= 228 * 1024, "shared memory budget");
};

// The row tiles of a piece: key tiles of each in the whole item, and in the piece.
struct Tiles {
    int t[2], n[2];
};
template <int NT>
__device__ __forceinline__ Tiles tiles_of(const paged::Args &a, const Walk &w) {
    Tiles r;
    if (NT == 1) {
        r.t[0] = (w.keys + BK - 1) / BK;
        r.n[0] = max(0, min(w.j1, r.t[0]) - w.j0);
        r.t[1] = r.n[1] = 0;
        return r;
    }
    const int rows = w.seq.nq * a.G - w.k * a.R, half = a.R >> 1;  // rows >= 1; tile A takes `half`
    int ka = w.keys;
    if (rows > half && a.causal) {
        const int last = paged::div_g(a, w.k * a.R + half - 1);
        ka = min(max(w.seq.n - w.seq.nq + last + 1, 0), w.seq.n);
    }
    r.t[0] = (ka + BK - 1) / BK;
    r.t[1] = rows > half ? (w.keys + BK - 1) / BK : 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) r.n[x] = max(0, min(w.j1, r.t[x]) - w.j0);
    return r;
}

// A cut item's states: (m, l) as [slot][tile][128 rows], u as [slot][tile][D / 4][128 rows][4], so
// that neighbouring rows (lanes) are neighbours in memory.
template <int NT>
__device__ __forceinline__ float2 *state_ml(const paged::Args &a, int slot, int x, int r) {
    return reinterpret_cast<float2 *>(a.ml) + (slot * NT + x) * (long long)BQ + r;
}
// The item whose first part is the end of a share, for the merge: parts of each tile (0: no such item),
// its block's first row and the sequence's rows, its first token, its key head.
struct Cut {
    int n[2], row0, end;
    int q0, hk, pad[2];
};
static_assert(sizeof(Cut) == 32 && sizeof(Cut) == paged::kCutBytes, "two 16-byte loads");

template <int D, int NT>
__device__ __forceinline__ float4 *state_u(const paged::Args &a, int slot, int x, int r) {
    return reinterpret_cast<float4 *>(a.u) + (slot * NT + x) * (long long)(BQ * D / 4) + r;
}

// u <- alpha u for this lane's D columns, 16 at a time: the row's 128 logits are in registers beside them.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t taddr, float alpha) {
#pragma unroll 1
    for (int cc = 0; cc < D / 16; ++cc) {
        uint32_t ov[16];
        tmem_ld16(taddr + cc * 16, ov);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < 16; ++t) asm volatile("" : "+r"(ov[t]));
#pragma unroll
        for (int t = 0; t < 16; ++t) ov[t] = __float_as_uint(__uint_as_float(ov[t]) * alpha);
        tmem_st16(taddr + cc * 16, ov);
    }
    ptx::tmem_st_wait();
}

// o = u / l and lse of this thread's row (+0.0 and -inf for a row that saw no key; nothing where orow is
// null).  A row of 32 columns at a time is 64 bytes in one thread; stored so, each of a warp's stores
// would touch 32 lines for 512 bytes, and the stores of a block take 2 us.  So every four lanes
// transpose their 4 x 4 pieces of 16 bytes first (two exchanges), and each store writes 64 bytes of
// eight rows.  Whole warp.
template <int D>
__device__ __forceinline__ void write_rows(uint32_t taddr, float l_run, float m_run, __nv_bfloat16 *orow, float *lse) {
    const int lane = threadIdx.x & 31, i = lane & 3;
    const bool empty = l_run == 0.f, b0 = i & 1, b1 = i & 2;  // a NaN is no empty row
    const float inv = empty ? 0.f : 1.f / l_run;
    uint4 *to[4];  // the quad's rows
#pragma unroll
    for (int j = 0; j < 4; ++j)
        to[j] = reinterpret_cast<uint4 *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(orow), (lane & ~3) | j));
#pragma unroll 1
    for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t ov[32], v[4][4];
        ptx::tmem_ld32(taddr + cc * 32, ov);
        ptx::tmem_ld_wait();
        ptx::reg_fence(ov);
#pragma unroll
        for (int t = 0; t < 16; ++t)
            v[t / 4][t % 4] = empty ? 0u : ptx::pack_bf16x2(__uint_as_float(ov[2 * t]) * inv, __uint_as_float(ov[2 * t + 1]) * inv);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, b0 ? v[j][e] : v[j + 1][e], 1);
                if (b0) v[j][e] = got;
                else v[j + 1][e] = got;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? v[j][e] : v[j + 2][e], 2);
                if (b1) v[j][e] = got;
                else v[j + 2][e] = got;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (to[j]) to[j][cc * 4 + i] = make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
    }
    if (lse) *lse = empty ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
}

template <int D, int NT, int QR>
__global__ void __launch_bounds__(threads(NT), NT == 2 ? 1 : 2)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const paged::Args a) {
    using L = Layout<D, NT, QR>;
    constexpr int KS = L::kKStages, VS = L::kVStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem + L::kDataBytes);
    volatile int *abort = &ctrl->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int x = 0; x < NT; ++x) {
            ptx::mbar_init(&ctrl->q_full[x], 1);
            ptx::mbar_init(&ctrl->s_full[x], 1);
            ptx::mbar_init(&ctrl->p_full[x], BQ);
            ptx::mbar_init(&ctrl->o_final[x], 1);
        }
        for (int s = 0; s < KS; ++s) {
            ptx::mbar_init(&ctrl->k_full[s], 1);
            ptx::mbar_init(&ctrl->k_empty[s], 1);
        }
        for (int s = 0; s < VS; ++s) {
            ptx::mbar_init(&ctrl->v_full[s], 1);
            ptx::mbar_init(&ctrl->v_empty[s], 1);
        }
        ptx::mbar_init(&ctrl->final_mma, 1);
        ctrl->abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&ctrl->tmem_base, L::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    int *sums_of_32 = reinterpret_cast<int *>(smem);  // where the copies will go
    if (a.B > 32) {
        paged::line_sums(a, sums_of_32);
        __syncthreads();
    }
    if (warp == 2) {
        const Share sh = paged::find_share(a, blockIdx.x, gridDim.x, sums_of_32);
        if (lane == 0) ctrl->share = sh;
    }
    if (a.B > 32) ptx::fence_proxy_async_smem();  // the sums, before a copy takes their place
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    // (a walk of its own in each role: one made here, before the roles part, would be spilled in all of them)

    if (warp < 4) {
        ptx::regs_dec<L::kIssueRegs>();
        Walk w;
        if (warp == 0 && w.begin(a, ctrl->share)) {
            // -------------------------------------------------------- TMA producer
            const int pb_log2 = min(a.page_log2, 7), boxes = BK >> pb_log2;
            int ks = 0, vs = 0, kp = 0, vp = 0, nk = 0, nv = 0;
            bool ok = true;
            do {
                if (w.keys == 0) continue;
                if (lane < NT * (D / 64)) {  // the block's queries into L2: they are asked for some tiles later
                    const int tok = w.seq.q0 + paged::div_g(a, w.k * a.R + (lane % NT) * (a.R / NT));
                    tma_prefetch_3d(&tm_q, (lane / NT) * 64, w.hk * a.G, tok);
                }
                const int *row = a.bt + w.b * a.bt_s;
                int held = -1, pages = 0;  // this lane holds the page of table entry held + lane
                for (int j = w.j0; j < w.j1; ++j) {
                    const int kv0 = j * BK, first = kv0 >> a.page_log2;
                    const int last = (min(kv0 + BK, w.seq.n) - 1) >> a.page_log2;
                    if (held < 0 || last >= held + 32) {
                        held = first;
                        const int at = held + lane, end = (w.seq.n - 1) >> a.page_log2;
                        pages = at <= end ? __ldg(row + at) : 0;
                        if (pages < 0 || pages >= a.num_pages) {
                            atomicOr(a.flags, kFlagBadIndex);
                            pages = a.num_pages;  // outside the tensor: TMA fills zeros
                        }
                    }
                    // boxes that hold a key of the sequence, D / 64 copies each
                    const int nbox = min(boxes, ((w.seq.n - kv0 - 1) >> pb_log2) + 1);
                    const uint32_t bytes = (uint32_t)(nbox * (D / 64)) << (pb_log2 + 7);
                    const int box = lane / (D / 64), panel = lane % (D / 64);
                    const int key = kv0 + (box << pb_log2), slot = key & ((1 << a.page_log2) - 1);
                    const int page = __shfl_sync(0xffffffffu, pages, min(max((key >> a.page_log2) - held, 0), 31));
                    const int off = panel * kPanelBytes + (box << (pb_log2 + 7));
                    if (nk >= KS) ok = ptx::mbar_wait(&ctrl->k_empty[ks], kp ^ 1, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&ctrl->k_full[ks], bytes);
                    __syncwarp();
                    if (box < nbox)
                        ptx::tma_load_4d(smem + L::kKOff + ks * L::kTile + off, &tm_k, &ctrl->k_full[ks], panel * 64, slot, w.hk, page);
                    ++nk;
                    if (++ks == KS) { ks = 0; kp ^= 1; }
                    if (nv >= VS) ok = ptx::mbar_wait(&ctrl->v_empty[vs], vp ^ 1, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&ctrl->v_full[vs], bytes);
                    __syncwarp();
                    if (box < nbox)
                        ptx::tma_load_4d(smem + L::kVOff + vs * L::kTile + off, &tm_v, &ctrl->v_full[vs], panel * 64, slot, w.hk, page);
                    ++nv;
                    if (++vs == VS) { vs = 0; vp ^= 1; }
                }
            } while (ok && w.next(a));
            if (!ok || *abort) {  // copies in flight land before the CTA leaves
                for (int i = min(nk, KS); i > 0; --i) {
                    if (--ks < 0) { ks = KS - 1; kp ^= 1; }
                    ptx::mbar_wait_quiet(&ctrl->k_full[ks], kp, kWaitLimitNs);
                }
                for (int i = min(nv, VS); i > 0; --i) {
                    if (--vs < 0) { vs = VS - 1; vp ^= 1; }
                    ptx::mbar_wait_quiet(&ctrl->v_full[vs], vp, kWaitLimitNs);
                }
            }
        } else if (warp == 3 && lane == 0 && a.marks) {
            // -------------------------------------------------------- what the merge has to know
            Cut cut{};
            bool more = w.begin(a, ctrl->share);
            while (more) {
                cut = Cut{};
                if (w.j0 == 0 && w.j1 < w.tiles) {
                    const Tiles tl = tiles_of<NT>(a, w);
                    for (int x = 0; x < NT; ++x) cut.n[x] = w.parts(a, blockIdx.x, tl.t[x]);
                    cut.row0 = w.k * a.R;
                    cut.end = w.seq.nq * a.G;
                    cut.q0 = w.seq.q0;
                    cut.hk = w.hk;
                }
                more = w.next(a);
            }
            reinterpret_cast<Cut *>(a.marks)[blockIdx.x] = cut;
        } else if (warp == 1 && lane == 0 && w.begin(a, ctrl->share)) {
            // -------------------------------------------------------- tensor-core issuer
            constexpr uint32_t kIdS = ptx::idesc_bf16_f32(BQ, BK, false);
            constexpr uint32_t kIdO = ptx::idesc_bf16_f32(BQ, D, true);
            const uint32_t q_lo = ptx::sdesc_lo(ptx::smem_u32(smem), 16);
            constexpr uint32_t kStep = L::kTile >> 4, kKLo = L::kKOff >> 4;
            constexpr uint32_t kVLo = (L::kVOff >> 4) + (((uint32_t)kPanelBytes >> 4) << 16) - (1u << 16);
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return ptx::mbar_wait(bar, parity, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
            };
            auto s_products = [&](int x, int ks) {
                uint32_t ql = q_lo, tm = tmem;
                ptx::opaque(ql);
                ptx::opaque(tm);
                const uint32_t qt = ql + x * (L::kQTile >> 4), kt = ql + kKLo + ks * kStep;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t qo = ((kk / 4) * L::kQPanel + (kk % 4) * 32) >> 4, ko = ((kk / 4) * kPanelBytes + (kk % 4) * 32) >> 4;
                    ptx::mma_ss_lo(tm + x * BQ, qt + qo, kt + ko, kIdS, kk > 0 ? 1u : 0u);
                }
                ptx::mma_commit(&ctrl->s_full[x]);
            };
            auto pv_products = [&](int x, int vs, bool first) {
                uint32_t ql = q_lo, tm = tmem;
                ptx::opaque(ql);
                ptx::opaque(tm);
                const uint32_t vt = ql + kVLo + vs * kStep;
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk)
                    ptx::mma_ts_lo(tm + NT * BQ + x * BQ, tm + x * BQ + kk * 8, vt + ((kk * 16 * 128) >> 4), kIdO,
                                   (!first || kk > 0) ? 1u : 0u);
            };
            // ring slots and barrier parities: 0 K full, 1 V full, 2/3 Q_A/Q_B, 4/5 P_A/P_B
            int ks = 0, vs = 0;
            uint32_t ph = 0;
            auto par = [&](int bit) -> uint32_t { return (ph >> bit) & 1u; };
            auto flip = [&](int bit) { ph ^= 1u << bit; };
            bool ok = true;
            do {
                if (w.keys == 0) continue;
                const Tiles tl = tiles_of<NT>(a, w);
                const int nmax = w.j1 - w.j0;
                if (!wait(&ctrl->k_full[ks], par(0))) break;
#pragma unroll
                for (int x = 0; x < NT; ++x)
                    if (ok && tl.n[x] > 0) {
                        ok = wait(&ctrl->q_full[x], par(2 + x));
                        if (!ok) break;
                        flip(2 + x);
                        ptx::tc_fence_after();
                        s_products(x, ks);
                    }
                if (!ok) break;
                ptx::mma_commit(&ctrl->k_empty[ks]);
                if (++ks == KS) { ks = 0; flip(0); }
                for (int i = 0; ok && i < nmax; ++i) {
                    // O_x += P_x V, then S_x of the next tile into the columns P_x occupies: the
                    // products of one thread execute in issue order
                    const bool more = i + 1 < nmax;
                    if (!wait(&ctrl->v_full[vs], par(1)) || (NT == 2 && more && !wait(&ctrl->k_full[ks], par(0)))) { ok = false; break; }
#pragma unroll
                    for (int x = 0; x < NT; ++x)
                        if (ok && i < tl.n[x]) {
                            ok = wait(&ctrl->p_full[x], par(4 + x));
                            if (!ok) break;
                            flip(4 + x);
                            ptx::tc_fence_after();
                            pv_products(x, vs, i == 0);
                            if (NT == 1) {  // a ring of one: the next V is asked for while its K is waited for
                                ptx::mma_commit(&ctrl->v_empty[vs]);
                                if (more && !wait(&ctrl->k_full[ks], par(0))) { ok = false; break; }
                            }
                            if (i == tl.n[x] - 1) ptx::mma_commit(&ctrl->o_final[x]);
                            else s_products(x, ks);
                        }
                    if (!ok) break;
                    if (NT == 2) ptx::mma_commit(&ctrl->v_empty[vs]);
                    if (more) {
                        ptx::mma_commit(&ctrl->k_empty[ks]);
                        if (++ks == KS) { ks = 0; flip(0); }
                    }
                    if (++vs == VS) { vs = 0; flip(1); }
                }
            } while (ok && w.next(a));
            ptx::mma_commit(&ctrl->final_mma);
            if (!ptx::mbar_wait_quiet(&ctrl->final_mma, 0, kWaitLimitNs)) atomicOr(a.flags, kFlagWaitTimeout);
        }
    } else {
        ptx::regs_inc<L::kSoftmaxRegs>();
        Walk w;
        // ------------------------------------------------------------ softmax warpgroups
        const int X = NT == 2 && warp >= 8 ? 1 : 0;
        const int r = (int)threadIdx.x - 128 - X * BQ;  // row in the tile == TMEM lane
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_col = X * BQ, o_col = NT * BQ + X * BQ;
        const float c = a.scale_log2;
        auto wait_warp = [&](uint64_t *bar, uint32_t parity) -> bool {
            const bool ok = ptx::mbar_wait(bar, parity, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
            return __all_sync(0xffffffffu, ok);
        };
        const int half = a.R / NT;
        // tile X's queries of a piece on their way into its buffer: whole tokens (those past the
        // sequence are another's, or zeros; rows past `half` hold whatever was there: a row's
        // values reach that row alone, and none of those is stored)
        int asked = 0;
        auto bring_q = [&](const Walk &p) {
            if (r == 0) {
                ptx::mbar_arrive_expect_tx(&ctrl->q_full[X], (uint32_t)half * (D * 2));
                const int tok = p.seq.q0 + paged::div_g(a, p.k * a.R + X * half);
#pragma unroll
                for (int pn = 0; pn < D / 64; ++pn)
                    tma_load_3d(smem + X * L::kQTile + pn * L::kQPanel, &tm_q, &ctrl->q_full[X], pn * 64, p.hk * a.G, tok);
                ++asked;
            }
        };
        auto has_tile = [&](const Walk &p) {
            const Tiles t = tiles_of<NT>(a, p);
            return (X ? t.n[1] : t.n[0]) > 0;
        };
        int vs = 0;                     // V ring slot and phase, for the rows that are zeroed
        uint32_t vph = 0, sph = 0, oph = 0;
        bool ok = true, more = w.begin(a, ctrl->share);
        if (more && has_tile(w)) bring_q(w);
        while (more && ok) {
            __syncwarp();
            const Tiles tl = tiles_of<NT>(a, w);
            const int n = X ? tl.n[1] : tl.n[0], tx = X ? tl.t[1] : tl.t[0], i0 = w.k * a.R + X * half, i = i0 + r, nmax = w.keys == 0 ? 0 : w.j1 - w.j0;
            const bool mine = r < half && i < w.seq.nq * a.G;
            const int tok = paged::div_g(a, i), seqn = w.seq.n;
            const int lim = a.causal && mine ? min(max(seqn - w.seq.nq + tok + 1, 0), seqn) : seqn;
            const int lim0 = a.causal ? min(max(seqn - w.seq.nq + paged::div_g(a, i0) + 1, 0), seqn) : seqn;
            const int j0 = w.j0, na = tl.n[0];
            if (lane == 0) ctrl->parked[warp - 4] = w;
            __syncwarp();
            float m_run = -INFINITY, l_run = 0.f;
            for (int jj = 0; jj < n; ++jj) {
                const int kv0 = (j0 + jj) * BK;
                if (!wait_warp(&ctrl->s_full[X], sph)) { ok = false; break; }
                sph ^= 1;
                ptx::tc_fence_after();
                float x[BK];
                bf16fwd::load_s_row(lane_addr + s_col, x);
                const float mt = bf16fwd::tile_logits<false>(x, c, kv0, kv0 + BK > lim0, lim);
                bool rescale;
                const float alpha = bf16fwd::update_max(mt, m_run, rescale);
                const float lsum = bf16fwd::tile_exp<false>(x, c, m_run);
                l_run = fmaf(alpha, l_run, lsum);
                if (__any_sync(0xffffffffu, rescale)) scale_o<D>(lane_addr + o_col, alpha);
                // value rows past the sequence may hold anything: the first of the two tiles that
                // uses this V zeroes them before its product reads them
                if (kv0 + BK > seqn && (X == 0 || jj >= na)) {
                    if (!wait_warp(&ctrl->v_full[vs], vph)) { ok = false; break; }
                    if (kv0 + r >= seqn) bf16fwd::zero_v_row<D>(smem + L::kVOff + vs * L::kTile, r);
                    ptx::fence_proxy_async_smem();
                }
                if (++vs == VS) { vs = 0; vph ^= 1; }
                // the weights go to the product in bf16, half a step of 2^-8 each (l_run has them in fp32):
                // V in 32 bits would take twice the room and run at half the rate
                bf16fwd::store_p(lane_addr + s_col, x);
                ptx::tc_fence_before();
                ptx::mbar_arrive(&ctrl->p_full[X]);
            }
            if (!ok) break;
            w = ctrl->parked[warp - 4];
            for (int jj = n; jj < nmax; ++jj)  // tiles that only the other rows see
                if (++vs == VS) { vs = 0; vph ^= 1; }
            // where this row goes, before the walk moves on
            const bool whole = w.j0 == 0 && w.j1 >= tx;
            const int c0 = w.first_share(a);
            const bool first = w.j0 == 0;
            __nv_bfloat16 *orow = nullptr;
            float *lrow = nullptr;
            if (mine) {
                const long long t = w.seq.q0 + tok;
                const int h = w.hk * a.G + i - tok * a.G;
                orow = a.o + t * a.os0 + h * a.os1;
                lrow = a.lse ? a.lse + t * a.Hq + h : nullptr;
            }
            // the next block's queries, under the last product of this one (this tile's last S, the
            // buffer's last reader, is done)
            more = w.next(a);
            if (more && has_tile(w)) bring_q(w);
            if (n == 0) {
                // no key tile here: the item's first share writes rows that see no key at all
                if (tx == 0 && first && mine) bf16fwd::write_empty_row<D>(orow, lrow);
                continue;
            }
            if (!wait_warp(&ctrl->o_final[X], oph)) { ok = false; break; }
            oph ^= 1;
            ptx::tc_fence_after();
            if (whole) {
                write_rows<D>(lane_addr + o_col, l_run, m_run, orow, lrow);
                ptx::tc_fence_before();
                continue;
            }
            // the state of this part, for paged_tc_merge_kernel
            const int slot = paged::state_slot(blockIdx.x, c0);
            *state_ml<NT>(a, slot, X, r) = make_float2(l_run == 0.f ? -INFINITY : m_run, l_run);
            float4 *u4 = state_u<D, NT>(a, slot, X, r);
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t ov[32];
                ptx::tmem_ld32(lane_addr + o_col + cc * 32, ov);
                ptx::tmem_ld_wait();
                ptx::reg_fence(ov);
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    u4[(cc * 8 + t) * BQ] = make_float4(__uint_as_float(ov[4 * t]), __uint_as_float(ov[4 * t + 1]),
                                                        __uint_as_float(ov[4 * t + 2]), __uint_as_float(ov[4 * t + 3]));
            }
            ptx::tc_fence_before();
        }
        // the queries asked for have arrived (their block's S waited for them, unless a wait gave up)
        if (!ok && asked > 0) ptx::mbar_wait_quiet(&ctrl->q_full[X], (asked - 1) & 1, kWaitLimitNs);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Merges the states of cut items ("How Does FlashAttention Preserve Global Softmax Across Tiles?",
// section 3), in share order.  CTA (c, tile, columns / 32) takes the item whose first part is the end of
// share c, if there is one; GR threads share a row, each every GR-th part: four where items are cut into
// many parts (launch_paged_tc), else one.  A kernel of its own: the merge's registers in the
// attention kernel's made its softmax spill (a 2048-token chunk 420 -> 800 us), and at its end one
// warpgroup merging 128 rows took 8 to 11 us.  No CTA of it finds room on an SM before the attention
// kernel's are done, so what it has to know is written down for it (Cut) instead of searched for.
constexpr int kMergeCols = 32;
template <int D, int NT, int GR>
__global__ void __launch_bounds__(BQ *GR, GR == 1 ? 8 : 2) paged_tc_merge_kernel(const paged::Args a) {
    static_assert(GR == 1 || GR == 4, "the sums below");
    __shared__ float top[GR][BQ], part[GR == 1 ? 1 : 2][GR == 1 ? 1 : BQ][kMergeCols + 1];
    const int c = blockIdx.x, X = blockIdx.y, col = blockIdx.z * kMergeCols, r = threadIdx.x % BQ, g = threadIdx.x / BQ;
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    const int4 *rec = reinterpret_cast<const int4 *>(reinterpret_cast<const Cut *>(a.marks) + c);
    const int4 c0 = __ldcg(rec), c1 = __ldcg(rec + 1);  // n[2], row0, end | q0, hk
    const int n = X ? c0.y : c0.x, half = a.R / NT, row = c0.z + X * half + r;
    if (n < 2) return;  // the whole CTA
    const bool mine = r < half && row < c0.w;
    const int parts = mine ? n : 0;
    auto slot = [&](int p) { return paged::state_slot(c + p, c); };
    float M = -INFINITY, sum = 0.f, v[kMergeCols];
#pragma unroll 4
    for (int p = g; p < parts; p += GR) M = fmaxf(M, __ldcg(state_ml<NT>(a, slot(p), X, r)).x);
    if (GR > 1) {
        top[g][r] = M;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < GR; ++k) M = fmaxf(M, top[k][r]);
    }
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int t = 0; t < kMergeCols; ++t) v[t] = 0.f;
#pragma unroll 1
    for (int p = g; p < parts; p += GR) {
        const float2 ml = __ldcg(state_ml<NT>(a, slot(p), X, r));
        const float4 *src = state_u<D, NT>(a, slot(p), X, r) + (col / 4) * BQ;
        float4 y[kMergeCols / 4];
#pragma unroll
        for (int t = 0; t < kMergeCols / 4; ++t) y[t] = __ldcg(src + t * BQ);
        const float f = ptx::ex2(ml.x - ref);
        sum = fmaf(f, ml.y, sum);
#pragma unroll
        for (int t = 0; t < kMergeCols / 4; ++t) {
            v[4 * t] = fmaf(f, y[t].x, v[4 * t]);
            v[4 * t + 1] = fmaf(f, y[t].y, v[4 * t + 1]);
            v[4 * t + 2] = fmaf(f, y[t].z, v[4 * t + 2]);
            v[4 * t + 3] = fmaf(f, y[t].w, v[4 * t + 3]);
        }
    }
    // groups 2 and 3 to 0 and 1, then 1 to 0 (through the buffer that it read itself)
#pragma unroll
    for (int from = GR / 2; from > 0; --from) {
        if (g >= from && g < 2 * from) {
            float *to = part[from == 2 ? g - 2 : 1][r];
#pragma unroll
            for (int t = 0; t < kMergeCols; ++t) to[t] = v[t];
            to[kMergeCols] = sum;
        }
        __syncthreads();
        if (g < from) {
            const float *other = part[from == 2 ? g : 1][r];
#pragma unroll
            for (int t = 0; t < kMergeCols; ++t) v[t] += other[t];
            sum += other[kMergeCols];
        }
    }
    if (g > 0 || !mine) return;
    const bool empty = sum == 0.f;  // (a part whose sum is NaN makes it NaN, whatever its weight)
    const float inv = empty ? 0.f : 1.f / sum;
    const int tok = paged::div_g(a, row), h = c1.y * a.G + row - tok * a.G;
    const long long t0 = c1.x + tok;
    uint4 *o4 = reinterpret_cast<uint4 *>(a.o + t0 * a.os0 + h * a.os1 + col);
#pragma unroll
    for (int t = 0; t < kMergeCols / 8; ++t) {
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pk[e] = empty ? 0u : ptx::pack_bf16x2(v[8 * t + 2 * e] * inv, v[8 * t + 2 * e + 1] * inv);
        o4[t] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
    if (a.lse && col == 0) a.lse[t0 * a.Hq + h] = empty ? -INFINITY : (M + log2f(sum)) * kLn2;
}

template <int D, int NT, int QR>
attn_status_t launch(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const paged::Args &a, int grid,
                     bool cuts, bool many, cudaStream_t st) {
    auto kern = paged_tc_kernel<D, NT, QR>;
    int smem = Layout<D, NT, QR>::kBytes;
    if (NT == 2 && smem < 116 * 1024) smem = 116 * 1024;  // one CTA an SM: it owns all 512 TMEM columns
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(grid), dim3(threads(NT)), smem, st, mq, mk, mv, a);
    if (e == cudaSuccess && cuts)
        e = many ? launch_pdl(paged_tc_merge_kernel<D, NT, 4>, dim3(grid, NT, D / kMergeCols), dim3(4 * BQ), 0, st, a)
                 : launch_pdl(paged_tc_merge_kernel<D, NT, 1>, dim3(grid, NT, D / kMergeCols), dim3(BQ), 0, st, a);
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "paged_tc launch: %s", cudaGetErrorString(e));
}
template <int D>
attn_status_t launch(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const paged::Args &a, int tiles,
                     int tile_rows, int grid, bool cuts, bool many, cudaStream_t st) {
    return tiles == 2        ? launch<D, 2, 128>(mq, mk, mv, a, grid, cuts, many, st)
           : tile_rows == 64 ? launch<D, 1, 64>(mq, mk, mv, a, grid, cuts, many, st)
                             : launch<D, 1, 128>(mq, mk, mv, a, grid, cuts, many, st);
}

}  // namespace

attn_status_t launch_paged_tc(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const paged::Args &a,
                              int d, int tiles, int tile_rows, int grid, bool cuts, cudaStream_t st) {
    // Items cut into more than four parts or so (16 tokens of 4 query heads over a key head, d 128, 131072
    // keys in all): 8 items 47 us with one thread a row, 27 with four; 32 items 25.8 and 23.2; 64 items
    // 24.9 and 25.7; the 77 us of a ragged batch of chunks become 82.
    const bool many = (double)a.Hkv * ((double)a.T * a.G / a.R + a.B) * 4. < (double)grid;
    return d == 64 ? launch<64>(mq, mk, mv, a, tiles, tile_rows, grid, cuts, many, st)
                   : launch<128>(mq, mk, mv, a, tiles, tile_rows, grid, cuts, many, st);
}

}  // namespace attn
