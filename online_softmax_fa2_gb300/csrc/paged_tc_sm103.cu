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
//   Over a cache in 8 bits warps 12-15 (with one tile warps 2 and 3) make fp16 operands of the codes, warp 0 brings K's and
//   warp 2 V's (with one tile warp 0 both): see "a cache of codes" below.
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

#include <type_traits>

#include "fwd_bf16_common.cuh"
#include "paged.h"
#include "q8.cuh"
#include "paged_state.cuh"

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
// Over codes two tiles have a warpgroup more: 512 x 128 = 65536, split 256 x 48 + 256 x 208.
constexpr bool own_converters(int NT, bool q8) { return q8 && NT == 2; }
constexpr int threads(int NT, bool q8) { return 128 + 128 * NT + (own_converters(NT, q8) ? 128 : 0); }
constexpr int launch_regs(int NT, bool q8) { return NT == 2 && !q8 ? 168 : 128; }
constexpr uint32_t issue_regs(int NT, bool q8) { return NT == 2 && !q8 ? 56 : 48; }
constexpr uint32_t softmax_regs(int NT, bool q8) { return NT == 2 && !q8 ? 224 : 208; }
constexpr bool split_fits(int NT, bool q8) {
    return (int)((threads(NT, q8) - 128 * NT) * issue_regs(NT, q8) + 128 * NT * softmax_regs(NT, q8)) <= threads(NT, q8) * launch_regs(NT, q8);
}
static_assert(split_fits(1, false) && split_fits(2, false) && split_fits(1, true) && split_fits(2, true), "register split");

template <int NT, int ST>
struct Ctrl {
    uint64_t q_full[NT], s_full[NT], p_full[NT], o_final[NT];
    uint64_t k_full[ST], k_empty[ST], v_full[ST], v_empty[ST];  // as many as a layout's stages, or more
    uint64_t final_mma;
    Share share;
    Walk parked[4 * NT];  // a softmax warp's walk while it goes through the key tiles of a piece
    uint32_t tmem_base;
    int abort;
};

// What a cache of codes needs besides.  A tile's codes come in four units of 64 keys, K's two and V's two, each with a place
// of its own; its scale bytes lie in a ring of two.  What the softmax has to know of a tile lies in a ring of eight (the
// conversion runs at most four tiles ahead of it, the producers two tiles ahead of that).
constexpr int kUnitKeys = 64, kNotes = 8;
template <int NT, int ST>
struct CtrlQ8 : Ctrl<NT, ST> {
    uint64_t q_ready[NT], raw_full[4], raw_empty[4];
    uint64_t sc_full[2][2], sc_empty[2][2];  // K's and V's scale bytes, two slots each
    volatile uint32_t notes[kNotes];  // of a tile: what its keys and, << 16, its values are relative to (next_unit)
};

// D dimensions, NT row tiles of QR rows.  A tile of 64 rows is multiplied as one of 128 whose upper half
// is whatever lies behind it in shared memory (a row's values reach that row alone).  The room that it
// leaves is L1's: 1024 sequences of 128 keys, 64 rows a head of 128, 157 us in tiles of 128, 147 in tiles
// of 64, 160 with a second K tile in its place; long sequences alike (87 to 89 us for 64 of 2048 keys).
template <int D, int NT, int QR, bool kQ8>
struct Layout {
    static constexpr uint32_t kTmemCols = 256 * NT, kIssueRegs = issue_regs(NT, kQ8), kSoftmaxRegs = softmax_regs(NT, kQ8);
    static constexpr int kQPanel = QR * 128, kQTile = (D / 64) * kQPanel;
    static constexpr int kTile = (D / 64) * kPanelBytes;  // 128 keys of K or V
    static constexpr int kKStages = kQ8 && NT == 2 ? 2 : NT == 2 ? (D == 128 ? 3 : 4) : D == 64 ? 2 : 1;
    static constexpr int kVStages = kQ8 && NT == 2 ? 2 : NT == 2 ? (D == 128 ? 2 : 4) : D == 64 ? 2 : 1;
    static constexpr int kKOff = NT * kQTile, kVOff = kKOff + kKStages * kTile;
    // codes: four units of [64 keys][D]; scale bytes [K, V][slot][128]
    static constexpr int kRawUnit = kUnitKeys * D, kRawOff = kVOff + kVStages * kTile;
    static constexpr int kScaleOff = kRawOff + (kQ8 ? 4 * kRawUnit : 0), kDataBytes = kScaleOff + (kQ8 ? 4 * BK : 0);
    static constexpr int kMostStages = kKStages > kVStages ? kKStages : kVStages;
    using Control = typename std::conditional<kQ8, CtrlQ8<NT, kMostStages>, Ctrl<NT, kMostStages>>::type;
    static constexpr int kBytes = kDataBytes + (int)sizeof(Control);
    // the warps that make operands of codes: a warpgroup of their own, or the two that are idle otherwise
    static constexpr int kConvWarps = own_converters(NT, kQ8) ? 4 : 2, kConvFirst = own_converters(NT, kQ8) ? 4 + 4 * NT : 2;
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
template <int D, bool kQ8>
__device__ __forceinline__ void write_rows(uint32_t taddr, float l_run, float m_run, int unit, __nv_bfloat16 *orow, float *lse) {
    const int lane = threadIdx.x & 31, i = lane & 3;
    const bool empty = l_run == 0.f, b0 = i & 1, b1 = i & 2;  // a NaN is no empty row
    const float inv = empty ? 0.f : 1.f / l_run, back = kQ8 ? q8::pow2_low(unit) : 1.f;
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
            v[t / 4][t % 4] = empty ? 0u
                              : kQ8 ? ptx::pack_bf16x2(__uint_as_float(ov[2 * t]) * inv * back, __uint_as_float(ov[2 * t + 1]) * inv * back)
                                    : ptx::pack_bf16x2(__uint_as_float(ov[2 * t]) * inv, __uint_as_float(ov[2 * t + 1]) * inv);
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

// The same of a row that leaves its state, or starts from one (paged_state.cuh); tok < 0: no row.
template <int D, bool kQ8>
__device__ __forceinline__ void end_row(const paged::Args &a, uint32_t taddr, float sum, float m, int unit, int tok, int g, int hk) {
    const bool on = tok >= 0;
    const paged::StateAt at = paged::state_at(a, D, hk, (long long)tok * a.G + g);
    const int h = hk * a.G + g;
    paged::wait_for_states(a);
    paged::Ending e{1.f, 0.f, false, false, nullptr, nullptr, false};
    if (on) e = paged::ending<true>(a, at, tok, m, sum);
    const bool empty = sum == 0.f;  // a NaN is no empty row
    const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll 1
    for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t ov[32];
        ptx::tmem_ld32(taddr + cc * 32, ov);
        ptx::tmem_ld_wait();
        ptx::reg_fence(ov);
        float v[32];
#pragma unroll
        for (int t = 0; t < 32; ++t) v[t] = __uint_as_float(ov[t]) * (kQ8 ? q8::pow2_low(unit) : 1.f);
        if (on) paged::end_u<32, D>(a, e, at, cc * 32, v, sum);
        if (on && !e.written) {
            uint4 *to = reinterpret_cast<uint4 *>(a.o + tok * a.os0 + h * a.os1 + cc * 32);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t pk[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) pk[e] = empty ? 0u : ptx::pack_bf16x2(v[8 * t + 2 * e] * inv, v[8 * t + 2 * e + 1] * inv);
                to[t] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
        }
        __syncwarp();  // the next columns are loaded by the whole warp
    }
    if (on && e.written) paged::write_ml(e, at, m, sum);
    else if (on && a.lse) a.lse[(long long)tok * a.Hq + h] = empty ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// And of one that sees no key here.
template <int D>
__device__ __forceinline__ void end_empty_row(const paged::Args &a, int tok, int g, int hk) {
    float m = -INFINITY, sum = 0.f;
    const paged::StateAt at = paged::state_at(a, D, hk, (long long)tok * a.G + g);
    const int h = hk * a.G + g;
    paged::wait_for_states(a);
    const paged::Ending e = paged::ending<true>(a, at, tok, m, sum);
    const bool empty = sum == 0.f;
    const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll 1
    for (int c = 0; c < D; c += 8) {
        float v[8] = {};
        paged::end_u<8, D>(a, e, at, c, v, sum);
        if (e.written) continue;
        uint32_t pk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pk[i] = empty ? 0u : ptx::pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
        *reinterpret_cast<uint4 *>(a.o + tok * a.os0 + h * a.os1 + c) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
    if (e.written) paged::write_ml(e, at, m, sum);
    else if (a.lse) a.lse[(long long)tok * a.Hq + h] = empty ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// Writes down what the merge has to know of the item that goes on past the share's end.  One thread.
template <int NT>
__device__ __forceinline__ void write_cut(const paged::Args &a, const Share &share) {
    if (!a.marks) return;
    Walk w;
    Cut cut{};
    bool more = w.begin(a, share);
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
}

// ---------------------------------------------------------------- a cache of codes
//
// The products take fp16, where codes are exact (paged_rows_q8.cu): warps make an operand of each 64 keys of codes that
// TMA brings, code times 2^(e - E) with an E that holds for as many tiles as all scale bytes e lie where that is
// exact, from 15 below it to 6 above it (448 * 2^6 < 65504); K's and V's go to the softmax, which takes K's into the
// tile's factor of the logits.  (Keys that no row of the block sees become zeros; so
// does beside others, from 25 below E on, a row of scale byte 0, of zeros nearly always.)
// A tile whose scale bytes lie further apart is a wide one: its codes go in as they are.  The softmax then multiplies S by the
// keys' own scales, or the weights by the values' own relative to what the row's largest weight times
// scale has been (odd_tile), so that a row loses nothing to keys that it does not see, or that weigh nothing in it,
// whatever their scales.  A row's u is in a unit of its own, which is V's E as long as that stays.
// The reference of a row's weights lies 2^7 below its maximum: as it may lag by 2^8, the weights reach 2^15, and lose
// bits from 2^-21 of the largest on, 2^-32 of it at most.
//
// What bounds it, as far as it is known: a 256 x 128 tile takes 3700 clocks, 3030 over bf16.  Shared memory is busy four fifths of
// them: the products read 192 KB of it (1536 clocks of 128 bytes), the codes come in by TMA (32 KB), and all loads and
// stores of the threads, the codes' way out to registers and back as fp16 above all, take 1150.  The issuer waits for operands
// 220 clocks of a tile, for weights 670, so the softmax's warps come next, which share their issue slots with the converting
// ones.  (The kernels spill 290 to 400 bytes a thread, 30 loads of them a tile over all warps.)  2048 tokens over 18432 keys of
// 32/8 heads 462 us against 394, 1.26 PFLOP/s; 16 ragged sequences to 4096 keys, chunks to 512 tokens, 28/4 heads 99 us against
// 75.  With every tile a wide one 2440 and 405 us.

// A tile's 128 scale bytes, four a lane (of keys past the held ones 0), against what its operand is relative to, `unit` (below 0:
// nothing yet), which stays as long as they all lie where codes are exact: from kExact below to kAbove above.  Otherwise the
// largest of them is the unit, or, where they lie further apart than kExact, the tile is a wide one, which keeps the unit and
// adds kWide.  (0, a row of zeros, and 255, a NaN, are none of them.)  Whole warp.
constexpr int kExact = 15, kAbove = 6, kWide = 256;
__device__ __forceinline__ int next_unit(int unit, uint32_t e4, int held) {
    const int left = held - 4 * (int)(threadIdx.x & 31), now = unit & 255;
    // nearly always: no key past the held ones, no byte of the two, all in range (two bytes a step)
    const uint32_t lo = e4 & 0xff00ffu, hi = (e4 >> 8) & 0xff00ffu;
    const uint32_t least = (uint32_t)max(now - kExact, 1) * 0x10001u, most = (uint32_t)min(now + kAbove, 254) * 0x10001u;
    const bool in = __vminu2(__vminu2(lo, hi), least) == least && __vmaxu2(__vmaxu2(lo, hi), most) == most;
    if (__all_sync(0xffffffffu, in && left >= 4 && unit >= 0)) return now;
    e4 &= left >= 4 ? 0xffffffffu : left > 0 ? 0xffffffffu >> (32 - 8 * left) : 0u;
    uint32_t big = 0, small = 255;
#pragma unroll 1
    for (int i = 0; i < 4; ++i, e4 >>= 8) {
        const uint32_t e = e4 & 255u;
        if (e - 1u < 254u) {
            big = max(big, e);
            small = min(small, e);
        }
    }
    const int b = (int)__reduce_max_sync(0xffffffffu, big), t = (int)__reduce_min_sync(0xffffffffu, small);
    if (unit >= 0 && b <= now + kAbove && t >= now - kExact) return now;  // (none: 0 and 255)
    if (b == 0) return unit < 0 ? 0 : now;
    return b - t <= kExact ? b : kWide | (unit < 0 ? 0 : now);
}

// A producer of K's (0), V's (1) or both kinds' (2) codes, in the order in which the converting warps come to them, and
// scale bytes, four a lane, loaded a tile ahead.  (Copies by lanes of a warp go out one after the other, each as long as a
// step here: with scale bytes in bulk copies of a page, 20 a tile, one producer of units in halves took 867 us for a
// chunk of 2048 tokens over 18432 keys, two 555.)  Its code is there once for both: the CTA's roles together fill the
// instruction cache, and what makes a loop longer costs all of them (two copies of this one 644 us for 554; waits in line
// 560 for 511; the converters' loop unrolled 638 for 544).  Whole warp.
template <class L, int D, int NT>
__device__ __forceinline__ void produce_codes(int kinds, const paged::Args &a, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                              const CUtensorMap &tm_v, uint8_t *smem, typename L::Control *ctrl, Walk &w) {
    const int steps = kinds == 2 ? 4 : 2;  // units a tile
    const int lane = threadIdx.x & 31;
    volatile int *abort = &ctrl->abort;
    if (!w.begin(a, ctrl->share)) return;
    const int pb_log2 = min(a.page_log2, 6);  // keys of a box
    auto unit_of = [&](int i) { return kinds == 2 ? 2 * (i & 1) + (i >> 1) : 2 * kinds + i; };
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        const bool ok = ptx::mbar_wait_short(bar, parity, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
        return __all_sync(0xffffffffu, ok);
    };
    int tile = 0, step = 0;
    bool ok = true;
    do {
        if (w.keys == 0) continue;
        if (kinds != 1 && lane < NT * (D / 64)) {  // the block's queries into L2: they are asked for some tiles later
            const int tok = w.seq.q0 + paged::div_g(a, w.k * a.R + (lane % NT) * (a.R / NT));
            tma_prefetch_3d(&tm_q, (lane / NT) * 64, w.hk * a.G, tok);
        }
        const int *row = a.bt + w.b * a.bt_s;
        int held = -1, pages = 0;  // this lane holds the page of table entry held + lane
        uint32_t ahead[2];
        int unit_k = -1, unit_v = -1;
        bool loaded = false;
        auto last_page = [&](int kv0) { return (min(kv0 + BK, w.seq.n) - 1) >> a.page_log2; };
        auto page_of = [&](int key) { return __shfl_sync(0xffffffffu, pages, min(max((key >> a.page_log2) - held, 0), 31)); };
        auto load_scales = [&](int kv0) {
            const int key = kv0 + 4 * lane, slot = key & ((1 << a.page_log2) - 1);
            int page = page_of(key);
            page = page < a.num_pages ? page : 0;  // (of a page out of range, whose codes are zeros, another page's)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (kinds == 2 || kinds == x) {
                    const uint8_t *at = x ? a.vs + page * a.vss[0] + w.hk * a.vss[1] : a.ks + page * a.kss[0] + w.hk * a.kss[1];
                    ahead[x] = key < w.seq.n ? __ldg(reinterpret_cast<const uint32_t *>(at + slot)) : 0u;
                }
        };
        // a step of the loop is tile j's copies, then what tile j + 1 needs: its unit is found under those copies (before its own
        // it took a 2048-token chunk over 18432 keys from 462 to 474 us)
        for (int j = w.j0 - 1; ok;) {
            if (j >= w.j0) {
                const int kv0 = j * BK;
#pragma unroll 1
                for (int x = kinds == 1; x <= (kinds > 0); ++x) {
                    if (tile > 1) ok = wait(&ctrl->sc_empty[x][tile & 1], ((tile >> 1) - 1) & 1);
                    if (!ok) break;
                    *reinterpret_cast<uint32_t *>(smem + L::kScaleOff + (2 * x + (tile & 1)) * BK + 4 * lane) = x ? ahead[1] : ahead[0];
                    if (lane == 0) reinterpret_cast<volatile uint16_t *>(&ctrl->notes[tile % kNotes])[x] = (uint16_t)(x ? unit_v : unit_k);
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&ctrl->sc_full[x][tile & 1]);
                }
                if (!ok) break;
                loaded = j + 1 < w.j1 && last_page(kv0 + BK) < held + 32;
                if (loaded) load_scales(kv0 + BK);
                const int held_keys = w.seq.n - kv0;  // of the tile: 1 or more
#pragma unroll 1
                for (step = 0; step < steps; ++step) {
                    const int u = unit_of(step);
                    if (tile > 0) ok = wait(&ctrl->raw_empty[u], (tile - 1) & 1);
                    if (!ok) break;
                    // boxes that hold a key of the sequence
                    const int c0 = (u & 1) * kUnitKeys;
                    const int nbox = held_keys > c0 ? min(kUnitKeys >> pb_log2, ((held_keys - c0 - 1) >> pb_log2) + 1) : 0;
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&ctrl->raw_full[u], (uint32_t)(nbox * D) << pb_log2);
                    __syncwarp();
                    const int key = kv0 + c0 + (lane << pb_log2), page = page_of(key);
                    if (lane < nbox)
                        ptx::tma_load_4d(smem + L::kRawOff + u * L::kRawUnit + ((lane << pb_log2) * D), u >= 2 ? &tm_v : &tm_k,
                                         &ctrl->raw_full[u], 0, key & ((1 << a.page_log2) - 1), w.hk, page);
                }
                if (!ok) break;
                step = 0;
                ++tile;
            }
            if (++j == w.j1) break;
            const int kv0 = j * BK;
            if (!loaded) {
                if (held < 0 || last_page(kv0) >= held + 32) {
                    held = kv0 >> a.page_log2;
                    const int at = held + lane, end = (w.seq.n - 1) >> a.page_log2;
                    pages = at <= end ? __ldg(row + at) : 0;
                    if (pages < 0 || pages >= a.num_pages) {
                        atomicOr(a.flags, kFlagBadIndex);
                        pages = a.num_pages;  // outside the tensor: TMA fills zeros
                    }
                }
                load_scales(kv0);
            }
            loaded = false;
#pragma unroll 1
            for (int x = kinds == 1; x <= (kinds > 0); ++x) {  // (keys that no row of the block sees have no say)
                const int unit = next_unit(x ? unit_v : unit_k, x ? ahead[1] : ahead[0], w.keys - kv0);
                if (x) unit_v = unit;
                else unit_k = unit;
            }
        }
    } while (ok && w.next(a));
    if (!ok || *abort)  // copies in flight land before the CTA leaves
        for (int i = 0; i < steps; ++i) {
            const int fills = tile + (i < step ? 1 : 0);
            if (fills > 0) ptx::mbar_wait_quiet(&ctrl->raw_full[unit_of(i)], (fills - 1) & 1, kWaitLimitNs);
        }
}

// 2^(e - top) for the scale byte e, 0 from 25 below on; NaN for 255.
__device__ __forceinline__ __half2 factor_of(int e, int top) {
    return __float2half2_rn(e == 255 ? NAN : __uint_as_float((uint32_t)max(e - top + 127, 0) << 23));
}

// A unit of codes to fp16, key 32 i + k times lane k's factor[i], into the panels of an operand; keys from `held` on become
// zeros.  Whole warp.  Eight neighbouring lanes take eight keys' chunks of one column: TMA's swizzle of the codes and that of
// the operand both spread those over all banks.
template <int D>
__device__ __forceinline__ void convert_unit(const uint8_t *raw, uint8_t *to, int held, __half2 factor0, __half2 factor1) {
    constexpr int C = D / 64;  // chunks of a key and lane, a panel apart
    const int lane = threadIdx.x & 31, r8 = lane & 7, col = lane >> 3;
    const uint8_t *from = raw + r8 * D;
    uint8_t *out = to + r8 * 128;
    const int lo = ((2 * col) ^ r8) << 4;
#pragma unroll 1
    for (int g = 0; g < kUnitKeys / 8; ++g) {
        uint4 x[C];
#pragma unroll
        for (int t = 0; t < C; ++t)
            x[t] = *reinterpret_cast<const uint4 *>(from + g * 8 * D + (((col + 4 * t) ^ (D == 128 ? r8 : (r8 >> 1) & 3)) << 4));
        const __half2 f2 = __shfl_sync(0xffffffffu, g < 4 ? factor0 : factor1, 8 * (g & 3) + r8);
#pragma unroll
        for (int t = 0; t < C; ++t) {
            uint32_t h[8];
            const uint32_t w[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                q8::decode4(w[k], h[2 * k], h[2 * k + 1]);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&h[2 * k + z]), f2);
                    h[2 * k + z] = *reinterpret_cast<const uint32_t *>(&v);
                }
            }
            uint8_t *at = out + g * 8 * 128 + t * kPanelBytes;
            *reinterpret_cast<uint4 *>(at + lo) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(at + (lo ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
    if (held < kUnitKeys) {  // the tile's end: whatever lies there
        __syncwarp();
#pragma unroll 1
        for (int i = max(held, 0) * 8 + lane; i < kUnitKeys * 8; i += 32)
#pragma unroll
            for (int t = 0; t < C; ++t) *reinterpret_cast<uint4 *>(to + t * kPanelBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
}


// A converting warp: with four of them a unit of each tile, with two K's or V's units.  (Four warps that took every unit
// together waited for one another and for a fence after each: 2450 clocks a tile beside the 2200 of the conversion.)
template <class L, int D>
__device__ __forceinline__ void convert_codes(const paged::Args &a, uint8_t *smem, typename L::Control *ctrl, Walk &w) {
    constexpr int H = 4 / L::kConvWarps;  // units of a tile
    const int lane = threadIdx.x & 31, cw = (int)(threadIdx.x >> 5) - L::kConvFirst;
    const int kind = cw * H >> 1, h0 = H == 1 ? cw & 1 : 0;  // 0 K, 1 V; the first of its units
    volatile int *abort = &ctrl->abort;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        const bool ok = ptx::mbar_wait_short(bar, parity, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
        return __all_sync(0xffffffffu, ok);
    };
    uint64_t *full = kind ? ctrl->v_full : ctrl->k_full, *empty = kind ? ctrl->v_empty : ctrl->k_empty;
    uint8_t *ring = smem + (kind ? L::kVOff : L::kKOff);
    const int stages = kind ? L::kVStages : L::kKStages;
    if (!w.begin(a, ctrl->share)) return;
    int st = 0;
    uint32_t sp = 1, tile = 0;  // a fresh barrier's phase before the first counts as complete
    do {
        if (w.keys == 0) continue;
        for (int j = w.j0; j < w.j1; ++j, ++tile) {
            const int held = w.keys - j * BK;  // (keys that no row of the block sees become zeros)
            const uint8_t *scales = smem + L::kScaleOff + (2 * kind + (tile & 1)) * BK;
            if (!wait(&ctrl->sc_full[kind][tile & 1], (tile >> 1) & 1u)) return;
            const int unit = reinterpret_cast<volatile uint16_t *>(&ctrl->notes[tile % kNotes])[kind];
            if (cw == 0) {  // V's note is there before the tile's S is
                if (!wait(&ctrl->sc_full[1][tile & 1], (tile >> 1) & 1u)) return;
                if (lane == 0) ptx::mbar_arrive(&ctrl->sc_empty[1][tile & 1]);
            }
            __half2 factor[2 * H];
#pragma unroll
            for (int i = 0; i < 2 * H; ++i) {
                const int e = scales[h0 * kUnitKeys + 32 * i + lane];
                factor[i] = factor_of(e, unit >= kWide && e != 255 ? e : unit & 255);
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->sc_empty[kind][tile & 1]);
            if (!wait(&empty[st], sp)) return;
#pragma unroll
            for (int k = 0; k < H; ++k) {
                const int h = h0 + k, u = 2 * kind + h;
                if (!wait(&ctrl->raw_full[u], tile & 1u)) return;
                convert_unit<D>(smem + L::kRawOff + u * L::kRawUnit, ring + st * L::kTile + h * kUnitKeys * 128, held - h * kUnitKeys,
                                factor[2 * k], factor[2 * k + 1]);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&ctrl->raw_empty[u]);
                ptx::fence_proxy_async_smem();  // the operand, before a product reads it
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&full[st]);
            }
            if (++st == stages) { st = 0; sp ^= 1; }
        }
    } while (w.next(a));
}

// Row r of a tile of queries from bf16 to fp16 in place, times a power of two that brings its largest finite element
// into [2^14, 2^15).  Returns the inverse.
template <int D>
__device__ __forceinline__ float queries_to_f16(uint8_t *tile, int panel_bytes, int r) {
    uint32_t top = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        const int ex = max((int)(top >> 7), 27);  // its exponent field, or one whose 2^(141 - ex) is finite
        const float up = __uint_as_float((uint32_t)(127 + 141 - ex) << 23);
#pragma unroll 2
        for (int c = 0; c < D / 8; ++c) {
            uint4 *at = reinterpret_cast<uint4 *>(tile + (c >> 3) * panel_bytes + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            const uint4 v = *at;
            uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (pass == 0) {
                    const uint32_t lo = x[k] & 0x7fffu, hi = (x[k] >> 16) & 0x7fffu;
                    top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                } else {
                    x[k] = q8::pack_f16(__uint_as_float(x[k] << 16) * up, __uint_as_float(x[k] & 0xffff0000u) * up);
                }
            }
            if (pass == 1) *at = make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
    return __uint_as_float((uint32_t)(max((int)(top >> 7), 27) - 14) << 23);
}

// The reference of a row's weights over codes: as bf16fwd::update_max, kRoom below the maximum.
constexpr float kRoom = 7.f;
// (moved: where it is set for the first time too, with an alpha of 1)
__device__ __forceinline__ float update_reference(float mt, float &m_run, bool &moved) {
    moved = mt > m_run + (kRoom + bf16fwd::kRescaleThreshold);
    if (!moved) return 1.f;
    const float alpha = m_run == -INFINITY ? 1.f : ptx::ex2(m_run - (mt - kRoom));
    m_run = mt - kRoom;
    return alpha;
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// 16 keys of a tile at this lane's row, and their scale bytes out of `word`, of which lane l has those of keys 4 l ..
template <class Body>
__device__ __forceinline__ void for_keys(uint32_t taddr, uint32_t word, Body body) {
#pragma unroll 1
    for (int cc = 0; cc < BK / 16; ++cc) {
        uint32_t r[16], e[4];
        tmem_ld16(taddr + cc * 16, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = __shfl_sync(0xffffffffu, word, 4 * cc + i);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < 16; ++t) asm volatile("" : "+r"(r[t]));
        body(cc, r, [&](int t) { return (int)((e[t / 4] >> (8 * (t % 4))) & 255u); });
    }
}

// Four scale bytes from position `key` of a sequence of n keys on, whose pages `row` lists.
__device__ __forceinline__ uint32_t load_scales(const paged::Args &a, const int *row, const uint8_t *from, long long stride, int key, int n) {
    if (key >= n) return 0u;
    int page = __ldg(row + (key >> a.page_log2));
    page = page < 0 || page >= a.num_pages ? 0 : page;
    return __ldg(reinterpret_cast<const uint32_t *>(from + page * stride + (key & ((1 << a.page_log2) - 1))));
}

// A row on its way through a piece: the reference and the sum of its weights, and u's unit, 2^(unit - 127); `own` where that has
// been the tiles' own so far, from which u may be scaled up by 2^24.
struct Row {
    float m, l;
    int unit, own;
};
// Logits from which a product that is rounded in the maximum and not in the exponent would part the two.
constexpr float kLarge = 1048576.f;
// The softmax of a tile that is a wide one in K or V, or relative to something else than a row's u, or with logits of kLarge: 16
// keys at a time, three times through S.  Its logits are the products times each key's own factor.  Its weights go in times
// 2^(e - unit), e a key's scale byte (of a tile that is not wide what V's operand is relative to), in a unit that brings the
// largest of these near 2^14, or keeps what u has; u is scaled to that unit.  Rare, and out of line, where it takes no room
// in the instruction cache: within the loop it took chunks from 463 to 634 us.  Returns whether the row can go on without.  Whole warp.
template <int D>
__device__ __noinline__ bool odd_tile(const paged::Args &a, const Walk &w, uint32_t s_addr, uint32_t o_addr, int kv0, int lim, int k_unit,
                                      int v_unit, float c_row, bool first, Row &row) {
    Row s = row;
    constexpr int kNone = -100000;
    constexpr uint32_t kLeast = 0x800000u, kMost = 0x7f000000u;  // bits of a weight less kLeast: below kMost, not 0 nor a NaN
    const int key = kv0 + 4 * (int)(threadIdx.x & 31);
    const int *pages = a.bt + w.b * a.bt_s;
    const bool even = v_unit < kWide;
    const uint32_t kw = k_unit < kWide ? (uint32_t)k_unit * 0x01010101u : load_scales(a, pages, a.ks + w.hk * a.kss[1], a.kss[0], key, w.seq.n);
    const uint32_t vw = even ? (uint32_t)v_unit * 0x01010101u : load_scales(a, pages, a.vs + w.hk * a.vss[1], a.vss[0], key, w.seq.n);
    float mt = -INFINITY;
    for_keys(s_addr, kw, [&](int cc, uint32_t (&r)[16], auto byte) {
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float x = __uint_as_float(r[t]) * q8::factor(c_row * q8::pow2((uint32_t)byte(t)));
            if (kv0 + 16 * cc + t >= lim) x = -INFINITY;
            mt = fmaxf(mt, x);
            r[t] = __float_as_uint(x);
        }
        tmem_st16(s_addr + cc * 16, r);
    });
    ptx::tmem_st_wait();
    bool rescale;
    const float alpha = update_reference(mt, s.m, rescale), ref = s.m == -INFINITY ? 0.f : s.m;
    float sum = 0.f;
    int need = kNone;  // the largest exponent, as in the bits of a weight, and scale byte
    for_keys(s_addr, vw, [&](int cc, uint32_t (&r)[16], auto byte) {
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const float p = ptx::ex2(__uint_as_float(r[t]) - ref);
            sum += p;
            r[t] = __float_as_uint(p);
            if (r[t] - kLeast < kMost && byte(t) != 255) need = max(need, (int)(r[t] >> 23) + byte(t));
        }
        tmem_st16(s_addr + cc * 16, r);
    });
    ptx::tmem_st_wait();
    const bool old = !first && s.l != 0.f && alpha > 0.f, some = need != kNone;
    s.l = fmaf(alpha, s.l, sum);
    const int now = s.unit, al = (int)(__float_as_uint(alpha) >> 23);
    need -= 127 + 14;
    int to = some ? need : kNone;
    if (old) to = max(to, now + al - 127 - (some && s.own ? 24 : 0));
    bool own = old && !some && s.own;
    if (even && (to == kNone || (to <= v_unit && to >= v_unit - 20))) {  // the tiles' own again
        to = v_unit;
        own = true;
    }
    to = to == kNone ? 127 : min(max(to, -15), 254);
    if (!first) {
        const int e = al + now - to;
        const float f = !old || e <= 0 ? 0.f : __uint_as_float((__float_as_uint(alpha) & 0x7fffffu) | ((uint32_t)min(e, 254) << 23));
        if (__any_sync(0xffffffffu, f != 1.f)) scale_o<D>(o_addr, f);
    }
    s.unit = to;
    s.own = own;
    for_keys(s_addr, vw, [&](int cc, uint32_t (&r)[16], auto byte) {
        uint32_t pk[8];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const int e = (int)(r[t] >> 23) + byte(t) - to;
            if (r[t] - kLeast < kMost && byte(t) != 255) r[t] = e <= 0 ? 0u : (r[t] & 0x7fffffu) | ((uint32_t)min(e, 254) << 23);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) pk[t] = q8::pack_f16(__uint_as_float(r[2 * t]), __uint_as_float(r[2 * t + 1]));
        tmem_st8(s_addr + cc * 8, pk);  // (columns that have been read)
    });
    ptx::tmem_st_wait();
    row = s;
    return even && to == v_unit && !(fabsf(s.m) > kLarge && s.m != -INFINITY);
}

__device__ __forceinline__ void store_p_f16(uint32_t taddr, const float (&x)[BK]) {
#pragma unroll
    for (int cc = 0; cc < BK / 64; ++cc) {
        uint32_t pk[32];
#pragma unroll
        for (int t = 0; t < 32; ++t) pk[t] = q8::pack_f16(x[cc * 64 + 2 * t], x[cc * 64 + 2 * t + 1]);
        ptx::tmem_st32(taddr + cc * 32, pk);
    }
    ptx::tmem_st_wait();
}

// kState: with states of the packed tokens' rows.
template <int D, int NT, int QR, bool kState, bool kQ8>
__global__ void __launch_bounds__(threads(NT, kQ8), NT == 2 ? 1 : 2)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ paged::Args a) {
    using L = Layout<D, NT, QR, kQ8>;
    using Control = typename L::Control;
    constexpr int KS = L::kKStages, VS = L::kVStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control *ctrl = reinterpret_cast<Control *>(smem + L::kDataBytes);
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
            ptx::mbar_init(&ctrl->k_full[s], kQ8 ? 2 : 1);  // (an arrival for each half of the tile)
            ptx::mbar_init(&ctrl->k_empty[s], 1);
        }
        for (int s = 0; s < VS; ++s) {
            ptx::mbar_init(&ctrl->v_full[s], kQ8 ? 2 : 1);
            ptx::mbar_init(&ctrl->v_empty[s], 1);
        }
        if constexpr (kQ8) {
            for (int x = 0; x < NT; ++x) ptx::mbar_init(&ctrl->q_ready[x], BQ);
            for (int s = 0; s < 4; ++s) {
                ptx::mbar_init(&ctrl->raw_full[s], 1);
                ptx::mbar_init(&ctrl->raw_empty[s], 1);
            }
            for (int x = 0; x < 2; ++x)
                for (int s = 0; s < 2; ++s) {
                    ptx::mbar_init(&ctrl->sc_full[x][s], 1);
                    ptx::mbar_init(&ctrl->sc_empty[x][s], L::kConvWarps / 2 + x);  // V's are read for the notes too
                }
        }
        ptx::mbar_init(&ctrl->final_mma, 1);
        ctrl->abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&ctrl->tmem_base, L::kTmemCols);
        ptx::tmem_relinquish();
    }
    paged::begin_after_earlier_grids(a, kState);
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

    if (warp < 4 || (own_converters(NT, kQ8) && warp >= L::kConvFirst)) {
        ptx::regs_dec<L::kIssueRegs>();
        Walk w;
        if (kQ8 && (warp == 0 || (own_converters(NT, kQ8) && warp == 2))) {
            if constexpr (kQ8) produce_codes<L, D, NT>(own_converters(NT, kQ8) ? warp >> 1 : 2, a, tm_q, tm_k, tm_v, smem, ctrl, w);
        } else if (kQ8 && warp >= L::kConvFirst && warp < L::kConvFirst + L::kConvWarps) {
            if constexpr (kQ8) {
                convert_codes<L, D>(a, smem, ctrl, w);
                if (!own_converters(NT, kQ8) && warp == 3 && lane == 0) write_cut<NT>(a, ctrl->share);
            }
        } else if (warp == 0 && w.begin(a, ctrl->share)) {
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
        } else if (warp == 3 && lane == 0) {
            write_cut<NT>(a, ctrl->share);
        } else if (warp == 1 && lane == 0 && w.begin(a, ctrl->share)) {
            // -------------------------------------------------------- tensor-core issuer
            constexpr uint32_t kIdS = kQ8 ? ptx::idesc_f16_f32(BQ, BK, false) : ptx::idesc_bf16_f32(BQ, BK, false);
            constexpr uint32_t kIdO = kQ8 ? ptx::idesc_f16_f32(BQ, D, true) : ptx::idesc_bf16_f32(BQ, D, true);
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
                        if constexpr (kQ8) ok = wait(&ctrl->q_ready[x], par(2 + x));
                        else ok = wait(&ctrl->q_full[x], par(2 + x));
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
        uint32_t vph = 0, sph = 0, oph = 0, qph = 0, tiles = 0;
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
            float c_row = c;
            int unit = 0, own = 1;  // u is in units of 2^(unit - 127) (odd_tile)
            int even = 0;           // that of V's operand which all rows' u is in, -1: none
            if constexpr (kQ8) {
                if (n > 0) {
                    if (!wait_warp(&ctrl->q_full[X], qph)) { ok = false; break; }
                    qph ^= 1;
                    if (QR == BQ || r < QR) c_row *= queries_to_f16<D>(smem + X * L::kQTile, L::kQPanel, r);
                    ptx::fence_proxy_async_smem();
                    ptx::mbar_arrive(&ctrl->q_ready[X]);
                }
            }
            int jj = 0;
            bool odd = false;
            for (;;) {
                for (; jj < n; ++jj) {
                    const int kv0 = (j0 + jj) * BK;
                    if (!wait_warp(&ctrl->s_full[X], sph)) { ok = false; break; }
                    sph ^= 1;
                    ptx::tc_fence_after();
                    float x[BK], ct = c_row, alpha;
                    bool moved;
                    if constexpr (kQ8) {
                        const uint32_t note = ctrl->notes[(tiles + jj) % kNotes];
                        if (jj == 0) even = unit = (int)(note >> 16);
                        odd = (note & kWide) || (int)(note >> 16) != even || (note >> 16) >= kWide;
                        if (odd) break;
                        ct = q8::factor(c_row * q8::pow2(note & 255u));
                    }
                    bf16fwd::load_s_row(lane_addr + s_col, x);
                    const float mt = bf16fwd::tile_logits<false>(x, ct, kv0, kv0 + BK > lim0, lim);
                    if constexpr (kQ8) {
                        const float before = m_run;
                        alpha = update_reference(mt, m_run, moved);
                        if (__any_sync(0xffffffffu, moved)) {
                            // (rows that are none of the block's hold anything, and have no say)
                            odd = __any_sync(0xffffffffu, mine && moved && fabsf(m_run) > kLarge);
                            if (odd) {
                                m_run = before;
                                break;
                            }
                            if (jj > 0) scale_o<D>(lane_addr + o_col, alpha);
                        }
                    } else {
                        alpha = bf16fwd::update_max(mt, m_run, moved);
                    }
                    const float lsum = bf16fwd::tile_exp<false>(x, ct, m_run);
                    l_run = fmaf(alpha, l_run, lsum);
                    if (!kQ8 && __any_sync(0xffffffffu, moved)) scale_o<D>(lane_addr + o_col, alpha);
                    // value rows past the sequence may hold anything: the first of the two tiles that
                    // uses this V zeroes them before its product reads them
                    if (!kQ8 && kv0 + BK > seqn && (X == 0 || jj >= na)) {
                        if (!wait_warp(&ctrl->v_full[vs], vph)) { ok = false; break; }
                        if (kv0 + r >= seqn) bf16fwd::zero_v_row<D>(smem + L::kVOff + vs * L::kTile, r);
                        ptx::fence_proxy_async_smem();
                    }
                    if (++vs == VS) { vs = 0; vph ^= 1; }
                    // the weights go to the product in bf16, half a step of 2^-8 each (l_run has them in fp32):
                    // V in 32 bits would take twice the room and run at half the rate
                    if constexpr (kQ8) store_p_f16(lane_addr + s_col, x);
                    else bf16fwd::store_p(lane_addr + s_col, x);
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&ctrl->p_full[X]);
                }
                if (!kQ8 || !odd) break;
                if constexpr (kQ8) {  // tile jj, behind the loop
                    const uint32_t note = ctrl->notes[(tiles + jj) % kNotes];
                    Row row{m_run, l_run, unit, own};
                    const bool fits = odd_tile<D>(a, ctrl->parked[warp - 4], lane_addr + s_col, lane_addr + o_col, (j0 + jj) * BK, lim,
                                                  (int)(note & 0xffffu), (int)(note >> 16), c_row, jj == 0, row);
                    even = __all_sync(0xffffffffu, fits || !mine) ? (int)(note >> 16) : -1;
                    m_run = row.m;
                    l_run = row.l;
                    unit = row.unit;
                    own = row.own;
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&ctrl->p_full[X]);
                    odd = false;
                    ++jj;
                }
            }
            if (!ok) break;
            if constexpr (kQ8) {  // relative to the maximum, as others' states are
                m_run += kRoom;
                l_run *= 0.0078125f;
                unit -= (int)kRoom;
            }
            w = ctrl->parked[warp - 4];
            tiles += nmax;
            for (jj = n; jj < nmax; ++jj)  // tiles that only the other rows see
                if (++vs == VS) { vs = 0; vph ^= 1; }
            // where this row goes, before the walk moves on
            const bool whole = w.j0 == 0 && w.j1 >= tx;
            const int c0 = w.first_share(a), parts = kState ? w.parts(a, c0, tx) : 0;
            const bool first = w.j0 == 0;
            __nv_bfloat16 *orow = nullptr;
            float *lrow = nullptr;
            int to_tok = -1, to_g = 0;
            const int hk = w.hk;
            if (mine) {
                const long long t = w.seq.q0 + tok;
                const int h = w.hk * a.G + i - tok * a.G;
                if (kState) {
                    to_tok = (int)t;
                    to_g = i - tok * a.G;
                } else {
                    orow = a.o + t * a.os0 + h * a.os1;
                    lrow = a.lse ? a.lse + t * a.Hq + h : nullptr;
                }
            }
            // the next block's queries, under the last product of this one (this tile's last S, the
            // buffer's last reader, is done)
            more = w.next(a);
            if (more && has_tile(w)) bring_q(w);
            if (n == 0) {
                // no key tile here: the item's first share writes rows that see no key at all
                if (tx == 0 && first && mine) {
                    if (kState) end_empty_row<D>(a, to_tok, to_g, hk);
                    else bf16fwd::write_empty_row<D>(orow, lrow);
                }
                continue;
            }
            if (!wait_warp(&ctrl->o_final[X], oph)) { ok = false; break; }
            oph ^= 1;
            ptx::tc_fence_after();
            if (whole) {
                if (kState) end_row<D, kQ8>(a, lane_addr + o_col, l_run, m_run, unit, to_tok, to_g, hk);
                else write_rows<D, kQ8>(lane_addr + o_col, l_run, m_run, unit, orow, lrow);
                ptx::tc_fence_before();
                continue;
            }
            // the state of this part, for paged_tc_merge_kernel
            if (kState && a.state.marks && first && mine)
                a.state.ml[paged::state_at(a, D, hk, (long long)to_tok * a.G + to_g).ml] =
                    make_float2(paged::cut_row(c0, X, r, parts), paged::kCutRow);
            const int slot = paged::state_slot(blockIdx.x, c0);
            *state_ml<NT>(a, slot, X, r) = make_float2(l_run == 0.f ? -INFINITY : m_run, l_run);
            float4 *u4 = state_u<D, NT>(a, slot, X, r);
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t ov[32];
                ptx::tmem_ld32(lane_addr + o_col + cc * 32, ov);
                ptx::tmem_ld_wait();
                ptx::reg_fence(ov);
                if constexpr (kQ8) {
                    const float vu = q8::pow2_low(unit);
#pragma unroll
                    for (int t = 0; t < 32; ++t) ov[t] = __float_as_uint(__uint_as_float(ov[t]) * vu);
                }
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
    if (kState) paged::end_after_earlier_grids(a);
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Merges the states of cut items ("How Does FlashAttention Preserve Global Softmax Across Tiles?",
// section 3), in share order.  A kernel of its own: the merge's registers in the attention kernel's made its softmax spill
// (a 2048-token chunk 420 -> 800 us), and at its end one warpgroup merging 128 rows took 8 to 11 us.  No CTA of it finds
// room on an SM before the attention kernel's are done, so what it has to know is written down for it (Cut) instead of
// searched for.
//
// CTA (c, tile, columns) takes the item whose first part is the end of share c, if there is one; with GR = 4, where
// items are cut into many parts (launch_paged_tc_merge), four threads share a row, each every fourth part, and a CTA looks
// at merge_shares shares, so that the few CTAs with work and the others are one wave: 64 tokens of 32/8 heads over 8192
// keys, in 19 parts an item, 8.5 us with a CTA a share and 32 columns, 6 so.
// With states a thread takes 16 columns, so that what it asks for ahead stays in registers (of 32, the rows that were finished
// alone took 8 us more).
constexpr int merge_cols(int GR, bool state) { return GR == 1 && !state ? 32 : 16; }
constexpr int merge_shares(int GR) { return GR == 1 ? 1 : 8; }

template <int D, int NT, int GR, bool kState>
__device__ __forceinline__ void merge_item(const paged::Args &a, int c, int X, int col, int4 c0, int4 c1,
                                           float (&top)[GR][BQ], float (&part)[GR == 1 ? 1 : 2][GR == 1 ? 1 : BQ][merge_cols(GR, kState) + 1]) {
    constexpr int C = merge_cols(GR, kState);
    const int r = threadIdx.x % BQ, g = threadIdx.x / BQ;
    const int n = X ? c0.y : c0.x, half = a.R / NT, row = c0.z + X * half + r;
    const bool mine = r < half && row < c0.w;
    const int parts = mine ? n : 0;
    auto slot = [&](int p) { return paged::state_slot(c + p, c); };
    float M = -INFINITY, sum = 0.f, v[C];
    const paged::StateAt at = paged::state_at(a, D, c1.y, (long long)c1.x * a.G + row);
    paged::Earlier<kState ? C : 4, D> earlier;  // under the parts, as far as registers go
    if (kState) {
        earlier.ask_ml(a, at, c1.x + paged::div_g(a, row), mine && g == 0);
        if (GR == 1) earlier.ask_u(a, at, col);
    }
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
    for (int t = 0; t < C; ++t) v[t] = 0.f;
#pragma unroll(kState && GR == 1 ? 2 : 1)
    for (int p = g; p < parts; p += GR) {
        const float2 ml = __ldcg(state_ml<NT>(a, slot(p), X, r));
        const float4 *src = state_u<D, NT>(a, slot(p), X, r) + (col / 4) * BQ;
        float4 y[C / 4];
#pragma unroll
        for (int t = 0; t < C / 4; ++t) y[t] = __ldcg(src + t * BQ);
        const float f = ptx::ex2(ml.x - ref);
        sum = fmaf(f, ml.y, sum);
#pragma unroll
        for (int t = 0; t < C / 4; ++t) {
            v[4 * t] = fmaf(f, y[t].x, v[4 * t]);
            v[4 * t + 1] = fmaf(f, y[t].y, v[4 * t + 1]);
            v[4 * t + 2] = fmaf(f, y[t].z, v[4 * t + 2]);
            v[4 * t + 3] = fmaf(f, y[t].w, v[4 * t + 3]);
        }
    }
    if (kState && GR > 1) earlier.ask_u(a, at, col);
    // groups 2 and 3 to 0 and 1, then 1 to 0 (through the buffer that it read itself)
#pragma unroll
    for (int from = GR / 2; from > 0; --from) {
        if (g >= from && g < 2 * from) {
            float *to = part[from == 2 ? g - 2 : 1][r];
#pragma unroll
            for (int t = 0; t < C; ++t) to[t] = v[t];
            to[C] = sum;
        }
        __syncthreads();
        if (g < from) {
            const float *other = part[from == 2 ? g : 1][r];
#pragma unroll
            for (int t = 0; t < C; ++t) v[t] += other[t];
            sum += other[C];
        }
    }
    if (g > 0 || !mine) return;
    if constexpr (kState) {
        if (!paged::is_wanted(a, c1.x + paged::div_g(a, row))) return;
        earlier.join_parts(a, col);
        earlier.merge(v, M, sum);
    }
    const bool empty = sum == 0.f;  // (a part whose sum is NaN makes it NaN, whatever its weight)
    const float inv = empty ? 0.f : 1.f / sum;
    const int tok = paged::div_g(a, row), h = c1.y * a.G + row - tok * a.G;
    const long long t0 = c1.x + tok;
    uint4 *o4 = reinterpret_cast<uint4 *>(a.o + t0 * a.os0 + h * a.os1 + col);
#pragma unroll
    for (int t = 0; t < C / 8; ++t) {
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pk[e] = empty ? 0u : ptx::pack_bf16x2(v[8 * t + 2 * e] * inv, v[8 * t + 2 * e + 1] * inv);
        o4[t] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
    if (a.lse && col == 0) a.lse[t0 * a.Hq + h] = empty ? -INFINITY : (M + log2f(sum)) * kLn2;
}

// Rows that the prefixes' attention has finished, 128 of a key head, and the own keys' states of them: eight columns a
// thread, GR groups of them a CTA.
template <int D, int GR>
__device__ __forceinline__ void merge_whole(const paged::Args &a, int block) {
    constexpr int C = 8, Z = D / C / GR;
    const int n = a.T * a.G, blocks = (n + BQ - 1) / BQ, rows = block / Z, hk = rows / blocks, row = rows % blocks * BQ + threadIdx.x % BQ;
    if (hk >= a.Hkv || row >= n) return;
    const int tok = paged::div_g(a, row), h = hk * a.G + row - tok * a.G, col = (block % Z * GR + threadIdx.x / BQ) * C;
    if (!paged::is_wanted(a, tok)) return;
    const paged::StateAt at = paged::state_at(a, D, hk, row);
    paged::Earlier<C> own;
    own.ask_ml(a, at, tok, true);
    if (!own.on) return;
    own.ask_u(a, at, col);
    const float4 *u = reinterpret_cast<const float4 *>(a.state.u2) + at.u + col / 4 * at.n;
    const float2 ml = __ldcg(a.state.ml2 + at.ml);
    float m = ml.x, sum = ml.y, v[C];  // (of a cut row whatever lies there)
#pragma unroll
    for (int c = 0; c < C; c += 4) *reinterpret_cast<float4 *>(v + c) = __ldcg(u + c / 4 * at.n);
    if (ml.y == paged::kCutRow) return;
    own.merge(v, m, sum);
    const bool empty = sum == 0.f;
    const float inv = empty ? 0.f : 1.f / sum;
    uint32_t pk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pk[i] = empty ? 0u : ptx::pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
    *reinterpret_cast<uint4 *>(a.o + tok * a.os0 + h * a.os1 + col) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    if (a.lse && col == 0) a.lse[(long long)tok * a.Hq + h] = empty ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// Blocks from `items` on take rows that were finished.
template <int D, int NT, int GR, bool kState>
__global__ void __launch_bounds__(BQ *GR, GR > 1 ? 2 : kState ? 4 : 8) paged_tc_merge_kernel(const paged::Args a, int shares, int items) {
    static_assert(GR == 1 || GR == 4, "the sums of merge_item");
    constexpr int S = merge_shares(GR);
    __shared__ float top[GR][BQ], part[GR == 1 ? 1 : 2][GR == 1 ? 1 : BQ][merge_cols(GR, kState) + 1];
    const int X = blockIdx.y, col = blockIdx.z * merge_cols(GR, kState);
    ptx::grid_dep_wait();
    ptx::launch_dependents();
    if (kState && (int)blockIdx.x >= items) {
        merge_whole<D, GR>(a, (((int)blockIdx.x - items) * NT + X) * (int)gridDim.z + (int)blockIdx.z);
        return;
    }
    // a record a lane: one look at all
    const int4 *rec = reinterpret_cast<const int4 *>(reinterpret_cast<const Cut *>(a.marks) + blockIdx.x * S);
    const int lane = threadIdx.x & 31;
    int4 r0 = make_int4(0, 0, 0, 0), r1 = r0;  // n[2], row0, end | q0, hk
    if (lane < S && (int)blockIdx.x * S + lane < shares) {
        r0 = __ldcg(rec + 2 * lane);
        r1 = __ldcg(rec + 2 * lane + 1);
    }
    bool again = false;
#pragma unroll 1
    for (unsigned cut = __ballot_sync(0xffffffffu, (X ? r0.y : r0.x) >= 2); cut; cut &= cut - 1) {
        const int i = __ffs(cut) - 1;
        auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, i); };
        const int4 c0 = make_int4(of(r0.x), of(r0.y), of(r0.z), of(r0.w)), c1 = make_int4(of(r1.x), of(r1.y), 0, 0);
        if (GR > 1 && again) __syncthreads();  // the last one's buffers
        again = true;
        merge_item<D, NT, GR, kState>(a, blockIdx.x * S + i, X, col, c0, c1, top, part);
    }
}

template <int D, int NT, int QR, bool kQ8>
attn_status_t launch(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const paged::Args &a, int grid, cudaStream_t st) {
    auto kern = a.state.mode != paged::kNone ? paged_tc_kernel<D, NT, QR, true, kQ8> : paged_tc_kernel<D, NT, QR, false, kQ8>;
    int smem = Layout<D, NT, QR, kQ8>::kBytes;
    if (NT == 2 && smem < 116 * 1024) smem = 116 * 1024;  // one CTA an SM: it owns all 512 TMEM columns
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(grid), dim3(threads(NT, kQ8)), smem, st, mq, mk, mv, a);
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "paged_tc launch: %s", cudaGetErrorString(e));
}
template <int D, bool kQ8>
attn_status_t launch(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const paged::Args &a, int tiles,
                     int tile_rows, int grid, cudaStream_t st) {
    return tiles == 2        ? launch<D, 2, 128, kQ8>(mq, mk, mv, a, grid, st)
           : tile_rows == 64 ? launch<D, 1, 64, kQ8>(mq, mk, mv, a, grid, st)
                             : launch<D, 1, kQ8 && D == 128 ? 64 : 128, kQ8>(mq, mk, mv, a, grid, st);
}

template <int D, int NT, int GR, bool kState>
cudaError_t launch_merge(const paged::Args &a, int grid, cudaStream_t st) {
    constexpr int Z = D / merge_cols(GR, kState);
    const int items = a.marks ? (grid + merge_shares(GR) - 1) / merge_shares(GR) : 0;
    const int whole = a.state.ml2 ? (a.Hkv * ((a.T * a.G + BQ - 1) / BQ) * (D / 8 / GR) + NT * Z - 1) / (NT * Z) : 0;
    return launch_pdl(paged_tc_merge_kernel<D, NT, GR, kState>, dim3(items + whole, NT, Z), dim3(GR * BQ), 0, st, a, grid, items);
}
template <int D, int NT, int GR>
cudaError_t launch_merge(const paged::Args &a, int grid, cudaStream_t st) {
    return a.state.mode != paged::kNone ? launch_merge<D, NT, GR, true>(a, grid, st) : launch_merge<D, NT, GR, false>(a, grid, st);
}
template <int D, int NT>
cudaError_t launch_merge(const paged::Args &a, int grid, bool many, cudaStream_t st) {
    return many ? launch_merge<D, NT, 4>(a, grid, st) : launch_merge<D, NT, 1>(a, grid, st);
}

}  // namespace

attn_status_t launch_paged_tc(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const paged::Args &a,
                              int d, int tiles, int tile_rows, int grid, cudaStream_t st) {
    if (a.ks)
        return d == 64 ? launch<64, true>(mq, mk, mv, a, tiles, tile_rows, grid, st)
                       : launch<128, true>(mq, mk, mv, a, tiles, tile_rows, grid, st);
    return d == 64 ? launch<64, false>(mq, mk, mv, a, tiles, tile_rows, grid, st)
                   : launch<128, false>(mq, mk, mv, a, tiles, tile_rows, grid, st);
}

attn_status_t launch_paged_tc_merge(const paged::Args &a, int d, int tiles, int grid, cudaStream_t st) {
    // Items cut into more than four parts or so (16 tokens of 4 query heads over a key head, d 128, 131072
    // keys in all): 8 items 47 us with one thread a row, 27 with four; 32 items 25.8 and 23.2; 64 items
    // 24.9 and 25.7; the 77 us of a ragged batch of chunks become 82.  With the own keys' states, which one thread a row
    // asks for ahead, from 16 parts on: 64 sequences behind 8192 keys, eight items in five parts each 52 and 56 us.
    const bool many = (double)a.Hkv * ((a.T * a.G + a.R - 1) / a.R + a.B - 1) * (a.state.ml2 ? 16. : 4.) < (double)grid;
    const cudaError_t e = d == 64 ? (tiles == 2 ? launch_merge<64, 2>(a, grid, many, st) : launch_merge<64, 1>(a, grid, many, st))
                                  : (tiles == 2 ? launch_merge<128, 2>(a, grid, many, st) : launch_merge<128, 1>(a, grid, many, st));
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "paged_tc merge launch: %s", cudaGetErrorString(e));
}

}  // namespace attn
