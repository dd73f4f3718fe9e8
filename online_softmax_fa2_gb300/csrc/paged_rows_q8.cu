// paged_rows_q8.cu -- attention over a paged cache in 8 bits for few rows per key/value head: R = 8 or 16 rows a
// block.
//
// As paged_rows.cu, with tiles of 128 keys: the same bytes a tile, and the same shares of the line.
//   x_ij = (q_i . code_j) scale 2^(e_j - 127);   u_i = sum_j p_ij 2^(f_j - 127) code_j
// The products run in fp16 (m16n8k16), where the codes are exact: cvt turns two codes into the two halves of an
// operand register, half an instruction a code.  bf16 would take five (there is no such cvt).  What fp16
// lacks is range, so nothing else of size goes in:
//   a query row is multiplied by a power of two that brings its largest finite element into [2^14, 2^15), and
//   the row's logits by its inverse;
//   a key's scale multiplies its logits, in fp32;
//   a value's scale goes into its weights, which are w_ij = 2^(x_ij log2 e - m_i + f_j - 127 - y_i + 14), with y_i a running
//   maximum of its own of what a row's keys count with, weight times scale.  u is held relative to y and l to the maximum
//   m of the logits; a key that the row does not see, or that weighs nothing in it, moves neither, whatever its value's scale.
//   The weights, at most 2^14, are rounded to fp16: half a step 2^-11 of one of 2^-14 or more, 2^-25 below, so a key loses
//   2^-39 at most of what the row's largest counts with.  (With a unit for all rows of a block, the largest
//   scale met, a value 2^26 above the others took the outputs of rows that gave it no weight to 0.)
// With 16 rows the rows are the products' 16 and the keys or dimensions their 8; with 8 rows or fewer (a decode step of up to 8
// query heads a key head) it is the other way round, S and O transposed: half the products, and half the logits a thread.
// Fragments come by ldmatrix from the codes as they lie, two codes an element, in an order of the
// contraction that the other operand is brought into:
//   K   a register holds four neighbouring dimensions of a key, in the places of 2t, 2t + 1, 2t + 8 and
//       2t + 9 of the product's 16: the queries are stored in that order;
//   V   transposed, a register holds two neighbouring dimensions of two keys: a byte permutation makes the keys
//       of the even dimension and those of the odd one neighbours, for two products of eight dimensions.
//
// The bound is the cache's bytes; measured, 32/8 heads of 128 unless said: 64 ragged sequences to 8192 keys (647 MB) 112 to 114 us,
// 5.7 TB/s (655 MB read, 43% of the issue slots used), with the consumers doing nothing but handing the stages back 113; of that the
// ends of the call are about 12.  With 16 rows a block for the same 4 it took 123, three CTAs of two stages an SM the same,
// tiles of 64 keys 136.  16 heads of 64: 136 us with 8 rows a block (130 with one unit for all rows and no bounds
// of a factor), with 16 some 30 more.  A cache
// whose heads lie apart (places first) gives TMA rows of d bytes instead of whole boxes: 120 to 130 and 217 to 239 us.
#include <cudaTypedefs.h>

#include "paged.h"
#include "paged_merge.cuh"
#include "q8.cuh"
#include "warp_mma.cuh"

namespace attn {

using namespace paged;
using namespace wmma16;

namespace {

constexpr int kConsumers = 128, kThreads = kConsumers + 32;
constexpr int KT = kRowsQ8Keys;  // keys a tile

template <int D, int R>
struct Rows {
    static constexpr int kTile = KT * D;                // codes of K or V; rows of 128 or 64 bytes, swizzled over as many
    static constexpr int kBlocks = rows_blocks(D);
    static constexpr int kStages = (kBlocks == 3 ? 64 : 96) * 1024 / (2 * kTile);
    static constexpr int kQRow = 2 * D + 16, kPRow = 2 * KT + 16;  // padded: ldmatrix without bank conflicts
    // the tiles of all stages first (a swizzled tile begins on 1024 bytes), then their scales
    static constexpr int kScaleOff = kStages * 2 * kTile;
    static constexpr int kQOff = kScaleOff + kStages * 2 * KT;
    static constexpr int kPOff = kQOff + R * kQRow;
    static constexpr int kRedOff = kPOff + R * kPRow;        // [4][R] maxima, [4][R] with scales, beside the first, [4][R] sums
    static constexpr int kUnitOff = kRedOff + 3 * 4 * R * 4; // [R] a row's inverse power of two, times the scale
    static constexpr int kCtrlOff = kUnitOff + R * 4;
};

struct Ctrl {
    uint64_t full[8], empty[8];
    Share share;
    int abort, last;
};

template <int D, int R>
constexpr int smem_bytes() {
    constexpr int n = Rows<D, R>::kCtrlOff + (int)sizeof(Ctrl) + 1024;
    static_assert((n + 1024) * Rows<D, R>::kBlocks <= 228 * 1024, "shared memory of the CTAs an SM holds");
    return n;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

constexpr float kRoom = 14.f;  // log2 of the largest weight as fp16 has it

// Where 16-byte chunk c of row r of a tile lies (TMA's swizzle of 128 or 64 bytes).
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
    return r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}

// d += a * b for one m16n8k16 tile of fp16
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8x8 matrices, each transposed as it is stored; lane i gives the address of row i % 8 (a column of the registers) of
// matrix i / 8.
__device__ __forceinline__ void stsm_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, Rows<D, R>::kBlocks)
    paged_rows_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Args a) {
    using L = Rows<D, R>;
    constexpr bool kTurned = R == 8;  // S and O transposed
    constexpr int NS = L::kStages, DW = D / 4;  // DW: a warp's dimensions of O
    constexpr int NG = DW / 16;                 // in groups of 16
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem + L::kCtrlOff);
    volatile int *abort = &ctrl->abort;
    float *red = reinterpret_cast<float *>(smem + L::kRedOff), *unit = reinterpret_cast<float *>(smem + L::kUnitOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(&ctrl->full[s], 1);
            ptx::mbar_init(&ctrl->empty[s], 4);
        }
        ctrl->abort = 0;
        ptx::fence_mbar_init();
    }
    begin_after_earlier_grids(a, true);
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
        end_after_earlier_grids(a);
        return;
    }

    if (warp == 4) {
        // ------------------------------------------------------------ TMA producer
        const int pb_log2 = min(a.page_log2, 7), boxes = KT >> pb_log2;  // 8 boxes at most
        const int box = lane >> 2, part = lane & 3;                      // parts: K, V, their scales
        const CUtensorMap *tm = (part & 1) ? &tm_v : &tm_k;
        const uint8_t *sc = (part & 1) ? a.vs : a.ks;
        const long long sc_page = (part & 1) ? a.vss[0] : a.kss[0], sc_head = (part & 1) ? a.vss[1] : a.kss[1];
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
                // boxes that hold a key of the sequence
                const int nbox = min(boxes, ((p.seq.n - kv0 - 1) >> pb_log2) + 1);
                if (lane == 0) ptx::mbar_arrive_expect_tx(&ctrl->full[st], (uint32_t)(nbox * 2 * (D + 1)) << pb_log2);
                __syncwarp();
                const int key = kv0 + (box << pb_log2), slot = key & ((1 << a.page_log2) - 1);
                const int page = __shfl_sync(0xffffffffu, pages, min(max((key >> a.page_log2) - held, 0), 31));
                if (box < nbox) {
                    if (part < 2) {
                        uint8_t *dst = smem + st * 2 * L::kTile + part * L::kTile + ((box << pb_log2) * D);
                        ptx::tma_load_4d(dst, tm, &ctrl->full[st], 0, slot, p.hk, page);
                        if (page == a.num_pages && part == 0) atomicOr(a.flags, kFlagBadIndex);
                    } else {
                        // (of a page out of range, whose codes are zeros, another page's scales)
                        const uint8_t *src = sc + (page < a.num_pages ? page : 0) * sc_page + p.hk * sc_head + slot;
                        ptx::bulk_load(smem + L::kScaleOff + st * 2 * KT + (part & 1) * KT + (box << pb_log2), src, 1u << pb_log2,
                                  &ctrl->full[st]);
                    }
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
    uint8_t *sP = smem + L::kPOff, *sQ = smem + L::kQOff;
    float *red_y = red + 4 * R, *sums = red + 8 * R;
    int st = 0, ph = 0;
    // a block's queries, D / 8 neighbouring threads a row, 16 bytes each (rows past the block's end are zero)
    constexpr int QN = R * (D / 8), QC = (QN + kConsumers - 1) / kConsumers;  // (whole warps without a row, with 8 of 64)
    uint4 qv[QC];
    auto bring_q = [&](const Walk &p) {
        const int left = p.seq.nq * a.G - p.k * R;
#pragma unroll
        for (int u = 0; u < QC; ++u) {
            const int i = threadIdx.x + u * kConsumers, r = i / (D / 8), c = i % (D / 8), row = p.k * R + r, tok = div_g(a, row);
            qv[u] = make_uint4(0u, 0u, 0u, 0u);
            if (i < QN && r < left)
                qv[u] = __ldg(reinterpret_cast<const uint4 *>(a.q + (p.seq.q0 + tok) * a.qs0 + (p.hk * a.G + row - tok * a.G) * a.qs1 + c * 8));
        }
    };
    // this lane's two rows
    auto row_of = [&](int e) { return kTurned ? 2 * t + e : 8 * e + g; };
    auto store_q = [&]() {
#pragma unroll
        for (int u = 0; u < QC; ++u) {
            const int i = threadIdx.x + u * kConsumers, r = i / (D / 8), c = i % (D / 8);
            if (i >= QN) break;
            const uint32_t w[4] = {qv[u].x, qv[u].y, qv[u].z, qv[u].w};
            uint32_t top = 0;  // the largest finite magnitude, as bits of a bf16
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
                top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            }
#pragma unroll
            for (int d = D / 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const int ex = max((int)(top >> 7), 27);  // its exponent field, or one whose 2^(141 - ex) is finite
            const float up = __uint_as_float((uint32_t)(127 + 141 - ex) << 23);
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = q8::pack_f16(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
            // dimensions 4s, 4s + 1 of a group of 16 to places 2s, 2s + 1; 4s + 2, 4s + 3 to 2s + 8, 2s + 9
            uint8_t *to = sQ + r * L::kQRow + (c >> 1) * 32 + (c & 1) * 8;
            *reinterpret_cast<uint2 *>(to) = make_uint2(h[0], h[2]);
            *reinterpret_cast<uint2 *>(to + 16) = make_uint2(h[1], h[3]);
            if (c == 0) unit[r] = __uint_as_float((uint32_t)(127 - 141 + ex) << 23) * a.scale_log2;
        }
    };
    bring_q(w);
    bool more = true;
    while (more) {
        const Walk p = w;
        const int rows = min(R, p.seq.nq * a.G - p.k * R), row0 = p.k * R;
        int lim[2];  // keys < lim are visible to this lane's rows
        float m[2], y[2], l[2], o[kTurned ? NG : DW / 8][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row_of(e);
            lim[e] = (a.causal && r < rows) ? min(max(p.seq.n - p.seq.nq + div_g(a, row0 + r) + 1, 0), p.seq.n) : p.seq.n;
            m[e] = y[e] = -INFINITY;
            l[e] = 0.f;
        }
        const int lim0 = a.causal ? min(max(p.seq.n - p.seq.nq + div_g(a, row0) + 1, 0), p.seq.n) : p.seq.n;
#pragma unroll
        for (int nt = 0; nt < (kTurned ? NG : DW / 8); ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
        consumer_sync();  // the last piece is done with the queries and with sums
        store_q();
        consumer_sync();
        more = w.next(a);
        if (more) bring_q(w);
        uint32_t qf[kTurned ? D / 32 : D / 16][4];  // of 16 dimensions, or 32
#pragma unroll
        for (int kk = 0; kk < (kTurned ? D / 32 : D / 16); ++kk)
            ldsm_x4(smem_addr(kTurned ? sQ + mr * L::kQRow + (4 * kk + mi) * 16
                                      : sQ + ((mi & 1) * 8 + mr) * L::kQRow + (2 * kk + (mi >> 1)) * 16), qf[kk]);
        const float un[2] = {unit[row_of(0)], unit[row_of(1)]};

        for (int j = p.j0; p.keys > 0 && j < p.j1; ++j) {
            const int kv0 = j * KT;
            // a wait that gave up is reported; the walk goes on (the four warps keep meeting at the
            // same barriers) and ends, its waits returning at once
            ptx::mbar_wait(&ctrl->full[st], ph, abort, a.flags, kFlagWaitTimeout, kWaitLimitNs);
            __syncwarp();
            uint8_t *sK = smem + st * 2 * L::kTile, *sV = sK + L::kTile;
            const uint8_t *sKs = smem + L::kScaleOff + st * 2 * KT, *sVs = sKs + KT;

            // S of this warp's 32 keys: s[n] of rows 8 e + g and keys 8 n + 2 t + i in 2 e + i, or (turned) of keys
            // 16 n + 8 i + g and rows 2 t + e in 2 i + e
            constexpr int NS_ = kTurned ? 2 : 4;
            float s[NS_][4];
#pragma unroll
            for (int nt = 0; nt < NS_; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t kf[4], lo[4], hi[4];
                ldsm_x4(smem_addr(sK + chunk_at<D>(32 * warp + 8 * mi + mr, kk)), kf);
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) q8::decode4(kf[nt], lo[nt], hi[nt]);
                if constexpr (kTurned) {
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const uint32_t k4[4] = {lo[2 * nt], lo[2 * nt + 1], hi[2 * nt], hi[2 * nt + 1]};
                        mma_f16(s[nt], k4, qf[kk / 2][2 * (kk & 1)], qf[kk / 2][2 * (kk & 1) + 1]);
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) mma_f16(s[nt], qf[kk], lo[nt], hi[nt]);
                }
            }
            // the places of s: key of the tile and element of row e's i-th
            auto key_of = [&](int nt, int i) { return 32 * warp + (kTurned ? 16 * nt + 8 * i + g : 8 * nt + 2 * t + i); };
            auto at_of = [](int e, int i) { return kTurned ? 2 * i + e : 2 * e + i; };
            auto bytes_of = [&](const uint8_t *from, int nt, uint32_t (&b)[2]) {
                if constexpr (kTurned) {
                    b[0] = from[key_of(nt, 0)];
                    b[1] = from[key_of(nt, 1)];
                } else {
                    const uint32_t two = *reinterpret_cast<const uint16_t *>(from + key_of(nt, 0));
                    b[0] = two & 255u;
                    b[1] = two >> 8;
                }
            };
            // scale, mask, row maxima of this warp's keys, of the logits and with the values' scales (255 is a NaN, which
            // becomes the weight, and which a maximum passes over)
            const bool edge = kv0 + KT > lim0;
            float mx[2] = {-INFINITY, -INFINITY}, my[2] = {-INFINITY, -INFINITY}, up[NS_][2];
#pragma unroll
            for (int nt = 0; nt < NS_; ++nt) {
                uint32_t b[2], f[2];
                bytes_of(sKs, nt, b);
                bytes_of(sVs, nt, f);
                const float sc[2] = {q8::pow2(b[0]), q8::pow2(b[1])};
#pragma unroll
                for (int i = 0; i < 2; ++i) up[nt][i] = f[i] == 255u ? NAN : (float)((int)f[i] - 127);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = s[nt][at_of(e, i)] * q8::factor(un[e] * sc[i]);
                        if (edge && kv0 + key_of(nt, i) >= lim[e]) x = -INFINITY;
                        s[nt][at_of(e, i)] = x;
                        mx[e] = fmaxf(mx[e], x);
                    }
            }
            // (differences of logits first: beside a large one an exponent would be lost)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int nt = 0; nt < NS_; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) my[e] = fmaxf(my[e], (s[nt][at_of(e, i)] - mx[e]) + up[nt][i]);
#pragma unroll
                for (int d = kTurned ? 4 : 1; d < (kTurned ? 32 : 4); d <<= 1) {
                    const float ox = __shfl_xor_sync(0xffffffffu, mx[e], d), oy = __shfl_xor_sync(0xffffffffu, my[e], d);
                    const float big = fmaxf(mx[e], ox);
                    my[e] = fmaxf(my[e] + (mx[e] - big), oy + (ox - big));
                    mx[e] = big;
                }
                if ((kTurned ? g : t) == 0) {
                    red[warp * R + row_of(e)] = mx[e];
                    red_y[warp * R + row_of(e)] = my[e];
                }
            }
            // value rows past the sequence may hold anything: zero, so that 0 * v is 0
            const bool ragged = kv0 + KT > p.seq.n;
            if (ragged)
                for (int i = threadIdx.x; i < KT * (D / 16); i += kConsumers)
                    if (kv0 + i / (D / 16) >= p.seq.n) *reinterpret_cast<uint4 *>(sV + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            consumer_sync();
            float al[2], ref[2], ref_y[2];  // al: of u
            bool moved = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row_of(e);
                const float mn = fmaxf(fmaxf(m[e], fmaxf(red[r], red[R + r])), fmaxf(red[2 * R + r], red[3 * R + r]));
                ref[e] = mn == -INFINITY ? 0.f : mn;
                const float old = y[e] + (m[e] - ref[e]);
                float yn = old;
#pragma unroll
                for (int w = 0; w < 4; ++w) yn = fmaxf(yn, red_y[w * R + r] + (red[w * R + r] - ref[e]));
                const float base = yn == -INFINITY ? 0.f : yn;
                al[e] = ptx::ex2(old - base);
                ref_y[e] = base - kRoom;
                l[e] *= ptx::ex2(m[e] - ref[e]);
                moved |= al[e] != 1.f;
                m[e] = mn;
                y[e] = yn;
            }
            uint32_t pk[NS_][2];  // weights: two keys of row e, or (turned) two rows of the i-th key
#pragma unroll
            for (int nt = 0; nt < NS_; ++nt) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = s[nt][at_of(e, i)] - ref[e];
                        l[e] += ptx::ex2(x);
                        w[at_of(e, i)] = x == -INFINITY ? 0.f : ptx::ex2(x + (up[nt][i] - ref_y[e]));  // (a hidden key's scale may be anything)
                    }
                pk[nt][0] = q8::pack_f16(w[0], w[1]);
                pk[nt][1] = q8::pack_f16(w[2], w[3]);
            }
            if constexpr (kTurned) {
                stsm_x4_trans(smem_addr(sP + mr * L::kPRow + (32 * warp + 8 * mi) * 2), pk[0][0], pk[0][1], pk[1][0], pk[1][1]);
            } else {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<uint32_t *>(sP + row_of(e) * L::kPRow + (32 * warp + 8 * nt + 2 * t) * 2) = pk[nt % NS_][e];
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nt = 0; nt < (kTurned ? NG : DW / 8); ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][e] *= al[kTurned ? e & 1 : e >> 1];
            }
            consumer_sync();
            // O of this warp's dimensions: o[2 gi] and o[2 gi + 1] of the even and the odd dimensions of a group, or (turned)
            // o[gi] of dimensions 2 g in 0, 1 and 2 g + 1 in 2, 3
#pragma unroll
            for (int kk = 0; kk < KT / 32; ++kk) {
                uint32_t pf[2][4];
                if constexpr (kTurned) {
                    ldsm_x4(smem_addr(sP + mr * L::kPRow + (4 * kk + mi) * 16), pf[0]);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        ldsm_x4(smem_addr(sP + ((mi & 1) * 8 + mr) * L::kPRow + (4 * kk + 2 * h + (mi >> 1)) * 16), pf[h]);
                }
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    uint32_t vf[4];  // 32 keys of 16 dimensions
                    ldsm_x4_trans(smem_addr(sV + chunk_at<D>(32 * kk + 8 * mi + mr, warp * NG + gi)), vf);
                    uint32_t ev[4], od[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) q8::decode4(__byte_perm(vf[k], 0, 0x3120), ev[k], od[k]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (kTurned) {
                            const uint32_t v4[4] = {ev[2 * h], od[2 * h], ev[2 * h + 1], od[2 * h + 1]};
                            mma_f16(o[gi], v4, pf[0][2 * h], pf[0][2 * h + 1]);
                        } else {
                            mma_f16(o[2 * gi], pf[h], ev[2 * h], ev[2 * h + 1]);
                            mma_f16(o[2 * gi + 1], pf[h], od[2 * h], od[2 * h + 1]);
                        }
                    }
                }
            }
            if (ragged) ptx::fence_proxy_async_smem();  // the zeros above, before the stage's next copy
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->empty[st]);
            if (++st == NS) { st = 0; ph ^= 1; }
        }

        // ------------------------------------------------------------ the piece's rows
        // row sums: over the lanes of a row, then over the four warps
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = l[e];
            if constexpr (kTurned) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
                if (g == 0) sums[warp * R + row_of(e)] = v;
            } else {
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (t == 0) sums[warp * R + row_of(e)] = v;
            }
        }
        consumer_sync();
        wait_for_states(a);
        const bool whole = p.whole();
        const int c0 = whole ? 0 : p.first_share(a);
        const long long slot = whole ? 0 : state_slot(blockIdx.x, c0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row_of(e);
            if (r >= rows) continue;
            // u relative to m, in two steps: the factor itself may be past fp32's range
            const float vu = y[e] == -INFINITY ? 0.f : ptx::ex2(0.5f * (y[e] - kRoom));
            float sum = (sums[r] + sums[R + r]) + (sums[2 * R + r] + sums[3 * R + r]);
            const int tg = div_g(a, row0 + r), tok = p.seq.q0 + tg, h = p.hk * a.G + row0 + r - tg * a.G;
            const StateAt at = state_at(a, D, p.hk, (long long)p.seq.q0 * a.G + row0 + r);
            Ending end{1.f, 0.f, false, false, nullptr, nullptr};
            if (whole) end = ending(a, at, tok, m[e], sum);
            const bool empty = sum == 0.f;  // a NaN is no empty row: it goes on into o and lse
            const float inv = empty ? 0.f : 1.f / sum;
            constexpr int C = kTurned ? 2 : 4;  // neighbouring columns a lane has of a group
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                const int col = warp * DW + 16 * gi + C * (kTurned ? g : t);
                float v[C];
                if constexpr (kTurned) {
                    v[0] = o[gi][e] * vu * vu;
                    v[1] = o[gi][2 + e] * vu * vu;
                } else {
                    v[0] = o[2 * gi][2 * e] * vu * vu;
                    v[1] = o[2 * gi + 1][2 * e] * vu * vu;
                    v[2] = o[2 * gi][2 * e + 1] * vu * vu;
                    v[3] = o[2 * gi + 1][2 * e + 1] * vu * vu;
                }
                if (whole) end_u<C>(a, end, at, col, v, sum);
                if (whole && end.written) continue;
#pragma unroll
                for (int c = 0; c < C; c += 2) {
                    if (!whole) *reinterpret_cast<float2 *>(a.u + (slot * R + r) * D + col + c) = make_float2(v[c], v[c + 1]);
                    else *reinterpret_cast<uint32_t *>(a.o + tok * a.os0 + h * a.os1 + col + c) = empty ? 0u : pack_bf16(v[c] * inv, v[c + 1] * inv);
                }
            }
            if (warp == 0 && (kTurned ? g : t) == 0) {
                if (!whole)
                    *reinterpret_cast<float2 *>(a.ml + (slot * R + r) * 2) = make_float2(empty ? -INFINITY : m[e], sum);
                else if (end.written) write_ml(end, at, m[e], sum);
                else if (a.lse) a.lse[(long long)tok * a.Hq + h] = empty ? -INFINITY : (m[e] + log2f(sum)) * kLn2;
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
                        end_row<D, true>(a, p.seq.q0, p.hk, row0 + r, v, mx, sum);
                    });
                });
    }
    end_after_earlier_grids(a);
}

template <int D, int R>
attn_status_t launch(const CUtensorMap &mk, const CUtensorMap &mv, const Args &a, int grid, cudaStream_t st) {
    auto kern = paged_rows_q8_kernel<D, R>;
    const int smem = smem_bytes<D, R>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, mk, mv, a);
    return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "paged_rows_q8 launch: %s", cudaGetErrorString(e));
}

}  // namespace

attn_status_t launch_paged_rows_q8(const CUtensorMap &mk, const CUtensorMap &mv, const Args &a, int d, int grid, cudaStream_t st) {
    if (a.R == 8) return d == 64 ? launch<64, 8>(mk, mv, a, grid, st) : launch<128, 8>(mk, mv, a, grid, st);
    return d == 64 ? launch<64, 16>(mk, mv, a, grid, st) : launch<128, 16>(mk, mv, a, grid, st);
}

}  // namespace attn
