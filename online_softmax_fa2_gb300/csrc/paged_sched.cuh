// paged_sched.cuh -- how the attention over a paged cache cuts its work, shared by its kernels.
//
// The rows of a sequence that share key/value head hk are numbered token * G + g (G = Hq / Hkv
// query heads a key head) and taken R at a time: block k holds rows [k R, (k + 1) R).  An item
// (b, hk, k) walks the 2^kt-key tiles up to the last key that its last row sees.  All items' tiles
// in order (sequence, head, block), `cost` more a block for its beginning and end, form one line,
// cut at equal distances into shares, one a CTA, whatever the lengths: a batch of one long and many short sequences, or a
// single one, loads every SM alike.  A boundary that falls less than min_cut tiles inside an item
// goes to that end of it (a cut costs about as much as so many tiles).  An item inside one share
// is finished there.  An item cut by a boundary leaves one state (m, l, u) per share in the
// workspace; one of the shares that come last merges them (paged_merge.cuh).
//
// A share holds at most one cut item that began before it (slot 2 c) and one that goes on past its
// end (slot 2 c + 1).
#pragma once

#include <cuda_bf16.h>

#include "attn_more.h"
#include "fwd_bf16_common.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr long long kLongestLine = 0x7fff0000;  // tiles of a line, so that a distance along it is an int
constexpr size_t kCutBytes = 32;  // a share's record of the item that it cuts (paged_tc_sm103.cu)
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // every mbarrier wait gives up after 1 s

// The states of all packed tokens' rows over keys that another call holds (a shared prefix); with the G query heads of a
// key head in a row, token t's are rows t G .. t G + G - 1 of N = T G: ml [Hkv][N], u [Hkv][D / 4][N][4], so that
// neighbouring rows (lanes) are neighbours in memory.  (As [row][D] the tiles' states took 42 us more for 14000 rows of
// four key heads.)  Written in place of the outputs by the call over those keys, merged into the outputs by the other.
//
// Where the own keys' attention runs beside the prefixes' (paged_fwd.cu), neither waits for the other: its states go to ml2
// and u2 (kLeft; rows of tokens without a prefix are finished), and the prefixes' merge, which comes last, merges both
// (kMerged, the own states as ml and u): of the items that it merges, and of the rows that the prefixes' attention has
// finished, whose states are its ml2 and u2 (other rows hold kCutRow as l there).
//
// Where tiles take both, one after the other, no merge lies between: of a row that the prefixes' attention has cut, ml holds
// kCutRow as l and, as m, which parts it is in (cut_row of paged_state.cuh); the own keys' attention joins them.
struct State {
    int mode;      // kNone, kWritten, kMerged, kLeft
    int P;         // (merged, left) tokens cu[0] .. cu[P] - 1 have one; cu null: all
    int B;         // (merged) rows of tokens outside only[0] .. only[B] - 1 are left as they were; only null: none
    const int *cu, *only;
    float2 *ml, *ml2;
    float *u, *u2;
    bool marks;    // (written) cut rows are marked
    unsigned long long *begun, tag;  // the call's tag, once what the call reads is there (begin_after_earlier_grids)
    const float *part_ml, *part_u;  // (merged) the parts of cut rows, of `shares` shares and `tiles` row tiles an item
    int shares, tiles;
};
constexpr int kNone = 0, kWritten = 1, kMerged = 2, kLeft = 3;
constexpr float kCutRow = -1.f;

struct Args {
    int B, T, Hq, Hkv, G, causal, R, kt;  // R rows a block, 2^kt keys a tile
    int page_log2, width, num_pages, min_share, min_cut, cost;
    float scale_log2;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    long long qs0, qs1, os0, os1, bt_s;
    const int *bt, *lens, *cu;
    uint32_t g_m, r_m;  // division by G and by R as a multiply-high and shifts (bf16fwd::fast_div_params)
    int g_s, r_s;
    unsigned long long *marks;  // what is written (paged_merge.cuh), or the cuts (paged_tc_sm103.cu)
    unsigned long long tag;
    float *ml, *u;  // states: (m, l) [slot][R][2], u [slot][R][D]
    uint32_t *flags;
    // a cache in 8 bits: its scale bytes and their strides (page, head)
    const uint8_t *ks, *vs;
    long long kss[2], vss[2];
    State state;
};

__device__ __forceinline__ int div_g(const Args &a, int x) { return (int)bf16fwd::div_fast((uint32_t)x, a.g_m, a.g_s); }

struct Seq {
    int q0, nq, n;  // first packed token, new tokens, keys
};

__device__ __forceinline__ Seq seq_info(const Args &a, int b, bool report) {
    Seq s;
    if (a.cu) {
        const int r0 = __ldg(a.cu + b), r1 = __ldg(a.cu + b + 1);
        const int c0 = min(max(r0, 0), a.T), c1 = min(max(r1, c0), a.T);
        if (report && (c0 != r0 || c1 != r1)) atomicOr(a.flags, kFlagBadIndex);
        s.q0 = c0;
        s.nq = c1 - c0;
    } else {
        s.nq = a.T / a.B;
        s.q0 = b * s.nq;
    }
    const int raw = __ldg(a.lens + b), room = a.width << a.page_log2;
    s.n = min(max(raw, 0), room);
    if (report && s.n != raw) atomicOr(a.flags, kFlagKvLenClamped);
    return s;
}

__device__ __forceinline__ int num_blocks(const Args &a, const Seq &s) { return (int)bf16fwd::div_fast((uint32_t)(s.nq * a.G + a.R - 1), a.r_m, a.r_s); }

// Keys that the last row of block k sees, and the tiles that hold them; a block that sees none
// counts as one tile (its rows are written all the same).
__device__ __forceinline__ int block_keys(const Args &a, const Seq &s, int k) {
    if (!a.causal) return s.n;
    const int last = min((k + 1) * a.R, s.nq * a.G) - 1;
    return min(max(s.n - s.nq + div_g(a, last) + 1, 0), s.n);
}
__device__ __forceinline__ int block_tiles(const Args &a, const Seq &s, int k) {
    return max(1, (block_keys(a, s, k) + (1 << a.kt) - 1) >> a.kt);
}
// What the block takes of the line.
__device__ __forceinline__ int block_len(const Args &a, const Seq &s, int k) { return a.cost + block_tiles(a, s, k); }

// The line of all blocks of a lane's sequence (one head); the whole warp helps with long ones.
__device__ __forceinline__ int seq_len_of(const Args &a, const Seq &s, int nb) {
    const int lane = threadIdx.x & 31;
    int w = 0;
    if (nb <= 4)
        for (int k = 0; k < nb; ++k) w += block_len(a, s, k);
    for (unsigned big = __ballot_sync(0xffffffffu, nb > 4); big; big &= big - 1) {
        const int src = __ffs(big) - 1;
        Seq o;
        o.q0 = 0;
        o.nq = __shfl_sync(0xffffffffu, s.nq, src);
        o.n = __shfl_sync(0xffffffffu, s.n, src);
        const int onb = __shfl_sync(0xffffffffu, nb, src);
        int t = 0;
        for (int k = lane; k < onb; k += 32) t += block_len(a, o, k);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
        if (lane == src) w = t;
    }
    return w;
}

struct Share {
    int per, t0, t1;  // the line between two boundaries, and this CTA's [t0, t1); an int: kLongestLine
    int b, hk, k, j;  // where t0 lies (j = the item's tiles: at its end)
    Seq seq;
};

// The sum over the warp of v >= 0.
__device__ __forceinline__ long long wide_sum(int v) {
    const unsigned u = (unsigned)v;
    return ((long long)__reduce_add_sync(0xffffffffu, u >> 16) << 16) + __reduce_add_sync(0xffffffffu, u & 0xffffu);
}

// The line of one head of every 32 sequences, into sums[0 .. (B - 1) / 32] of shared memory (at most
// 8 KB); all warps of the CTA, which meet afterwards.  (One warp walking over 1024 sequences, once
// for the total and once for each boundary, took 52 us at the start of a call.)
__device__ __forceinline__ void line_sums(const Args &a, int *sums) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int g = threadIdx.x >> 5; g * 32 < a.B; g += blockDim.x >> 5) {
        Seq s{0, 0, 0};
        if (g * 32 + lane < a.B) s = seq_info(a, g * 32 + lane, blockIdx.x == 0);
        const long long w = wide_sum(seq_len_of(a, s, num_blocks(a, s)));
        if (lane == 0) sums[g] = (int)min(w, 0x7fffffffll);
    }
}

// The warp's running sum of v.
__device__ __forceinline__ int warp_scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// The share of CTA c of C; sums: line_sums, for more than 32 sequences.  One warp; every lane gets the
// result.  It runs once, cold, before anything else can: short code counts for more than fast code.
__device__ __forceinline__ Share find_share(const Args &a, int c, int C, const int *sums) {
    const int lane = threadIdx.x & 31, groups = (a.B + 31) / 32;
    Share r;
    r.b = r.hk = r.k = r.j = 0;
    r.seq = Seq{0, 0, 0};
    Seq s{0, 0, 0};
    int w = 0, nb = 0;
    long long line = 0;
    if (groups == 1) {
        if (lane < a.B) s = seq_info(a, lane, c == 0);
        nb = num_blocks(a, s);
        w = seq_len_of(a, s, nb);
        line = wide_sum(w);
    } else {
#pragma unroll 1
        for (int g = lane; g < groups + lane; g += 32) line += wide_sum(g < groups ? sums[g] : 0);
    }
    line *= a.Hkv;
    r.per = 1;
    r.t0 = r.t1 = 0;
    if (line > kLongestLine) {  // entries of cu_q that go back and forth: more rows than the batch has tokens
        if (c == 0 && lane == 0) atomicOr(a.flags, kFlagBadIndex);
        return r;
    }
    const int total = (int)line;
    r.per = max((int)((unsigned)(total + C - 1) / (unsigned)C), a.min_share);
    // the boundaries c + 1, then c: the item that each falls into, and which side of it it goes to
#pragma unroll 1
    for (int e = 1; e >= 0; --e) {
        const int at = (int)min((long long)r.per * (c + e), (long long)total);
        if (at >= total) {
            if (e == 0) r.t0 = total;
            else r.t1 = total;
            continue;
        }
        int left = at, b0 = 0;
        if (groups > 1) {
#pragma unroll 1
            for (int g0 = 0; g0 < groups; g0 += 32) {
                const int v = g0 + lane < groups ? sums[g0 + lane] * a.Hkv : 0, incl = warp_scan(v);
                const unsigned past = __ballot_sync(0xffffffffu, incl > left);
                if (past) {
                    const int l = __ffs(past) - 1;
                    b0 = 32 * (g0 + l);
                    left -= __shfl_sync(0xffffffffu, incl - v, l);
                    break;
                }
                left -= __shfl_sync(0xffffffffu, incl, 31);
            }
            s = Seq{0, 0, 0};
            if (b0 + lane < a.B) s = seq_info(a, b0 + lane, false);
            nb = num_blocks(a, s);
            w = seq_len_of(a, s, nb);
        }
        {
            const int incl = warp_scan(w * a.Hkv);
            const unsigned past = __ballot_sync(0xffffffffu, incl > left);
            const int src = __ffs(past) - 1, ws = __shfl_sync(0xffffffffu, w, src);
            r.b = b0 + src;
            r.seq.q0 = __shfl_sync(0xffffffffu, s.q0, src);
            r.seq.nq = __shfl_sync(0xffffffffu, s.nq, src);
            r.seq.n = __shfl_sync(0xffffffffu, s.n, src);
            left -= __shfl_sync(0xffffffffu, incl, src) - ws * a.Hkv;
            r.hk = min((int)((unsigned)left / (unsigned)ws), a.Hkv - 1);
            left -= r.hk * ws;
        }
        const int nbs = num_blocks(a, r.seq);
        r.k = 0;
#pragma unroll 1
        for (int k0 = 0; nbs > 1; k0 += 32) {
            const int k = k0 + lane, t = k < nbs ? block_len(a, r.seq, k) : 0, in = warp_scan(t);
            const unsigned hit = __ballot_sync(0xffffffffu, in > left);
            if (hit || k0 + 32 >= nbs) {
                const int l = hit ? __ffs(hit) - 1 : 0;
                r.k = k0 + l;
                left -= __shfl_sync(0xffffffffu, in, l) - __shfl_sync(0xffffffffu, t, l);
                break;
            }
            left -= __shfl_sync(0xffffffffu, in, 31);
        }
        const int tiles = block_tiles(a, r.seq, r.k), j = left - a.cost;
        r.j = j < a.min_cut ? 0 : tiles - j < a.min_cut ? tiles : j;
        // to the item's start, to its end, or between two tiles
        const int to = at - left + (r.j == 0 ? 0 : a.cost + r.j);
        if (e == 0) r.t0 = to;
        else r.t1 = to;
    }
    return r;
}

// A walk over the pieces of a share; every role of the CTA makes the same walk.
struct Walk {
    int per, t, t1;  // the line between two boundaries; where the item begins; where the share ends
    Seq seq;
    int b, hk, k, nb;
    int j0, j1, tiles, keys;  // the piece: tiles [j0, j1) of the block's `tiles`, which hold `keys` keys

    __device__ __forceinline__ void piece(const Args &a, int j) {
        keys = block_keys(a, seq, k);
        tiles = max(1, (keys + (1 << a.kt) - 1) >> a.kt);
        j0 = j;
        j1 = min(tiles, t1 - t - a.cost);
    }
    // false when the share is empty
    __device__ __forceinline__ bool begin(const Args &a, const Share &sh) {
        if (sh.t0 >= sh.t1) return false;
        per = sh.per;
        b = sh.b;
        hk = sh.hk;
        k = sh.k;
        seq = sh.seq;
        nb = num_blocks(a, seq);
        t = sh.t0 - (sh.j == 0 ? 0 : a.cost + sh.j);
        t1 = sh.t1;
        piece(a, sh.j);
        return j0 < tiles || next(a);
    }
    __device__ __forceinline__ bool next(const Args &a) {
        t += a.cost + tiles;
        if (t >= t1) return false;
        if (++k == nb) {
            k = 0;
            if (++hk == a.Hkv) {
                hk = 0;
                do {
                    if (++b >= a.B) return false;
                    seq = seq_info(a, b, false);
                    nb = num_blocks(a, seq);
                } while (nb == 0);
            }
        }
        piece(a, 0);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == tiles; }
    // the share that holds the first part of the item, and the parts that its first n tiles fall
    // into: the boundaries c per that lie min_cut tiles or more inside the item
    __device__ __forceinline__ int first_share(const Args &a) const {
        return (int)(((unsigned)t + (unsigned)(a.cost + a.min_cut + per - 1)) / (unsigned)per) - 1;  // (past 2^31 on the longest lines)
    }
    __device__ __forceinline__ int parts(const Args &a, int c0, int n) const {
        const int last = min(tiles - a.min_cut, n - 1);  // no boundary behind this tile counts
        return last < 0 ? 1 : max((int)((unsigned)(t + a.cost + last) / (unsigned)per) - c0, 0) + 1;
    }
};

__device__ __forceinline__ int state_slot(int share, int first) { return 2 * share + (share == first ? 1 : 0); }

}  // namespace paged
}  // namespace attn
