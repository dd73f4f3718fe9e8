// paged_sched.cuh -- how the attention over a paged cache cuts its work, shared by its kernels.
//
// The rows of a sequence that share key/value head hk are numbered token * G + g (G = Hq / Hkv
// query heads a key head) and taken R at a time: block k holds rows [k R, (k + 1) R).  An item
// (b, hk, k) walks the 2^kt-key tiles up to the last key that its last row sees.  All items' tiles
// in order (sequence, head, block) form one line of `total` tiles, cut into equal shares, one a
// CTA, whatever the lengths: a batch of one long and many short sequences, or a single one,
// loads every SM alike.  An item inside one share is finished there.  An item cut by a boundary
// leaves one state (m, l, u) per share in the workspace; the share that comes last, told by a
// counter, merges them in share order (so the bits do not depend on who came last).
//
// A share holds at most one cut item that began before it (slot 2 c) and one that goes on past its
// end (slot 2 c + 1; the counter of c counts that item's states).  A counter word holds
// (tag of the call, count); under another tag, or zero, it reads as zero, and whoever merges sets
// it to zero: the workspace may hold anything on entry, and a captured call, whose tag is
// the same at every replay, finds zero.
#pragma once

#include <cuda_bf16.h>

#include "attn_internal.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // every mbarrier wait gives up after 1 s

struct Args {
    int B, T, Hq, Hkv, G, causal, R, kt;  // R rows a block, 2^kt keys a tile
    int page_log2, width, num_pages, min_share;
    float scale_log2;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    long long qs0, qs1, os0, os1, bt_s;
    const int *bt, *lens, *cu;
    unsigned long long *counters;
    unsigned long long tag;
    float *ml, *u;  // states: (m, l) [slot][R][2], u [slot][R][D]
    uint32_t *flags;
};

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

__device__ __forceinline__ int num_blocks(const Args &a, const Seq &s) { return (s.nq * a.G + a.R - 1) / a.R; }

// Keys that the last row of block k sees, and the tiles that hold them; a block that sees none
// counts as one tile (its rows are written all the same).
__device__ __forceinline__ int block_keys(const Args &a, const Seq &s, int k) {
    if (!a.causal) return s.n;
    const int last = min((k + 1) * a.R, s.nq * a.G) - 1;
    return min(max(s.n - s.nq + last / a.G + 1, 0), s.n);
}
__device__ __forceinline__ int block_tiles(const Args &a, const Seq &s, int k) {
    return max(1, (block_keys(a, s, k) + (1 << a.kt) - 1) >> a.kt);
}

// Tiles of all blocks of lane's sequence (one head); the whole warp helps with long ones.
__device__ __forceinline__ int seq_tiles(const Args &a, const Seq &s, int nb) {
    const int lane = threadIdx.x & 31;
    int w = 0;
    if (nb <= 4)
        for (int k = 0; k < nb; ++k) w += block_tiles(a, s, k);
    for (unsigned big = __ballot_sync(0xffffffffu, nb > 4); big; big &= big - 1) {
        const int src = __ffs(big) - 1;
        Seq o;
        o.q0 = 0;
        o.nq = __shfl_sync(0xffffffffu, s.nq, src);
        o.n = __shfl_sync(0xffffffffu, s.n, src);
        const int onb = __shfl_sync(0xffffffffu, nb, src);
        int t = 0;
        for (int k = lane; k < onb; k += 32) t += block_tiles(a, o, k);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
        if (lane == src) w = t;
    }
    return w;
}

struct Share {
    long long per, t0, t1;  // tiles a share, and this CTA's [t0, t1)
    int b, hk, k, j;        // where t0 lies
};

// The share of CTA c of C.  One warp; every lane gets the result.
__device__ __forceinline__ Share find_share(const Args &a, int c, int C) {
    const int lane = threadIdx.x & 31;
    long long total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        Seq s{0, 0, 0};
        if (b < a.B) s = seq_info(a, b, c == 0);
        int w = seq_tiles(a, s, num_blocks(a, s));
        long long v = w;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        total += v;
    }
    total *= a.Hkv;
    Share r;
    r.per = max((total + C - 1) / C, (long long)a.min_share);
    r.t0 = min(r.per * c, total);
    r.t1 = min(r.t0 + r.per, total);
    r.b = r.hk = r.k = r.j = 0;
    if (r.t0 >= r.t1) return r;
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        Seq s{0, 0, 0};
        if (b < a.B) s = seq_info(a, b, false);
        const int nb = num_blocks(a, s), w = seq_tiles(a, s, nb);
        long long incl = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, (before + incl) * a.Hkv > r.t0);
        if (!past) {
            before += __shfl_sync(0xffffffffu, incl, 31);
            continue;
        }
        const int src = __ffs(past) - 1;
        Seq o;
        o.q0 = 0;
        o.nq = __shfl_sync(0xffffffffu, s.nq, src);
        o.n = __shfl_sync(0xffffffffu, s.n, src);
        const int ow = __shfl_sync(0xffffffffu, w, src), onb = __shfl_sync(0xffffffffu, nb, src);
        long long rest = r.t0 - (before + __shfl_sync(0xffffffffu, incl, src) - ow) * a.Hkv;
        r.b = b0 + src;
        r.hk = (int)(rest / ow);
        int left = (int)(rest - (long long)r.hk * ow);
        for (int k0 = 0; k0 < onb; k0 += 32) {
            const int k = k0 + lane, t = k < onb ? block_tiles(a, o, k) : 0;
            int in = t;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, in, d);
                if (lane >= d) in += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, in > left);
            if (hit) {
                const int l = __ffs(hit) - 1;
                r.k = k0 + l;
                r.j = left - (__shfl_sync(0xffffffffu, in, l) - __shfl_sync(0xffffffffu, t, l));
                break;
            }
            left -= __shfl_sync(0xffffffffu, in, 31);
        }
        break;
    }
    return r;
}

// A walk over the pieces of a share; every role of the CTA makes the same walk.
struct Walk {
    Share s;
    long long t;  // the line's tile at which the current piece begins
    Seq seq;
    int b, hk, k, nb;
    int j0, j1, tiles, keys;  // the piece: tiles [j0, j1) of the block's `tiles`, which hold `keys` keys

    __device__ __forceinline__ void piece(const Args &a, int j) {
        keys = block_keys(a, seq, k);
        tiles = max(1, (keys + (1 << a.kt) - 1) >> a.kt);
        j0 = j;
        j1 = (int)min((long long)tiles, j + (s.t1 - t));
    }
    // false when the share is empty
    __device__ __forceinline__ bool begin(const Args &a, const Share &sh) {
        s = sh;
        t = s.t0;
        if (t >= s.t1) return false;
        b = s.b;
        hk = s.hk;
        k = s.k;
        seq = seq_info(a, b, false);
        nb = num_blocks(a, seq);
        piece(a, s.j);
        return true;
    }
    __device__ __forceinline__ bool next(const Args &a) {
        t += j1 - j0;
        if (t >= s.t1) return false;
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
    // the shares that hold the item, and the slot of this one's state
    __device__ __forceinline__ int first_share() const { return (int)((t - j0) / s.per); }
    __device__ __forceinline__ int last_share() const { return (int)((t - j0 + tiles - 1) / s.per); }
};

__device__ __forceinline__ int state_slot(int share, int first) { return 2 * share + (share == first ? 1 : 0); }

// Counts this share's state of an item of n states whose counter is *cnt; true for the one that
// completes them, which then sees every state written before.  One thread, after a barrier behind
// the state's writes.  Retries only when another share counted in between (n - 1 times at most).
__device__ __forceinline__ bool count_state(const Args &a, unsigned long long *cnt, int n) {
    __threadfence();
    unsigned long long seen = *reinterpret_cast<volatile unsigned long long *>(cnt), mine = 0;
    for (int tries = 0;; ++tries) {
        mine = ((seen >> 16) == a.tag ? (seen & 0xffffull) : 0ull) + 1ull;
        // the last one leaves zero for the next call (which may be this one, replayed)
        const unsigned long long put = mine == (unsigned long long)n ? 0ull : (a.tag << 16) | mine;
        const unsigned long long prev = atomicCAS(cnt, seen, put);
        if (prev == seen) break;
        seen = prev;
        if (tries >= 65536) {
            atomicOr(a.flags, kFlagWaitTimeout);
            return false;
        }
    }
    if (mine != (unsigned long long)n) return false;
    __threadfence();
    return true;
}

}  // namespace paged
}  // namespace attn
