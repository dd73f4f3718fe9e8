/*
 * attn.h -- C ABI of the GB300 (sm_103a) exact-attention library.
 *
 * The library computes exact scaled-dot-product attention,
 *
 *     x_ij = scale * <q_i, k_j> + b_ij        for j in J_i (the visible keys of row i)
 *     o_i  = sum_j exp(x_ij - m_i) v_j / l_i,  m_i = max_j x_ij,  l_i = sum_j exp(x_ij - m_i)
 *     lse_i = m_i + ln l_i
 *
 * tile by tile with the mergeable per-row state (m, l, u): a running maximum, the
 * exponential sum measured against it and the unnormalised value sum, both rescaled by
 * exp(m_old - m_new) when the maximum grows, and divided once per row at the end.
 *
 * Sources (page title, then section / step / figure):
 *   "How Does FlashAttention Preserve Global Softmax Across Tiles?"
 *       section 1  the operator, visible set J_i, fixed bias b_ij, d_k != d_v allowed,
 *                  scale independent of tile size;
 *       section 3  the state (m, l, u) and the merge of disjoint key subsets;
 *       section 5  tile loop, rows keep their own state, divide once at the end;
 *       section 6  global positions; causal masks align the two sequences' ends
 *                  ("bottom-right"); an entirely empty row returns zero; dropout is
 *                  disabled there, and a training backward must reproduce the forward's
 *                  mask and scaling (the keep mask of attn_fwd is therefore an input);
 *       section 7  the saved log-sum-exp L_i, and the backward that rebuilds the
 *                  probabilities from it (attn_bwd);
 *       section 8  decode (one query row, or a few, against a long key/value cache) split
 *                  over the keys, the partial states merged.
 *   "Flash attention and efficient attention: Visual walkthrough", Steps 4-5 (the three
 *       running numbers; re-basing a sum to a new maximum by one multiply).
 *   "Reducing Memory Traffic with Output Accumulation in FlashAttention", Figures 1-3
 *       (value-weighted sum first, both accumulators rescaled, one division).
 *
 * Conventions shared by every entry point:
 *   - Every tensor pointer is a DEVICE pointer owned by the caller; it must stay valid until
 *     the work queued on `stream` has finished.  The library keeps no pointer after a call
 *     returns and allocates no device memory.
 *   - All work is queued asynchronously on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream) on the current CUDA device.
 *   - Arguments are checked on the host before anything is queued; a bad argument returns a
 *     non-zero attn_status_t and queues nothing.  attn_last_error() then describes it.
 *     No entry point throws or aborts.
 *   - Visible set J_i of query row i of batch entry b, with n_b = kv_lens[b] clamped to
 *     [0, Nk] (Nk when kv_lens is NULL):  j < n_b, and, when causal,
 *     j <= i + n_b - Nq (bottom-right alignment), and b_ij != -inf.
 *     Nothing stored at a masked position is ever used: NaN there cannot reach an output.
 *   - An empty row (J_i empty) gives o_i = +0.0 and lse_i = -inf, exactly.
 *   - Accumulation is fp32.  bf16 outputs are rounded to nearest even once, at the end.
 */
#ifndef ONLINE_SOFTMAX_FA2_GB300_ATTN_H
#define ONLINE_SOFTMAX_FA2_GB300_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *attn_stream_t;

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,    /* null pointer, negative size, bad stride, bad scale */
    ATTN_ERR_UNSUPPORTED = 2,    /* valid, but this build has no kernel for it (e.g. head dim) */
    ATTN_ERR_MISALIGNED = 3,     /* a pointer or stride breaks the 16-byte rule of the path */
    ATTN_ERR_CUDA = 4,           /* a CUDA runtime call or a launch failed */
    ATTN_ERR_DEVICE_TIMEOUT = 5, /* a kernel gave up a bounded wait (see attn_device_error_flags) */
    ATTN_ERR_WORKSPACE = 6       /* the workspace is missing, misaligned or too small */
} attn_status_t;

typedef enum {
    ATTN_DTYPE_F32 = 0,   /* q, k, v, o are float32 */
    ATTN_DTYPE_BF16 = 1   /* q, k, v, o are bfloat16 */
} attn_dtype_t;

/*
 * Arguments of one attention forward.
 *
 *   q  [B, Nq, H, dk]   element (b, i, h, c) at q + b*q_stride[0] + i*q_stride[1]
 *                       + h*q_stride[2] + c          (strides in ELEMENTS; c contiguous)
 *   k  [B, Nk, H, dk]   same with k_stride;  v [B, Nk, H, dv] with v_stride
 *   o  [B, Nq, H, dv]   written, with o_stride
 *   lse [B, H, Nq]      fp32, contiguous, written; may be NULL
 *   bias                NULL, or fp32 b_ij of (b, h, i, j) at
 *                       bias + b*bias_stride[0] + h*bias_stride[1] + i*bias_stride[2] + j;
 *                       a stride of 0 broadcasts; -inf masks the position; bias is added
 *                       after scaling and is not scaled
 *   kv_lens             NULL, or device int32 [B]: keys j >= kv_lens[b] are padding
 *   causal              0: no causal mask; 1: bottom-right causal mask
 *   scale               multiplies <q_i, k_j>; the standard operator uses 1/sqrt(dk)
 *   block_k             float32 path only: key tile size 16, 32 or 64 (0 picks 64);
 *                       must be 0 for bfloat16
 *
 * bfloat16 path (tcgen05 tensor cores): dk in {64, 128, 192}, dv in {64, 128},
 *   scale > 0; q, k, v, o base pointers 16-byte aligned and their b, n, h strides non-zero
 *   multiples of 8 elements (16 bytes); bias 4-byte aligned (rows that are 16-byte aligned
 *   are read with 16-byte loads).
 * float32 path (exact fp32 SIMT): 1 <= dk, dv <= 256; any finite scale.
 *
 *   dropout_mask        NULL: no dropout.  Otherwise the keep mask of a training forward:
 *                       key j of row i of (b, h) is kept iff bit (j % 8) of byte
 *                       dropout_mask[b*s0 + h*s1 + i*s2 + j/8] is set (s = dropout_mask_stride,
 *                       in bytes; each row holds at least 16*ceil(Nk/128) bytes).  Kept
 *                       weights p_ij are scaled by 1 / (1 - dropout_p), dropped ones count 0
 *                       in o; the row sum and lse are those of the undropped softmax.  The
 *                       mask is an input so that a backward can reproduce it ("How Does
 *                       FlashAttention Preserve Global Softmax Across Tiles?", section 6,
 *                       disables dropout and asks exactly that of a training backward).
 *                       bfloat16: dk <= 128 only, the mask 16-byte aligned with strides that
 *                       are multiples of 16 bytes.  Not taken by attn_decode_splitkv, nor by
 *                       attn_bwd together with a bias (ATTN_ERR_UNSUPPORTED).
 *   dropout_p           in [0, 1) with a mask or with dropout_rng = 1; must be 0 otherwise.
 *   dropout_rng         0: the keep decisions come from dropout_mask (or there is no dropout).
 *                       1: they are drawn in-kernel, and no mask is read or stored anywhere:
 *                       the drop probability is quantised to p8 / 256, p8 = round(256 p) (at
 *                       most 255), and key j of row i of (b, h) is kept iff byte j % 16 of the
 *                       counter-based generator Philox4x32-10 (Salmon, Moraes, Dror, Shaw,
 *                       "Parallel Random Numbers: As Easy as 1, 2, 3", SC'11) at counter
 *                       (i, j / 16, b*H + h, dropout_offset mod 2^32) under key (dropout_seed
 *                       mod 2^32, dropout_seed div 2^32) -- its four output words in order,
 *                       each little-endian -- is at least p8; kept weights are scaled by
 *                       256 / (256 - p8).  dropout_mask must then be NULL.  attn_bwd given the
 *                       forward's (dropout_p, dropout_rng, dropout_seed, dropout_offset) draws
 *                       the same decisions.  Where a mask is not taken (see dropout_mask), the
 *                       in-kernel draw is not either.
 *   dropout_seed, dropout_offset  the generator's key and the fourth counter word (a fresh
 *                       offset per training step gives fresh decisions).
 */
typedef struct {
    int32_t dtype;           /* attn_dtype_t */
    int32_t causal;          /* 0 or 1 */
    int64_t B, H, Nq, Nk, dk, dv;
    const void *q;
    const void *k;
    const void *v;
    void *o;
    int64_t q_stride[3];     /* b, n, h */
    int64_t k_stride[3];
    int64_t v_stride[3];
    int64_t o_stride[3];
    float *lse;
    const float *bias;
    int64_t bias_stride[3];  /* b, h, i (j stride is 1) */
    const int32_t *kv_lens;
    float scale;
    int32_t block_k;
    const uint8_t *dropout_mask;
    int64_t dropout_mask_stride[3];  /* b, h, i (bytes) */
    float dropout_p;
    int32_t dropout_rng;             /* 0: keep bits from dropout_mask; 1: drawn in-kernel */
    uint64_t dropout_seed;
    uint64_t dropout_offset;
} attn_fwd_params_t;

/*
 * attn_fwd -- O and lse of exact attention for every (b, h, i).
 * ("How Does FlashAttention Preserve Global Softmax Across Tiles?", sections 1, 5, 6, 7.)
 * Queues one kernel.  Nq == 0 or B*H == 0 queues nothing and returns ATTN_OK.  Nk == 0 is
 * legal (every row is empty; k and v may then be NULL).
 */
attn_status_t attn_fwd(const attn_fwd_params_t *params, attn_stream_t stream);

/*
 * Size in bytes of the workspace attn_decode_splitkv needs for Nq query rows per sequence:
 * the per-split partial states, float32 [B, H, Nq, num_splits, 2 + dv] laid out
 * (m, l, u[0..dv)), where m is the maximum logit of the split (natural-log units),
 * l = sum exp(x_j - m) and u = sum exp(x_j - m) v_j over the keys of the split visible to
 * that row; an empty split is (-inf, 0, 0...).  Returns 0 for a negative or zero size.
 */
size_t attn_decode_workspace_bytes_rows(int64_t B, int64_t H, int64_t Nq, int64_t dv,
                                        int32_t num_splits);

/* attn_decode_workspace_bytes_rows with Nq = 1: float32 [B, H, num_splits, 2 + dv]. */
size_t attn_decode_workspace_bytes(int64_t B, int64_t H, int64_t dv, int32_t num_splits);

/*
 * attn_decode_splitkv -- a few query rows per (b, h) (1 <= params->Nq <= 8: one decode
 * step, or several tokens of one sequence at once) against a long key/value cache, the keys
 * of each sequence split into num_splits contiguous near-equal ranges of [0, n_b) (split s
 * covers [floor(s*n_b/S), floor((s+1)*n_b/S))).  Each key row of the cache is read once for
 * all Nq query rows.  params->causal applies the bottom-right mask of the conventions above
 * (row i sees keys j <= i + n_b - Nq), so the last row sees the whole sequence; a row that
 * sees no key is empty.
 * ("How Does FlashAttention Preserve Global Softmax Across Tiles?", section 8, decode;
 *  section 6, bottom-right alignment; section 3, merge.)
 * Queues two kernels on `stream`: the split kernel writes every partial state into
 * `workspace` (layout above), then the merge kernel writes o and lse exactly as attn_fwd
 * would.  The workspace is caller-owned device memory of at least
 * attn_decode_workspace_bytes_rows(B, H, Nq, dv, num_splits) bytes, 16-byte aligned; after
 * the call it holds the partial states.  Supported: bfloat16, dk == dv in {64, 128},
 * 1 <= num_splits <= 256.  Nq outside [1, 8] returns ATTN_ERR_INVALID_ARG.  The cache may
 * use any strides that keep each key row contiguous and 16-byte aligned (e.g. a [B, H, L, d]
 * cache passed with k_stride = {H*L*d, d, L*d}).
 */
attn_status_t attn_decode_splitkv(const attn_fwd_params_t *params, int32_t num_splits,
                                  void *workspace, size_t workspace_bytes,
                                  attn_stream_t stream);

/*
 * Size in bytes of the workspace attn_decode_splitkv_fused needs: the partial states exactly as
 * for attn_decode_splitkv (attn_decode_workspace_bytes_rows, rounded up to a multiple of 16),
 * then one 64-bit arrival counter per (b, h), [B, H].  Returns 0 for a negative or zero size.
 */
size_t attn_decode_fused_workspace_bytes(int64_t B, int64_t H, int64_t Nq, int64_t dv,
                                         int32_t num_splits);

/*
 * attn_decode_splitkv_fused -- attn_decode_splitkv in one kernel: the split kernel also does
 * the merge.  ("How Does FlashAttention Preserve Global Softmax Across Tiles?", section 8:
 * the extra partial round trip and merge launch of split-KV decode; section 3, the merge.)
 * Every split CTA writes its partial states, makes them visible device-wide and counts itself
 * on its (b, h)'s counter; the CTA that counts last merges the S states of every query row of
 * that (b, h) (the arithmetic of attn_merge_states) and writes o and lse.  No CTA waits for
 * another.  A counter holds (the call's own tag, count), with a fresh tag for every call, so
 * a count left by an earlier call, or any other contents, reads as zero.
 *   - Same arguments, checks and supported shapes as attn_decode_splitkv; same results, bit
 *     for bit (the same split kernel and the same merge arithmetic).
 *   - workspace: caller-owned device memory of at least attn_decode_fused_workspace_bytes(...)
 *     bytes, 16-byte aligned; its contents on entry do not matter.  After the call the
 *     partial-state part holds the partial states.
 *   - Calls that share a workspace and overlap on the GPU race on it: order them on a stream.
 *   - Bit 0 of the device error word is set if a count had to give up (4096 retries of its
 *     compare-and-swap; with S counting CTAs it retries at most S - 1 times).
 * Queues one kernel.
 */
attn_status_t attn_decode_splitkv_fused(const attn_fwd_params_t *params, int32_t num_splits,
                                        void *workspace, size_t workspace_bytes,
                                        attn_stream_t stream);

/*
 * attn_decode_splitkv_noalloc -- attn_decode_splitkv for callers that cannot allocate device
 * memory when they decode (a framework whose allocator owns the device memory, a plugin
 * handed only its inputs and outputs, a latency-bound loop where cudaMalloc would
 * synchronise the device).  The paper has no counterpart: the pages describe no such variant.
 *   - Same arguments, checks, kernels and results as attn_decode_splitkv, without the
 *     workspace: the partial states go to a device array built into the library, 32 MiB
 *     (B * H * Nq * num_splits * (2 + dv) * 4 bytes must fit; larger problems return
 *     ATTN_ERR_WORKSPACE and queue nothing).  Every device that loads the library holds that
 *     array until the process exits.  No device memory is allocated by any call.
 *   - Arguments are checked exactly as attn_decode_splitkv checks them, and before the size
 *     limit: a bad argument returns its own status, not ATTN_ERR_WORKSPACE.
 *   - The first call from a CUDA context looks up the array's device address (with the
 *     device current) and caches it per device, together with that context's unique id; a
 *     call from a new context (e.g. after cudaDeviceReset) looks it up again.
 *   - All calls share the one array.  Every call writes each partial state it reads, so
 *     nothing needs clearing, but calls whose work overlaps on the GPU (different streams,
 *     several host threads) race on it: order them on one stream.
 */
attn_status_t attn_decode_splitkv_noalloc(const attn_fwd_params_t *params, int32_t num_splits,
                                          attn_stream_t stream);

/*
 * attn_merge_states -- merge S partial states per (b, h) and finalise.
 * ("How Does FlashAttention Preserve Global Softmax Across Tiles?", section 3: put both
 *  maxima into the common maximum, scale l and u of each part by exp(m_s - m), add;
 *  empty parts are skipped.  "Flash attention and efficient attention: Visual
 *  walkthrough", Step 5.)
 *   partials  device fp32 [B, H, S, 2 + dv] as (m, l, u); a part with l == 0 is empty
 *   o         written: row (b, h) at o + b*o_stride[0] + h*o_stride[2] (o_stride[1] unused),
 *             element type o_dtype; u/l, or +0.0 when every part is empty
 *   lse       device fp32 [B, H] written: m + ln l, or -inf when every part is empty; may be
 *             NULL
 * Queues one kernel.
 */
attn_status_t attn_merge_states(const float *partials, int64_t B, int64_t H, int32_t num_splits,
                                int64_t dv, int32_t o_dtype, void *o, const int64_t o_stride[3],
                                float *lse, attn_stream_t stream);

/*
 * attn_fwd_partial -- the state (m, l, u) of every query row over one shard of the keys, for
 * attention split over the key axis (sequence parallelism across devices, or any split that
 * the caller merges later).  ("How Does FlashAttention Preserve Global Softmax Across
 * Tiles?", section 3: the state of a key subset and the merge of disjoint subsets; section 4:
 * every key in exactly one part; section 6: global positions.)
 *   params        as for attn_fwd, with k, v (and bias, if any) holding only the shard's keys:
 *                 params->Nk keys, local key j being global key key_offset + j.  params->o and
 *                 params->lse are not used (may be NULL).  kv_lens and the causal mask are in
 *                 global positions: key J of sequence b is visible to row i iff
 *                 J < min(kv_lens[b], Nk_total) and, when causal, J <= i + n_b - Nq.
 *   key_offset, Nk_total  the shard [key_offset, key_offset + Nk) of a sequence of Nk_total
 *                 keys (0 <= key_offset, key_offset + Nk <= Nk_total <= 2^31 - 1).
 *   partials      device fp32 [B, H, Nq, 2 + dv], 16-byte aligned, written: (m, l, u) with
 *                 l = sum exp(x_j - m) and u = sum exp(x_j - m) v_j over the shard's visible
 *                 keys, measured against the row's reference m (natural-log units): the largest
 *                 visible logit, or a value at most 8 ln 2 below it (the kernel moves its
 *                 reference only when a larger logit exceeds it by more than that; the merge
 *                 is the same for any common reference); (-inf, 0, 0...) for a row that sees
 *                 none of them.
 * Supported: bfloat16, dk == dv in {64, 128}, with or without a bias; no dropout.  Merging the
 * states of shards that cover each sequence's keys exactly once (attn_merge_states_rows)
 * gives attn_fwd's o and lse.  Queues one kernel.
 */
attn_status_t attn_fwd_partial(const attn_fwd_params_t *params, int64_t key_offset, int64_t Nk_total,
                               float *partials, attn_stream_t stream);

/*
 * attn_merge_states_rows -- attn_merge_states for Nq rows per (b, h) and any layout of the
 * parts: state s of row r = (b*H + h)*Nq + i is the 2 + dv floats (m, l, u) at
 * partials + r*row_stride + s*split_stride (strides in floats; 0, 0 mean the decode layout
 * [B, H, Nq, num_splits, 2 + dv]; states gathered from R devices as [R, B, H, Nq, 2 + dv]
 * take row_stride = 2 + dv, split_stride = B*H*Nq*(2 + dv)).  Writes o row (b, i, h) at
 * o + b*o_stride[0] + i*o_stride[1] + h*o_stride[2] (element type o_dtype) and lse [B, H, Nq]
 * (may be NULL); a row whose parts are all empty gets +0.0 and -inf.  1 <= num_splits <= 4096,
 * 1 <= dv <= 1024.  Queues one kernel.
 */
attn_status_t attn_merge_states_rows(const float *partials, int64_t B, int64_t H, int64_t Nq,
                                     int32_t num_splits, int64_t dv, int64_t row_stride,
                                     int64_t split_stride, int32_t o_dtype, void *o,
                                     const int64_t o_stride[3], float *lse, attn_stream_t stream);

/*
 * Arguments of one attention backward: the forward's arguments and outputs (fwd.o and
 * fwd.lse as the forward wrote them; fwd.lse is required), the upstream gradient of O, and
 * the three gradients to write.
 *   dout [B, Nq, H, dv]   bf16, with dout_stride (b, n, h; elements)
 *   dq   [B, Nq, H, dk]   bf16, written;  dk [B, Nk, H, dk], dv [B, Nk, H, dv] likewise
 */
typedef struct {
    attn_fwd_params_t fwd;
    const void *dout;
    int64_t dout_stride[3];
    void *dq;
    int64_t dq_stride[3];
    void *dk;
    int64_t dk_stride[3];
    void *dv;
    int64_t dv_stride[3];
} attn_bwd_params_t;

/*
 * Size in bytes of the workspace attn_bwd needs: an fp32 dQ accumulator [B, Nq, H, dk], the
 * fp32 row terms c_i [B, H, Nq], and lse_i * log2 e [B, H, Nq rounded up to a multiple of 128]
 * in fp32, each part starting on a 16-byte boundary.  Returns 0 for a negative or zero size.
 */
size_t attn_bwd_workspace_bytes(int64_t B, int64_t H, int64_t Nq, int64_t dk);

/*
 * attn_bwd -- gradients dQ, dK, dV of a loss through O = attention(Q, K, V) given the
 * upstream gradient G = dL/dO.
 * ("How Does FlashAttention Preserve Global Softmax Across Tiles?", section 7: the forward
 *  saves each row's log-sum-exp L_i and its output; the backward rebuilds the probabilities
 *  p_ij = exp(x_ij - L_i) tile by tile from Q, K, the fixed mask and bias, takes
 *  c_i = g_i . o_i, dS_ij = p_ij (g_i . v_j - c_i), and accumulates dV_j += p_ij g_i,
 *  dK_j += scale dS_ij q_i, dQ_i += scale dS_ij k_j.)
 * The mask, bias, kv_lens, causal and dropout settings must be the forward's: with a
 * dropout_mask in fwd (the forward's keep bits and dropout_p) the gradient reaching the
 * weights carries the mask and the 1 / (1 - p) scale, dV is formed from the kept, scaled
 * weights, and c_i = g_i . o_i already holds the dropout through o (without a bias only;
 * with one ATTN_ERR_UNSUPPORTED).  The bias is fixed: no gradient is formed for it.  An empty row (lse = -inf) passes no gradient, and a key that no
 * row sees gets dK = dV = 0.
 * Queues three kernels on `stream`: the row terms, the products (on the 5th-generation
 * tensor cores), and the conversion of dQ to bf16.  Supported: bfloat16, dk == dv in {64, 128}; every tensor
 * 16-byte aligned with strides that are multiples of 8 elements.  The workspace is
 * caller-owned device memory of at least attn_bwd_workspace_bytes(B, H, Nq, dk) bytes,
 * 16-byte aligned; its contents on entry do not matter.  dQ is accumulated with atomic
 * additions, so its rounding can differ from run to run in the last bits.
 */
attn_status_t attn_bwd(const attn_bwd_params_t *params, void *workspace, size_t workspace_bytes,
                       attn_stream_t stream);

/*
 * Head norms and position rotation.
 *
 * For every query and key head row x of d elements at position pos:
 *     t_c = w_c x_c / sqrt(mean_c x_c^2 + eps)              (t = x when w is NULL)
 *     (y_a, y_b) = (t_a cos - t_b sin, t_a sin + t_b cos)   for the pairs of the first rot
 *     dimensions, y_c = t_c for the others
 * with cos and sin of pair c at cos_sin[pos*cos_sin_stride + c] and [... + rot/2 + c].
 *
 *   dtype         element type of every tensor but cos_sin, positions and the weight gradients
 *   interleaved   0: pair c is (c, c + rot/2);  1: pair c is (2c, 2c + 1)
 *   q, k          [B, N, Hq, d] and [B, N, Hkv, d], strides in elements (b, n, h), d contiguous
 *   q_out, k_out  written, same shapes; each may be its input itself (same strides), and must
 *                 not overlap it otherwise
 *   wq, wk        [d], or NULL: that tensor is not normalised
 *   cos_sin       fp32 [cos_sin_rows, rot], row stride cos_sin_stride floats, or NULL: nothing
 *                 is rotated (rot is then ignored)
 *   positions     int32, (b, n) at positions + b*positions_stride[0] + n*positions_stride[1], or
 *                 NULL: token n of every sequence is at position n.  A position outside
 *                 [0, cos_sin_rows) sets bit 2 of the device error word and is clamped.
 * Supported: d a multiple of 16 up to 256; rot a multiple of 16 up to d; Hq, Hkv >= 1; tensors
 * 16-byte aligned with strides that are multiples of 16 bytes.
 */
typedef struct {
    int32_t dtype;
    int32_t interleaved;
    int64_t B, N, Hq, Hkv, d, rot;
    const void *q;
    const void *k;
    void *q_out;
    void *k_out;
    int64_t q_stride[3];      /* b, n, h */
    int64_t k_stride[3];
    int64_t q_out_stride[3];
    int64_t k_out_stride[3];
    const void *wq;
    const void *wk;
    const float *cos_sin;
    int64_t cos_sin_rows;
    int64_t cos_sin_stride;
    const int32_t *positions;
    int64_t positions_stride[2];  /* b, n */
    float eps;                    /* > 0 */
} attn_qk_norm_rope_params_t;

/*
 * attn_qk_norm_rope -- both tensors in one pass, before attn_fwd.  The arithmetic is fp32, each
 * output rounded once; a normalised row whose sum of squares passes fp32's range (elements of 1e18 and
 * more) comes out as zeros.  An element that is not rotated reaches no other but through the norm.
 * Queues one kernel.
 */
attn_status_t attn_qk_norm_rope(const attn_qk_norm_rope_params_t *params, attn_stream_t stream);

/*
 * Arguments of its backward: the forward's arguments (fwd.q_out and fwd.k_out are not used; q and
 * k are the forward's inputs), the gradients of its outputs, and the gradients to write.
 *   dq_out, dk_out  [B, N, Hq, d], [B, N, Hkv, d]
 *   dq, dk          written; each may be dq_out / dk_out itself, and must not overlap an input otherwise
 *   dwq, dwk        fp32 [d], written; NULL exactly where the weight is NULL
 */
typedef struct {
    attn_qk_norm_rope_params_t fwd;
    const void *dq_out;
    const void *dk_out;
    void *dq;
    void *dk;
    int64_t dq_out_stride[3];
    int64_t dk_out_stride[3];
    int64_t dq_stride[3];
    int64_t dk_stride[3];
    float *dwq;
    float *dwk;
} attn_qk_norm_rope_bwd_params_t;

/* Bytes of workspace attn_qk_norm_rope_bwd needs on the current device (partial weight gradients; 0
 * for a negative or zero size). */
size_t attn_qk_norm_rope_bwd_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t Hkv, int64_t d);

/*
 * attn_qk_norm_rope_bwd -- with n_c = x_c r (r = 1 / sqrt(mean x^2 + eps)), dt = R^T dy:
 *     dw_c = sum over rows dt_c n_c,   dx_c = r (w_c dt_c - n_c mean_j w_j dt_j n_j).
 * The weight gradients are summed in fp32 in a fixed order (the same bits from run to run).  The
 * workspace is caller-owned device memory, 16-byte aligned, of any contents on entry; it may be NULL when both
 * weights are.  Queues one kernel, and one more for the weight gradients.
 */
attn_status_t attn_qk_norm_rope_bwd(const attn_qk_norm_rope_bwd_params_t *params, void *workspace,
                                    size_t workspace_bytes, attn_stream_t stream);

/*
 * A paged key/value cache and a ragged batch of new tokens over it.
 *
 *   k_pages, v_pages  [num_pages, page_size, Hkv, d]: strides in elements (page, slot, head), d
 *                     contiguous (a [num_pages, Hkv, page_size, d] cache is passed by its strides)
 *   block_table       int32 [B, table_width], row stride table_stride: the key at position j of
 *                     sequence b is slot j % page_size of page block_table[b][j / page_size].
 *                     Entries past a sequence's last page are never read.  A page outside
 *                     [0, num_pages) sets bit 2 of the device error word; nothing is read or
 *                     written there.
 *   kv_lens           int32 [B]: keys of each sequence, the new tokens included; clamped to
 *                     [0, table_width * page_size] (bit 1 of the device error word)
 *   cu_q              int32 [B + 1], not decreasing: tokens cu_q[b] .. cu_q[b + 1] - 1 of the T
 *                     packed tokens are sequence b's newest (token i of its nq lies at position
 *                     kv_lens[b] - nq + i).  NULL: every sequence has T / B of them.  Tokens
 *                     before cu_q[0] and from cu_q[B] on belong to no sequence: their outputs are
 *                     left as they were.  Entries outside [0, T] or decreasing set bit 2 and are
 *                     clamped (to [0, T], and to the entry before); a token that two sequences claim
 *                     then, or none, has no outputs that can be relied on.
 * B <= 65535, T < 2^31, table_width * page_size < 2^31.
 */
typedef struct {
    int32_t dtype;       /* attn_dtype_t */
    int32_t page_size;
    int64_t B, T, Hkv, d;
    void *k_pages;
    void *v_pages;
    int64_t k_stride[3]; /* page, slot, head */
    int64_t v_stride[3];
    int64_t num_pages;
    const int32_t *block_table;
    int64_t table_width;
    int64_t table_stride;
    const int32_t *kv_lens;
    const int32_t *cu_q;
} attn_paged_cache_t;

/*
 * Arguments of attn_paged_append: packed tokens q [T, Hq, d], k and v [T, Hkv, d] (strides token,
 * head), and the head norms and rotation of attn_qk_norm_rope (weights, cos_sin, rot, eps,
 * interleaved as there).
 *   q_out      [T, Hq, d], written; may be q itself, and must not overlap an input otherwise
 *   positions  int32 [T], the rotation's positions, or NULL: each token's place in its sequence
 *              (0 for a token with no place, see below)
 */
typedef struct {
    attn_paged_cache_t cache;
    int64_t Hq, rot;
    const void *q;
    const void *k;
    const void *v;
    void *q_out;
    int64_t q_stride[2];      /* token, head */
    int64_t k_stride[2];
    int64_t v_stride[2];
    int64_t q_out_stride[2];
    const void *wq;
    const void *wk;
    const float *cos_sin;
    int64_t cos_sin_rows;
    int64_t cos_sin_stride;
    const int32_t *positions;
    float eps;
    int32_t interleaved;
} attn_paged_append_params_t;

/*
 * attn_paged_append -- norms and rotates q and k, writes the keys and the values (as they are) to
 * their slots of the cache, and q to q_out, in one pass.  A token whose place kv_lens[b] - nq + i
 * is negative (a place of the batch without a sequence) writes no key or value.  No two tokens of a
 * call may have the same slot (sequences may share pages that no token of the call is written to).
 * Supported: as attn_qk_norm_rope; any page_size >= 1; B >= 1 when T > 0.  (More than attn_paged_fwd
 * reads: that takes bfloat16, d of 64 or 128 and pages of a power of two of 16 keys or more.)  Queues
 * one kernel.
 */
attn_status_t attn_paged_append(const attn_paged_append_params_t *params, attn_stream_t stream);

/*
 * Arguments of attn_paged_fwd: packed queries q [T, Hq, d] (strides token, head) of the batch that
 * cache describes; Hq is a multiple of Hkv, and query head h reads key/value head h / (Hq / Hkv).
 *   causal   0: a token sees all kv_lens[b] keys; 1: token i of nq sees keys j <= i + kv_lens[b] - nq
 *   max_q    the largest number of new tokens of any sequence, or 0 when it is not known: it
 *            chooses the kernel, one for the whole call, and the results hold for any value.  With 0
 *            the mean chooses, which suits even batches alone: a chunk of 2048 tokens over 18432 keys
 *            beside 255 single tokens (32/8 heads of 128) takes 0.58 ms with max_q = 2048, 1.05 with 0.
 *   o        [T, Hq, d], written;  lse fp32 [T, Hq] contiguous, written; may be NULL.  Neither may
 *            overlap an input.
 */
typedef struct {
    attn_paged_cache_t cache;
    int32_t causal;
    float scale;
    int64_t Hq, max_q;
    const void *q;
    void *o;
    int64_t q_stride[2];
    int64_t o_stride[2];
    float *lse;
} attn_paged_fwd_params_t;

/* Bytes of workspace attn_paged_fwd needs for these arguments on the current device (pointers are
 * not looked at); 0 for invalid ones. */
size_t attn_paged_fwd_workspace_bytes(const attn_paged_fwd_params_t *params);

/*
 * attn_paged_fwd -- attention of the new tokens, one or many per sequence in one call, over the
 * paged cache.  ("How Does FlashAttention Preserve Global Softmax Across Tiles?", sections 3, 6
 * and 8.)  A key or value row is read once for all query heads that share it.  The work is cut into
 * equal shares of key tiles over the GPU; a row whose keys fall into several shares is merged from
 * their states (m, l, u), in a fixed order: the same bits from run to run (another max_q may take
 * another kernel, and give other last bits).  The weights are rounded to bf16 before the value
 * product, as in attn_fwd; sums and states are fp32.
 * A row that sees no key, or only keys of logit -inf, has o = +0.0 and lse = -inf.  A NaN in a query or in
 * a visible key, and a logit of +inf, make o and lse of the rows that see them NaN, and of no others.
 * Values at positions >= kv_lens[b] are never used, whatever lies there.  A visible value that is
 * infinite or NaN reaches every query row of its tile, as 0 * inf does in a product.
 * workspace: caller-owned device memory, 16-byte aligned, of any contents on entry; calls that
 * overlap on the GPU need one each.  It may be NULL where attn_paged_fwd_workspace_bytes is 0.
 * Supported: bfloat16, d in {64, 128}, page_size a power of two >= 16, 1 <= Hq / Hkv <= 64,
 * T * Hq / Hkv <= 2^30, table_width * page_size <= 2^31 - 256, scale > 0; tensors 16-byte aligned,
 * strides non-zero multiples of 8 elements.  Queues one kernel or two.
 */
attn_status_t attn_paged_fwd(const attn_paged_fwd_params_t *params, void *workspace, size_t workspace_bytes,
                             attn_stream_t stream);

/*
 * A paged cache in 8 bits.
 *
 * A row (the d elements of one key head, key or value, of one token) is held as d codes of e4m3 (one
 * byte each: sign, 4 bits of exponent, 3 of mantissa, largest 448, no infinity) and one scale byte e: its
 * elements are code * 2^(e - 127).  A power of two costs a floating format nothing (an element is
 * off by half a step, 2^-4 of itself, wherever the row's largest lies, down to 2^-13 of that) and is exact in every product.
 *
 *   k_pages, v_pages  of attn_paged_cache_t: e4m3 codes, strides in elements, which are bytes
 *   k, v              scale bytes [num_pages, Hkv, page_size], strides in bytes (page, head), the
 *                     slots of a page contiguous; all 256 values are valid, 255 makes the row NaN
 */
typedef struct {
    void *k;
    void *v;
    int64_t k_stride[2];
    int64_t v_stride[2];
} attn_paged_scales_t;

/* Arguments of attn_paged_append_q8: those of attn_paged_append (cache.dtype is the type of q, k, v,
 * q_out and the weights), and the scales. */
typedef struct {
    attn_paged_append_params_t append;
    attn_paged_scales_t scales;
} attn_paged_append_q8_params_t;

/*
 * attn_paged_append_q8 -- attn_paged_append into a cache in 8 bits: the keys are quantised as they come
 * from the norm and the rotation, in fp32, the values as they are.  e - 127 is the smallest exponent >=
 * -127 that brings the row's largest finite magnitude within 448 * 2^(e - 127) (0 for a row of zeros), and
 * the elements are rounded to the nearest code, ties to even.  A NaN or an infinity is held as NaN.  Two tokens with one
 * place leave it with codes and a scale of either.
 * Supported: as attn_paged_append; the pages' strides are multiples of 16 bytes, as their bases.  Queues one kernel.
 */
attn_status_t attn_paged_append_q8(const attn_paged_append_q8_params_t *params, attn_stream_t stream);

/*
 * Arguments of attn_paged_read_q8: cache as for the append, with cu_q and T naming the rows: rows
 * cu_q[b] .. cu_q[b + 1] - 1 of the T are sequence b's last (row i of its n is the key at position
 * kv_lens[b] - n + i); cache.dtype is the type of k and v.
 *   k, v   [T, Hkv, d], written (strides token, head); either may be NULL
 */
typedef struct {
    attn_paged_cache_t cache;
    attn_paged_scales_t scales;
    void *k;
    void *v;
    int64_t k_stride[2];
    int64_t v_stride[2];
} attn_paged_read_q8_params_t;

/*
 * attn_paged_read_q8 -- rows of a cache in 8 bits as the numbers that they stand for, rounded once (in
 * bfloat16 exact but for values under 2^-126 or over its range).  Rows of no sequence, and those whose
 * position would be negative, are left as they were; a row on a page out of range too (bit 2).
 * Supported: as attn_paged_append_q8.  Queues one kernel.
 */
attn_status_t attn_paged_read_q8(const attn_paged_read_q8_params_t *params, attn_stream_t stream);

/* Arguments of attn_paged_fwd_q8: those of attn_paged_fwd (cache.dtype is the type of q and o), and the scales. */
typedef struct {
    attn_paged_fwd_params_t fwd;
    attn_paged_scales_t scales;
} attn_paged_fwd_q8_params_t;

/* Bytes of workspace attn_paged_fwd_q8 needs, as attn_paged_fwd_workspace_bytes. */
size_t attn_paged_fwd_q8_workspace_bytes(const attn_paged_fwd_q8_params_t *params);

/*
 * attn_paged_fwd_q8 -- attn_paged_fwd over a cache in 8 bits.  The products take the codes in fp16, where
 * they are exact; a query row goes in as its elements times a power of two that brings the largest finite one
 * near 2^14 (exact down to 2^-31 of it), the weights are rounded to fp16 before the value product.  Of a weight under 2^-21
 * of the row's largest bits under 2^-32 of that are lost, or, where a weight goes in times its value's scale (with up
 * to 16 rows a key head, and where the scales of 128 neighbouring keys lie 2^16 or more apart), bits under 2^-32 of
 * the largest such product that the row has.  What a row does not see, or gives no weight, takes nothing from it,
 * whatever its scale.  (With more than 16 rows, 128 keys whose scales lie so far apart take five times as long as others,
 * and rows of scale byte 0, under 2^-118, count as zeros beside ones of byte 25 and up among them.)
 * Everything else as attn_paged_fwd; a row that holds a NaN makes the rows that see it NaN.
 * Supported: as attn_paged_fwd; the bases and strides of pages and scales are multiples of 16 bytes.  A cache whose
 * heads lie apart ([num_pages, Hkv, page_size, d] in memory, passed by its strides) is read faster: 136 us for
 * 217 to 239 at 16 heads of 64, 113 for 120 to 130 at 8 of 128 (64 ragged sequences to 8192 keys).
 */
attn_status_t attn_paged_fwd_q8(const attn_paged_fwd_q8_params_t *params, void *workspace, size_t workspace_bytes,
                                attn_stream_t stream);

/*
 * Arguments of attn_paged_prefix_fwd: attention of a batch whose sequences share prefixes.  Besides its
 * sequence's own keys (fwd, as for attn_paged_fwd: kv_lens, the block table and the causal rule do not count the
 * prefix), a token sees every key of its prefix:
 *   prefix_table   int32 [P, prefix_width], row stride prefix_stride: pages of the same cache, as a block table
 *   prefix_lens    int32 [P], clamped to [0, prefix_width * page_size] (bit 1 of the device error word)
 *   cu_prefix      int32 [P + 1], not decreasing: tokens cu_prefix[p] .. cu_prefix[p + 1] - 1 of the T see
 *                  prefix p; tokens before cu_prefix[0] and from cu_prefix[P] on have none.  NULL: every
 *                  prefix has T / P of them.  Bad entries as for cu_q.
 *   scales         of a cache in 8 bits (codes and rules of attn_paged_fwd_q8), or k and v NULL: cache.dtype
 */
typedef struct {
    attn_paged_fwd_params_t fwd;
    attn_paged_scales_t scales;
    int64_t P, prefix_width, prefix_stride;
    const int32_t *prefix_table;
    const int32_t *prefix_lens;
    const int32_t *cu_prefix;
} attn_paged_prefix_params_t;

/* Bytes of workspace attn_paged_prefix_fwd needs for these arguments on the current device: the states of T * Hq rows,
 * (d + 2) * 4 bytes each, once or twice, and what the attentions need.  (Of the pointers only scales.k is looked at: NULL or
 * not.)  0 for invalid ones. */
size_t attn_paged_prefix_fwd_workspace_bytes(const attn_paged_prefix_params_t *params);

/*
 * attn_paged_prefix_fwd -- the prefix's keys and values are read once for all tokens that see it (rows of the
 * same product); the rows' states (m, l, u) over it and over the own keys meet in the workspace, in fp32, and are
 * merged.  ("How Does FlashAttention Preserve Global Softmax Across Tiles?", section 3.)  The result
 * is that of attn_paged_fwd over the prefix's keys followed by the own ones, lse included, with its rules for empty rows,
 * NaN and tokens of no sequence; no token has to belong to a prefix.  (A row that the causal rule lets see no own key, as it lies
 * before them all, sees its whole prefix.)  How the GPU is shared out between the prefixes and the own keys goes by the
 * tables' widths: tables no wider than their longest entry (a view will do) are fastest.  (One token of 64 sequences to
 * 1024 keys behind 8192, 32/8 heads of 128, 56 us: with a block table of 131072 keys 88, with such a prefix table 122, with
 * both 57; over 8 bits 54, 92, 67, 67.)
 * Supported: as attn_paged_fwd, or attn_paged_fwd_q8; 1 <= P <= 65535.  Queues two or three kernels.
 */
attn_status_t attn_paged_prefix_fwd(const attn_paged_prefix_params_t *params, void *workspace, size_t workspace_bytes,
                                    attn_stream_t stream);

/* Message describing the last non-OK status returned on the calling thread ("" if none). */
const char *attn_last_error(void);

/*
 * Device error word of the current device (synchronous: waits for the device to finish its
 * queued work first).  Bit 0: a kernel gave up a bounded wait on an mbarrier and returned
 * early (its outputs are then incomplete).  Bit 1: a kv_lens value was outside its range and
 * was clamped.  Bit 2: a page, a position or a cu_q entry was out of range (nothing out of bounds
 * was read or written).  clear != 0 resets the word to 0 after reading.  Returns ATTN_OK or
 * ATTN_ERR_CUDA.
 */
attn_status_t attn_device_error_flags(uint32_t *out, int32_t clear);

/* Library version, major*10000 + minor*100 + patch. */
int32_t attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ONLINE_SOFTMAX_FA2_GB300_ATTN_H */
