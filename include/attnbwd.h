/*
 * attnbwd.h -- C ABI of the GB300 (sm_103a) attention-backward library.
 *
 * Stateless, asynchronous calls on the caller's CUDA stream (passed as
 * void*; NULL is the legacy default stream):
 *
 *   sdpa_fwd_stats          O and the fp32 log-sum-exp stats of scaled dot
 *                           product attention (training-mode forward).
 *   sdpa_bwd                dQ, dK, dV of the same attention, FlashAttention-2
 *                           form: P is recomputed from the saved stats.
 *   nsa_selected_attn_bwd   dQ, dK, dV of NSA selected attention, where every
 *                           query token attends to selectedBlockCount blocks of
 *                           selectedBlockSize keys chosen by int32 topkIndices.
 *   sdpa_relbias_fwd_stats, the dense forward and backward with a learned relative
 *   sdpa_relbias_bwd        position bias by buckets added to the scores, and the
 *                           bias table's gradient.
 *   sdpa_relbias_decode     the same attention for one new token per sequence over
 *                           a key / value cache.
 *   paged_cache_write,      keys and values of new tokens into a paged cache, as they
 *   paged_cache_read        are or as e4m3 numbers with a scale a row, and back.
 *   sdpa_paged_fwd          attention of every sequence's new tokens (one, a few, or
 *                           a long chunk) over what it has in such a cache.
 *   qk_norm_rope_fwd, _bwd  RMS norm of every query / key head with the rotary
 *                           position embedding in the same pass, and its gradient:
 *                           what makes Q and K for the calls above and takes their
 *                           dQ and dK.
 *
 * Definitions.  With s_ij = scale * q_i . k_j over the visible keys,
 *   LSE_i = log sum_j exp(s_ij),  P_ij = exp(s_ij - LSE_i),  O_i = sum_j P_ij v_j,
 *   D_i = rowsum(dO_i * O_i),  dP = dO V^T,  dS = P * (dP - D),
 *   dV = P^T dO,  dQ = scale dS K,  dK = scale dS^T Q.
 * Pages cited below by title and section:
 *   [cuDNN]  cuDNN-frontend sample "51_scaled_dot_product_attention_backward"
 *   [Ascend] Ascend CANN page "aclnnNsaSelectedAttentionGrad"
 *   [PR]     PyTorch PR #94729 (matmul -> scale -> softmax -> matmul pattern)
 * Each call below names the passage that defines it.
 *
 * Conventions shared by every call.
 *  - Tensors are caller-owned device memory.  The library allocates nothing,
 *    keeps no state between calls, and fully overwrites its outputs.
 *  - The workspace is caller-owned device memory of at least the size the
 *    matching *_workspace_size call returns, 256-byte aligned.  Its contents
 *    need not be initialised.  Two calls in flight at once must not share it.
 *  - Every argument check runs on the host before anything is launched; a
 *    call that returns an error has launched nothing.  Errors the device
 *    finds (an index out of range, a duplicate selected block, a bounded wait
 *    that ran out) never trap: they set bits in a status word inside the
 *    workspace that attn_query_status reads back.
 *  - 16-bit tensors (fp16 or bf16, one type per call) must start on a 16-byte
 *    boundary and have element strides that are multiples of 8 (16 bytes);
 *    the innermost (head-dim) stride is 1.  Otherwise ATTN_ERR_ALIGN.
 *  - Query head hq uses key/value head hq / (h / h_kv).
 *  - A query row that sees no key (possible only when a bottom-right causal
 *    mask meets s_q > s_kv) has O = 0, LSE = +inf and zero gradients.
 */
#ifndef ATTNBWD_H
#define ATTNBWD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes.  [Ascend] "Return Value" table: a call returns a code; the
 * page's parameter-check failures map to NULLPTR / INVALID here, and its
 * run-time failure code to ATTN_ERR_CUDA.  Deviation from a single
 * "timeout" code: device-side failures (a wait that ran out, a bad index)
 * cannot be returned by an asynchronous call, so they set bits of a device
 * status word (ATTN_DEV_*), and attn_query_status returns ATTN_ERR_DEVICE
 * with those bits in *device_flags.                                          */
typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_NULLPTR = 1,     /* a required pointer is NULL                    */
    ATTN_ERR_INVALID = 2,     /* a size, dtype, mode or stride is not valid    */
    ATTN_ERR_UNSUPPORTED = 3, /* valid, but outside what the kernels cover     */
    ATTN_ERR_WORKSPACE = 4,   /* workspace NULL, too small or misaligned       */
    ATTN_ERR_ALIGN = 5,       /* a tensor breaks the 16-byte rule above        */
    ATTN_ERR_CUDA = 6,        /* a CUDA runtime / driver call failed           */
    ATTN_ERR_DEVICE = 7       /* attn_query_status: the device flagged an error */
} attn_status_t;

/* Bits of the device status word (attn_query_status).                        */
#define ATTN_DEV_TIMEOUT      0x1u  /* a bounded barrier wait ran out; the CTA quit */
#define ATTN_DEV_INDEX_RANGE  0x2u  /* a topk index outside [0, S2_b / block_size), or a
                                       position outside [0, max_pos), or a cache
                                       length outside [0, s_kv], or a page id outside
                                       [0, n_pages), or new tokens' counts that are
                                       not ascending                                 */
#define ATTN_DEV_INDEX_DUP    0x4u  /* a block listed twice for one (token, kv head) */

typedef enum { ATTN_F16 = 0, ATTN_BF16 = 1 } attn_dtype_t;

/* Causal alignment.  Top-left: key j is visible to query i iff j <= i.
 * Bottom-right: iff j <= i + (s_kv - s_q).  Both coincide when s_q == s_kv.   */
typedef enum {
    ATTN_MASK_NONE = 0,
    ATTN_CAUSAL_TOP_LEFT = 1,
    ATTN_CAUSAL_BOTTOM_RIGHT = 2
} attn_mask_t;

/* A 16-bit tensor seen as logical [B, H, S, D] with element strides
 * (sb, sh, ss, 1).  The sample's BSHD storage viewed as BHSD has
 * (S*H*D, D, H*D, 1).  In packed (varlen, TND) mode token t of head h is at
 * ptr + t*ss + h*sh and sb is ignored.  An input's stride may be 0 (the same for
 * all sequences, heads or tokens); the elements of an output are apart.      */
typedef struct {
    void *ptr;
    int64_t sb, sh, ss;
} attn_view_t;

typedef struct {
    attn_dtype_t dtype;
    int64_t b;              /* batch size (number of sequences)                */
    int64_t h;              /* query heads                                     */
    int64_t h_kv;           /* key/value heads; h % h_kv == 0                  */
    int64_t s_q, s_kv;      /* fixed lengths; ignored in packed mode           */
    int64_t d;              /* head dim: 64 or 128                             */
    double scale;           /* multiplies q.k, e.g. 1/sqrt(d)                  */
    attn_mask_t mask;
    /* Packed mode: host arrays of b inclusive cumulative lengths, no leading
     * zero (the Ascend page's actualSeqQLen / actualSeqKvLen form), b <= 256.
     * Both NULL: fixed-length mode.                                          */
    const int64_t *cu_seqlens_q;
    const int64_t *cu_seqlens_kv;
    /* sdpa_bwd only: an attn_dq_mode_t.  ATTN_DQ_ATOMIC: dQ accumulated with
     * fp32 reductions whose order varies from run to run.  ATTN_DQ_SPLIT:
     * bitwise reproducible dQ; each of dq_splits partial fp32 buffers (0: a
     * default) has one writer that adds in a fixed order, and the buffers are
     * summed in index order.  ATTN_DQ_ORDERED: bitwise reproducible dQ with
     * one fp32 buffer; the key tiles of each query tile add in decreasing
     * order, each waiting for a per-tile counter in the workspace (bounded
     * wait: ATTN_DEV_TIMEOUT), under a cooperative launch (every block of the
     * kernel resident at once); problems of more than 4096 work units (key
     * tiles of 128 rows x sequences x kv heads) return ATTN_ERR_UNSUPPORTED.
     * [Ascend] "Constraints": deterministic computation is opt-in.          */
    int deterministic;
    int dq_splits;
} attn_sdpa_desc_t;

typedef enum { ATTN_DQ_ATOMIC = 0, ATTN_DQ_SPLIT = 1, ATTN_DQ_ORDERED = 2 } attn_dq_mode_t;

/* Workspace bytes for sdpa_fwd_stats and for sdpa_bwd with this descriptor.
 * Either output pointer may be NULL.  Host only; no CUDA call.
 * [cuDNN] workspace cell (the caller queries the graph's workspace size and
 * allocates it); [Ascend] "Function Prototype" (first phase of the two-phase
 * API returns workspaceSize).                                               */
attn_status_t sdpa_workspace_size(const attn_sdpa_desc_t *desc, size_t *fwd_bytes, size_t *bwd_bytes);

/* Forward in training mode.  [cuDNN] forward-graph cell (sdpa with
 * is_inference=False, attn_scale, causal mask, emitting O and the (B,H,S,1)
 * float32 stats); [PR] the attention formula (softmax of scaled scores times
 * V).  q, o: [B,h,s_q,d] views; k, v: [B,h_kv,s_kv,d].
 * lse (fp32, natural log, contiguous): [B][h][s_q] in fixed-length mode,
 * [h][T_q] in packed mode (T_q = total query tokens).                        */
attn_status_t sdpa_fwd_stats(const attn_sdpa_desc_t *desc, attn_view_t q, attn_view_t k, attn_view_t v,
                             attn_view_t o, float *lse, void *workspace, size_t workspace_bytes,
                             void *stream);

/* Backward.  [cuDNN] backward-graph cell (sdpa_backward from Q, K, V, O, dO
 * and the stats, FlashAttention-2, attn_scale, causal mask; dQ, dK, dV
 * allocated like the inputs); [Ascend] "Function / Formula" for the
 * gradient formulas; [Ascend] "Constraints" for opt-in deterministic
 * computation.  q, o, dO, dQ: [B,h,s_q,d] views; k, v, dK, dV: [B,h_kv,s_kv,d];
 * lse as sdpa_fwd_stats writes it.  dQ / dK / dV may have any strides that
 * follow the 16-byte rule (the sample allocates them empty_like the inputs).
 * Outputs have the input dtype, rounded to nearest even.  No block of any
 * kernel waits for another block (in ATTN_DQ_ORDERED, blocks wait for one
 * another under a cooperative launch, which starts once all of them can be
 * resident), so the call is safe next to other work on the device (other
 * streams, other processes).                                                */
attn_status_t sdpa_bwd(const attn_sdpa_desc_t *desc, attn_view_t q, attn_view_t k, attn_view_t v,
                       attn_view_t o, attn_view_t dO, const float *lse, attn_view_t dQ, attn_view_t dK,
                       attn_view_t dV, void *workspace, size_t workspace_bytes, void *stream);

/* Allocation-free variant of sdpa_bwd.  The pages this library follows
 * have no counterpart to it; it exists for callers that cannot allocate
 * device memory when they run the backward (an engine or plugin that owns
 * all device memory and forbids side allocations, a loop that must not
 * allocate once running).  Instead of a caller workspace it uses a static
 * scratch array of ATTN_STATIC_SCRATCH_BYTES compiled into the library;
 * every GPU that loads the library holds those bytes until the process exits.
 * Arguments and results are those of sdpa_bwd; the call allocates nothing.
 *  - Problems whose sdpa_workspace_size exceeds ATTN_STATIC_SCRATCH_BYTES
 *    are rejected with ATTN_ERR_WORKSPACE before anything is launched.
 *  - The first call on a device looks up the array's device address (once
 *    per device, with that device current); make that first call before any
 *    stream capture begins.
 *  - All calls share the one array, so calls that overlap on the GPU (other
 *    streams, other host threads) race and corrupt each other's results;
 *    serialise them.  Each call re-initialises the scratch it reads, so what
 *    an earlier call left there does not matter.
 *  - Device status flags land in the static array; attn_static_scratch_status
 *    reads them back (and clears them) like attn_query_status.
 *  - The array's device address is looked up on every call (nothing is
 *    cached across contexts or cudaDeviceReset); errors of that lookup return
 *    ATTN_ERR_CUDA with the text in attn_last_error.                         */
#define ATTN_STATIC_SCRATCH_BYTES (16u << 20)
attn_status_t sdpa_bwd_static_scratch(const attn_sdpa_desc_t *desc, attn_view_t q, attn_view_t k, attn_view_t v,
                                      attn_view_t o, attn_view_t dO, const float *lse, attn_view_t dQ,
                                      attn_view_t dK, attn_view_t dV, void *stream);

/* Waits for the stream, then reads and clears the device status word that
 * the static scratch of sdpa_bwd_static_scratch holds (bits ATTN_DEV_*).
 * Returns ATTN_ERR_DEVICE when any bit was set.  No counterpart on the
 * pages.                                                                    */
attn_status_t attn_static_scratch_status(void *stream, uint32_t *device_flags);

typedef struct {
    attn_dtype_t dtype;
    int64_t b;              /* sequences; b <= 256                             */
    const int64_t *cu_seqlens_q;   /* host, b inclusive cumulative lengths   */
    const int64_t *cu_seqlens_kv;  /* host, b inclusive cumulative lengths   */
    int64_t n1;             /* query heads (headNum)                          */
    int64_t n2;             /* key/value heads; n1 % n2 == 0, n1/n2 <= 32     */
    int64_t d;              /* head dim of q and k: 128 or 192                */
    double scale;           /* scaleValue                                     */
    int64_t block_size;     /* selectedBlockSize: 64                          */
    int64_t block_count;    /* selectedBlockCount in [1, 128], count*size < 8192 */
    int sparse_mode;        /* 0: only the selection; 2: also causal,
                               bottom-right aligned per sequence              */
    int deterministic;      /* bitwise reproducible dQ, dK, dV, needing
                               d = d_v = 128 (ATTN_ERR_UNSUPPORTED otherwise):
                               0 off; 1 dQ per (token, selected slot) in the
                               workspace, summed in slot order (T1 n1
                               block_count d 4 bytes, plus the dK / dV rows of
                               every work unit); 2 one dQ accumulator
                               whose adds for a token go in decreasing block
                               order behind a counter per (token, kv head)
                               (T1 n2 (block_count + 1) 4 bytes; a
                               cooperative launch)                            */
    int64_t d_v;            /* head dim of v, O, dO and dv: 128 or 192; 0 means
                               d ([Ascend] Constraints: D is 192 or 128, and K
                               and V may differ)                              */
    int grad_fp32;          /* 1: dq, dk, dv are fp32; 0: the input dtype
                               ([Ascend] parameter table: FLOAT16, BFLOAT16,
                               FLOAT32 outputs)                               */
    /* attenMaskOptional ([Ascend] function prototype and parameter table: a
     * 2-D BOOL / UINT8 mask that no formula on the page uses).  Read here as:
     * device array [mask_rows][mask_cols] of uint8, row-major; entry (i, j)
     * nonzero removes key j for query i (positions local to the sequence),
     * on top of the selection and the sparse mode; it must cover every
     * sequence (mask_rows >= its query length, mask_cols >= its key length).
     * NULL: no mask.                                                       */
    const uint8_t *atten_mask;
    int64_t mask_rows, mask_cols;
} attn_nsa_desc_t;

/* NSA selected-attention forward (training mode): O and the softmax stats the
 * backward reads.  [Ascend] "Function / Formula" (gather of the selected
 * blocks, then attention over them) and parameter table (softmaxMax /
 * softmaxSum [T1, N1, 8]).  For query token t, kv head g and query head
 * h of g, over the keys of the selected blocks that the sparse mode leaves
 * visible: softmax_max = max_j s_j with s_j = scale q.k_j, softmax_sum =
 * sum_j exp(s_j - softmax_max), O = sum_j exp(s_j - softmax_max) v_j /
 * softmax_sum; all 8 lanes of a stats row hold the same value.  A row that
 * sees no key has O = 0, softmax_max = -inf, softmax_sum = 0.
 *   q : [T1][n1][d]  k : [T2][n2][d]  v : [T2][n2][d_v]  o : [T1][n1][d_v]
 *   topk : as for the backward; invalid indices are skipped and flagged.
 * Workspace: nsa_fwd_workspace_size bytes (d = d_v = 128 with blocks of 64
 * runs on the tensor cores and needs the backward's block lists and fp32
 * row / O accumulators; other shapes need the device status word alone). */
attn_status_t nsa_fwd_workspace_size(const attn_nsa_desc_t *desc, size_t *bytes);
attn_status_t nsa_selected_attn_fwd(const attn_nsa_desc_t *desc, const void *q, const void *k, const void *v,
                                    const int32_t *topk, void *o, float *softmax_max, float *softmax_sum,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes for nsa_selected_attn_bwd.  Host only; no CUDA call.
 * [Ascend] "Function Prototype": aclnnNsaSelectedAttentionGradGetWorkspaceSize. */
attn_status_t nsa_workspace_size(const attn_nsa_desc_t *desc, size_t *bytes);

/* NSA selected-attention backward.  [Ascend] "Function / Formula" (gather of
 * the selected blocks, then the attention backward; dK / dV scattered back
 * through the indices), parameter table (TND layout, actualSeqQLen /
 * actualSeqKvLen, softmaxMax / softmaxSum, topkIndices, scaleValue,
 * selectedBlockSize / Count, sparseMode) and "Constraints".  Layout, all
 * contiguous (d_v = value head dim):
 *   q, dq : [T1][n1][d]    o, dO : [T1][n1][d_v]
 *   k, dk : [T2][n2][d]    v, dv : [T2][n2][d_v]
 *   dq, dk, dv are fp32 when grad_fp32 is set, else the input dtype.
 *   softmax_max, softmax_sum : [T1][n1][8] fp32 (the 8 lanes hold one value;
 *       lane 0 is read): P = exp(scale q.k - max) / sum over the selection.
 *   topk : [T1][n2][block_count] int32 block ids local to the token's
 *       sequence, each in [0, S2_b / block_size), distinct per (token, head).
 * Every selected block must lie inside its sequence: S2_b % block_size == 0
 * and S2_b >= block_count * block_size for every sequence.  As for sdpa_bwd,
 * blocks wait for one another only in deterministic mode 2, under a
 * cooperative launch.                                                        */
attn_status_t nsa_selected_attn_bwd(const attn_nsa_desc_t *desc, const void *q, const void *k,
                                    const void *v, const void *o, const void *dO,
                                    const float *softmax_max, const float *softmax_sum,
                                    const int32_t *topk, void *dq, void *dk, void *dv,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* [Ascend] "Function / Formula" (Gather(key, topkIndices)), read in the
 * backward direction: which tokens selected each block.
 * The inverted index the NSA backward builds internally, exposed so callers
 * (and tests) can use or check it: for every (sequence b, kv head g, block k)
 * in that order, row r = (b * n2 + g) * nblk_max + k with
 * nblk_max = max_b S2_b / block_size, tokens[offsets[r] .. offsets[r+1]) are
 * the ascending global ids of the query tokens whose topk lists block k and
 * see at least one of its keys under the sparse mode.  offsets (int32,
 * nblk_max * n2 * b + 1 entries) and tokens (int32, T1 * n2 * block_count
 * entries) are device memory; *nblk_max_out (host) receives nblk_max.
 * Invalid indices are skipped and flagged in the device status word.        */
attn_status_t nsa_block_lists(const attn_nsa_desc_t *desc, const int32_t *topk, int32_t *offsets,
                              int32_t *tokens, int64_t *nblk_max_out, void *workspace, size_t workspace_bytes,
                              void *stream);

/* A learned relative position bias by buckets.  No counterpart on the pages: it
 * is what a model whose positions enter the scores this way adds to the dense
 * calls above.  The score of a query and a key becomes
 *   s = scale q.k + table[bucket(delta)][query head],
 *   delta = key position - query position,
 * where key j stands at position j of its sequence and query i at i, or at
 * i + s_kv - s_q under ATTN_CAUSAL_BOTTOM_RIGHT.
 * The bucket of delta: with both directions, keys after the query (delta > 0)
 * take the upper half of the buckets, n = num_buckets / 2 and x = |delta|; with
 * one, n = num_buckets and x = max(-delta, 0).  With e = n / 2 (rounded down):
 *   x < e: x;  else min(n - 1, e + floor(log(x / e) / log(max_distance / e) (n - e))),
 * in real arithmetic (attn_relbias_bucket evaluates it).
 * A table entry of -1e30 or less masks its bucket: keys in it are not visible to
 * that head.  A masked key of the same sequence still meets the products with
 * weight 0, so its k and v have to be finite (0 times infinity is NaN); keys of
 * other sequences, and a cache's from its length on, may hold anything.     */
typedef struct {
    const void *table;      /* device [num_buckets][h], contiguous              */
    int table_type;         /* ATTN_F16, ATTN_BF16 or ATTN_F32                  */
    int64_t num_buckets;    /* 2 .. 128; even and >= 4 with both directions     */
    int64_t max_distance;   /* e < max_distance <= 65536                        */
    int bidirectional;      /* 1: keys after the query have buckets of their own;
                               0: they share bucket 0                           */
} attn_relbias_t;

#define ATTN_F32 2

/* Bucket of a key delta positions after its query.  Host only; the table is not
 * read.                                                                     */
attn_status_t attn_relbias_bucket(const attn_relbias_t *bias, int64_t delta, int64_t *bucket);

/* Workspace bytes of the two calls below.  Either output pointer may be NULL.
 * Host only; no CUDA call.                                                  */
attn_status_t sdpa_relbias_workspace_size(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, size_t *fwd_bytes,
                                          size_t *bwd_bytes);

/* sdpa_fwd_stats with the bias in the scores: everything but bias as there. */
attn_status_t sdpa_relbias_fwd_stats(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, attn_view_t q,
                                     attn_view_t k, attn_view_t v, attn_view_t o, float *lse, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* sdpa_bwd with the bias in the scores, and the table's gradient
 *   dtable[n][head] = sum of dS over the queries and keys with bucket n
 * (fp32 [num_buckets][h], contiguous, overwritten): dS is summed in fp32 before
 * it is rounded for the other gradients, in an order that does not change from
 * run to run in any dQ mode.  P and dS are computed in fp32 for both types.
 * Everything else as in sdpa_bwd.                                           */
attn_status_t sdpa_relbias_bwd(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, attn_view_t q, attn_view_t k,
                               attn_view_t v, attn_view_t o, attn_view_t dO, const float *lse, attn_view_t dQ,
                               attn_view_t dK, attn_view_t dV, float *dtable, void *workspace, size_t workspace_bytes,
                               void *stream);

/* One new token of every sequence over a key / value cache: O of the biased
 * attention above, without stats.  desc: s_q = 1, s_kv = the keys a sequence's
 * cache has room for, mask = ATTN_CAUSAL_BOTTOM_RIGHT (the new token is the last of
 * its sequence), fixed-length mode; deterministic is ignored (the result is
 * always bitwise reproducible).  q, o: [b,h,1,d]; k, v: [b,h_kv,s_kv,d] views.
 * lens: device int32 [b], the keys cached for each sequence, the new token's own
 * among them (NULL: s_kv for all); read on the device, so a captured call
 * follows a growing cache.  Keys from lens[b] on are not read.  A sequence
 * without keys gets O = 0; a length outside [0, s_kv] is brought into it and
 * sets ATTN_DEV_INDEX_RANGE.                                                */
attn_status_t sdpa_relbias_decode_workspace_size(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias,
                                                 size_t *bytes);
attn_status_t sdpa_relbias_decode(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, attn_view_t q,
                                  attn_view_t k, attn_view_t v, const int32_t *lens, attn_view_t o, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* A paged key / value cache: pages of page_size tokens in any order, found through
 * a table.  No counterpart on the pages: it is what a program that serves a model
 * keeps its keys and values in.  Element (page p, token t, kv head g, i) of k and v
 * is at p*sp + t*ss + g*sh + i (elements of `type`), its row's scale at p*scale_sp +
 * t*scale_ss + g*scale_sh.  Strides are not negative; those of k and v are
 * multiples of 16 bytes, both start on a 16-byte boundary, and a page spans less
 * than 2^31 elements of each.                                                */
#define ATTN_E4M3 3
typedef struct {
    void *k, *v;
    float *k_scale, *v_scale;  /* ATTN_E4M3: a scale for each row; else ignored  */
    int type;                  /* the descriptor's dtype, or ATTN_E4M3            */
    int64_t n_pages;
    int64_t page_size;         /* 16, 32, 64, 128 or 256                          */
    int64_t sp, sh, ss;
    int64_t scale_sp, scale_sh, scale_ss;
} attn_paged_cache_t;

/* Where the sequences and their new tokens lie, all of it read on the device, so
 * that a captured call follows a growing cache.  Sequence n has lens[n] tokens
 * in the cache, its m new ones (the last) among them: new token i stands at position
 * lens[n] - m + i, and position x lies in page page_table[n*table_stride + x /
 * page_size].  The new tokens' rows: cu_new NULL: s_q of each sequence, in [b,h,s_q,d]
 * views.  Else packed views, token row t at t*ss: rows cu_new[n] .. cu_new[n+1] - 1,
 * of `tokens` in all; rows that belong to no sequence are not written, and what they
 * hold changes no result, but all `tokens` rows of a view that a call reads have to be
 * memory that it may read (it may load them and not use them).  A new token at a position below 0 (a sequence with more new tokens than
 * cached ones, padded in front) is not written to the cache, is read back as zeros
 * and sees no key.  Table entries of pages that hold no needed position are not
 * read.  Lengths outside [0, s_kv] and counts out of order or range are brought
 * into range, and they and page ids outside [0, n_pages) set ATTN_DEV_INDEX_RANGE; a
 * token of such a page is not written, and read as zeros.                    */
typedef struct {
    const int32_t *page_table;  /* device [b] rows of table_pages ids             */
    int64_t table_stride, table_pages;  /* table_pages*page_size >= s_kv          */
    const int32_t *lens;        /* device [b]                                     */
    const int32_t *cu_new;      /* device [b + 1], or NULL                        */
    int64_t tokens;             /* rows of the packed views; ignored without cu_new */
} attn_paged_seqs_t;

/* The three calls take an attn_sdpa_desc_t in fixed-length mode (its host arrays
 * NULL): s_kv = the most tokens a sequence may have cached (up to 2^30), s_q = the new
 * tokens of every sequence or, with cu_new, the most that a sequence is expected to
 * have (a longer one is computed all the same: it chooses the kernel); h / h_kv <= 128;
 * the new tokens times h, and times 2 h_kv, at most 2^31 - 4096;
 * mask ATTN_MASK_NONE (a new token sees all of its sequence) or
 * ATTN_CAUSAL_BOTTOM_RIGHT (up to its own position); deterministic is ignored: the
 * results are always bitwise reproducible.
 *
 * The new tokens' rows of k and v ([b,h_kv,s_q,d] or packed views) into their places of
 * the cache.  Into ATTN_E4M3, a row x of d elements goes as
 *   a = max(max |x|, 2^-110), scale = a / 448, code = e4m3(x (448 / a)),
 * in fp32, codes rounded to nearest even, the maximum over the finite elements (an
 * infinity becomes the largest code of its sign, a NaN stays one): the row stands for
 * code * scale.  No two of the call's tokens may have one place, nor two pages, tokens
 * or heads of the cache, nor a key and a value (a stride of 0 is refused here; the
 * other calls read through it).
 * paged_cache_read: the same rows from the cache, code * scale rounded to dtype.
 * Workspace of both: paged_cache_workspace_size bytes.                       */
attn_status_t paged_cache_workspace_size(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache, size_t *bytes);
attn_status_t paged_cache_write(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache,
                                const attn_paged_seqs_t *seqs, attn_view_t k, attn_view_t v, void *workspace,
                                size_t workspace_bytes, void *stream);
attn_status_t paged_cache_read(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache,
                               const attn_paged_seqs_t *seqs, attn_view_t k, attn_view_t v, void *workspace,
                               size_t workspace_bytes, void *stream);

/* Attention of the new tokens over everything their sequences have cached (which
 * includes their own keys and values: write them first).  q, o: [b,h,s_q,d] or packed
 * views; lse (fp32, natural log, contiguous): [b][h][s_q] or [h][tokens], or NULL when
 * it is not wanted.  A new token without a visible key has O = 0, LSE = +inf.  Cached
 * rows from lens[n] on may hold anything; those of a sequence that a new token does not
 * see still meet it with weight 0, so they have to be finite.  The weights are rounded
 * to 16 bits for their product with the values: to dtype, or over ATTN_E4M3 to half
 * precision, times their value's scale, relative to the largest such product that the
 * row sees (below 2^-25 of it, or of the largest weight of an ATTN_F16 cache, they
 * vanish).  Value scales may be of either sign, and a key's scale matters as far as its
 * weight does; weights are lost beside a key of a scale 2^100 larger, and bits of
 * scales below 2^-80.                                                        */
attn_status_t sdpa_paged_workspace_size(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache, size_t *bytes);
attn_status_t sdpa_paged_fwd(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache,
                             const attn_paged_seqs_t *seqs, attn_view_t q, attn_view_t o, float *lse, void *workspace,
                             size_t workspace_bytes, void *stream);

/* Norm and rotation of the query and key heads.  Like the relative-bias calls,
 * these have no counterpart on the pages: they are what a model runs between
 * its projections and the attention. */
typedef struct {
    attn_dtype_t dtype;     /* q, k, their outputs and gradients               */
    int64_t b, s;           /* sequences and tokens of each; packed (TND)
                               tensors: b = 1, s = all tokens, with positions   */
    int64_t h, h_kv;        /* query / key heads; one of them may be 0: that
                               side's pointers are then ignored                 */
    int64_t d;              /* head dim: 64, 128 or 192                         */
    int64_t rotary_dim;     /* leading elements of a head that are rotated: a
                               multiple of 16 up to d; 0: norm only             */
    int interleaved;        /* pairs are (2i, 2i + 1) when 1, (i, i + rotary_dim
                               / 2) when 0                                      */
    double eps;             /* added to the mean square; > 0 in fp32            */
    int weight_fp32;        /* q_weight, k_weight are fp32 when 1, dtype when 0 */
    int64_t max_pos;        /* rows of cos and sin (ignored with rotary_dim 0)  */
} attn_qk_norm_desc_t;

/* Workspace bytes of the two calls below.  Either pointer may be NULL.  Host
 * only; no CUDA call.                                                       */
attn_status_t qk_norm_rope_workspace_size(const attn_qk_norm_desc_t *desc, size_t *fwd_bytes, size_t *bwd_bytes);

/* For every token and head, with x the head's d elements:
 *   z = weight * x * r,  r = 1 / sqrt(mean(x^2) + eps),
 *   y = z with each pair (a, b) of its first rotary_dim elements turned by the
 *       token's angle: (a cos - b sin, b cos + a sin),
 * computed in fp32 and rounded once (the squares' sum too: elements of bf16 from
 * about 1e18 on pass its range).  q, q_out: [b,h,s,d] views; k, k_out:
 * [b,h_kv,s,d]; an output view may be its input view (in place), and must not
 * overlap it otherwise.  q_weight, k_weight: [d], shared by the heads (NULL:
 * ones).  cos, sin: fp32 [max_pos][rotary_dim / 2], 16-byte aligned;
 * positions: int32 [b][s] rows of them (NULL: a token's index in its
 * sequence).  A token whose position is outside [0, max_pos) gets zero
 * outputs and sets ATTN_DEV_INDEX_RANGE.                                    */
attn_status_t qk_norm_rope_fwd(const attn_qk_norm_desc_t *desc, attn_view_t q, attn_view_t k, const void *q_weight,
                               const void *k_weight, const float *cos, const float *sin, const int32_t *positions,
                               attn_view_t q_out, attn_view_t k_out, void *workspace, size_t workspace_bytes,
                               void *stream);

/* Gradients of the call above from its inputs and the gradients dq_out,
 * dk_out of its outputs (sdpa_bwd's dQ and dK), with xh = x r and dz = dy
 * turned back by the token's angle:
 *   dweight = sum over tokens and heads of dz * xh,
 *   dx = r (g - xh mean(g * xh)),  g = dz * weight.
 * dq, dk may be the views of dq_out, dk_out (in place).  dq_weight, dk_weight:
 * fp32 [d], or NULL when not wanted; summed in a fixed order, so the call is
 * bitwise reproducible.  A token whose position is out of range gets zero
 * gradients and adds nothing to the weights'.                              */
attn_status_t qk_norm_rope_bwd(const attn_qk_norm_desc_t *desc, attn_view_t q, attn_view_t k, attn_view_t dq_out,
                               attn_view_t dk_out, const void *q_weight, const void *k_weight, const float *cos,
                               const float *sin, const int32_t *positions, attn_view_t dq, attn_view_t dk,
                               float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                               void *stream);

/* Waits for the stream, then reads the device status word of a workspace a
 * previous call used (bits ATTN_DEV_*; 0 when clean) and clears it.
 * Returns ATTN_ERR_DEVICE when any bit was set.  [Ascend] "Return Value"
 * (failures reported as codes); see the deviation note above the enum.     */
attn_status_t attn_query_status(void *workspace, void *stream, uint32_t *device_flags);

/* Self-test of the device failure path: launches one block whose bounded
 * mbarrier wait (the same wait every tensor-core kernel uses) can never
 * complete, so after about limit_s seconds (0 < limit_s <= 2) it gives up,
 * sets ATTN_DEV_TIMEOUT in the status word at `workspace` (at least 4 bytes,
 * 4-byte aligned) and returns; the context stays usable.  Read the flag with
 * attn_query_status.  [Ascend] "Return Value" (failures as codes, never a
 * crash).                                                                   */
attn_status_t attn_selftest_wait_timeout(void *workspace, size_t workspace_bytes, double limit_s, void *stream);

/* Test aid: launches `blocks` blocks of 32 threads that each reserve
 * smem_bytes (<= 200 KiB) of shared memory and hold their SM for `seconds`
 * (0 < seconds <= 5) without touching memory, so a test can run the
 * backward while other work occupies part of the GPU.  No counterpart on the
 * pages.                                                                    */
attn_status_t attn_selftest_occupy(int blocks, size_t smem_bytes, double seconds, void *stream);

/* Optional instrumentation for benchmarks.  While set, every sdpa_bwd and
 * nsa_selected_attn_bwd call made from this host thread records the CUDA
 * event `before` on its stream just before its main backward kernel and
 * `after` just after it, so the main kernel can be timed alone.  Events are
 * cudaEvent_t handles passed as void*; NULL, NULL clears.  Never fails.    */
attn_status_t attn_set_main_kernel_events(void *before, void *after);

/* Text of the CUDA runtime / driver error behind the most recent
 * ATTN_ERR_CUDA returned to this host thread ("" if none).  Static storage. */
const char *attn_last_error(void);

/* Human-readable name of a status code (static storage).                    */
const char *attn_status_string(attn_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* ATTNBWD_H */
