/*
 * libspecverify -- the single-forward-pass verification step of
 * self-speculative decoding, for NVIDIA GB300 (sm_103a).
 *
 * One verification step, as the pages describe it:
 *   1. spec_mask_build   which speculative rows see which block columns
 *   2. spec_verify_attn  masked attention of the speculative rows over
 *                        (committed KV prefix || soft prompt || the block)
 *   3. spec_accept       vocab-wide argmax / log-sum-exp per judged row,
 *                        then the LA threshold longest prefix or the greedy
 *                        tree walk
 *   4. kv_commit         append the accepted rows' K/V to the cache; every
 *                        other speculative K/V row is dropped
 * and, around it: spec_accept_soft (soft matching), spec_draft_tree and
 * spec_prune_tree (the next draft), spec_stream_rotate_values (stream values
 * by rotation), spec_future_gather (ConFu's future token),
 * spec_la_prefill_attn (prefill-form LA).
 *
 * For serving: a KV cache in 8 bits with a scale per (page, KV head) --
 * spec_verify_attn_kv8 attends over it, kv8_commit and kv8_append write it,
 * spec_page_plan builds block tables and slot maps from request lengths --
 * and spec_logits_adjust (penalties, biases and grammar masks ahead of the
 * acceptance).  A prompt, or a chunk of one, passes through spec_page_plan,
 * spec_rope (rotary positions), kv_append or kv8_append (its keys and values
 * into either cache) and spec_chunk_attn or spec_chunk_attn_kv8 (its attention
 * over what the cache then holds).  The pages have no counterpart of these.
 *
 * Sources, cited by page title and section / equation:
 *   [LA]  "Lookahead Attention: Self-Speculative Verification via Parallel
 *         Token Proposals": sec. 2.1-2.4, sec. 3.1 (mask M_LA), sec. 3.2
 *         (lookahead KV discarded), sec. 3.3 (batched lookahead, padding).
 *   [CF]  "ConFu: Contemplate the Future for Better Speculative Sampling"
 *         (reading notes): key design 1 (soft prompt seen only by
 *         contemplate tokens, one contemplate token per draft node, 2T
 *         tokens in one verify pass).
 *   [SS]  "Speculative Streaming: Fast LLM Inference without Auxiliary
 *         Models": Eq. 1-2 (multi-stream attention), Eq. 4 and the text
 *         after it (tree attention mask), batching with streams, the
 *         verification step (hard matching, beta + 1 tokens advanced).
 *
 * Conventions for every call:
 *   - All tensor arguments are DEVICE pointers owned by the caller, dense
 *     and row-major in the layout stated; the library never frees them and
 *     keeps no reference after the call returns.
 *   - Calls are asynchronous on the caller's CUDA stream (`stream`, a
 *     cudaStream_t; NULL = legacy default stream) and launch only this
 *     library's kernels.  The library allocates no device memory: scratch
 *     comes from a caller-provided workspace (spec_verify_attn), or, for
 *     spec_verify_attn_noalloc, from one fixed array inside the library.
 *   - Errors visible on the host (bad sizes, NULL pointers, unsupported
 *     dtype/shape, a too-small workspace) are returned before anything is
 *     launched.  Errors only visible on the device (a bad parent pointer, a
 *     page id out of range, a full cache) set bits in a per-device status
 *     word and the kernel skips the offending work; nothing traps, and
 *     every wait inside a kernel is bounded (spec_set_wait_limit; on expiry
 *     SPEC_DEV_TIMEOUT is set and the kernel returns).  spec_get_status()
 *     reads and clears that word.
 *   - The status word is shared by all calls on a device: with concurrent
 *     streams, an error bit cannot be attributed to one call.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPECVERIFY_VERSION 100

typedef int spec_status_t;

/* return codes */
#define SPEC_OK              0
#define SPEC_ERR_INVALID_ARG 1  /* NULL pointer, negative / inconsistent size */
#define SPEC_ERR_UNSUPPORTED 2  /* dtype or shape this build does not handle */
#define SPEC_ERR_BAD_TREE    3  /* reserved: tree errors are device-detected */
#define SPEC_ERR_CAPACITY    4  /* workspace too small */
#define SPEC_ERR_CUDA        5  /* a CUDA runtime call failed */
#define SPEC_ERR_DEVICE      6  /* spec_get_status found device error bits */

/* element types */
#define SPEC_F32  0
#define SPEC_BF16 1

/* KV-cache layouts */
#define SPEC_KV_CONTIGUOUS 0
#define SPEC_KV_PAGED      1

/* acceptance modes */
#define SPEC_ACCEPT_THRESH_CHAIN 0  /* [LA] sec. 2.4 */
#define SPEC_ACCEPT_GREEDY_TREE  1  /* [SS] verification step, [CF] */

/* vparent codes (spec_mask_build) */
#define SPEC_VP_ROOT (-1)   /* row sees the prefix and itself only */
#define SPEC_VP_PAD  (-2)   /* padding row ([LA] sec. 3.3): sees nothing */

/* row_flags bits (spec_mask_build output, spec_verify_attn input) */
#define SPEC_ROW_VALID     1u
#define SPEC_ROW_SEES_SOFT 2u

/* device status bits (spec_get_status) */
#define SPEC_DEV_BAD_TREE     0x01  /* vparent not an earlier valid row */
#define SPEC_DEV_BAD_PAGE     0x02  /* page id (or slot) outside the cache */
#define SPEC_DEV_SEQ_OVERFLOW 0x04  /* seq_len outside [0, cache capacity] */
#define SPEC_DEV_CAPACITY     0x08  /* commit: cache or free list full */
#define SPEC_DEV_BAD_INDEX    0x10  /* path / row_of / acc_len out of range */
#define SPEC_DEV_TIMEOUT      0x20  /* an internal pipeline wait expired */

/* Maximum speculative rows per request (block columns). */
#define SPEC_MAX_ROWS 256

/*
 * The committed KV cache ([LA] sec. 3.2, [SS] "no additional KV caching":
 * only accepted tokens' K/V ever enter it).
 *
 * kind == SPEC_KV_CONTIGUOUS:
 *   k, v : [batch][n_kv_heads][max_seq][head_dim]   (dtype)
 *   request b's token t lives at k[b][h][t][:].
 * kind == SPEC_KV_PAGED:
 *   k, v : [n_pages][n_kv_heads][head_dim / 64][page_size][64] (dtype)
 *   page_table : int32 [batch][max_pages_per_seq]; token t of request b
 *   lives in page page_table[b][t / page_size], slot t % page_size, and its
 *   element j of KV head h is k[page][h][j / 64][t % page_size][j % 64].
 *   Within one (page, head) the head dimension is split into 64-element
 *   blocks, each holding page_size rows: one (page, head) is a single
 *   contiguous 2-D tile, fetched by one tensor copy.  For head_dim = 64
 *   this is [n_pages][n_kv_heads][page_size][64].
 *   Entries past ceil(seq_len[b] / page_size) are unused.
 */
typedef struct spec_kv_desc {
    int kind;
    int dtype;
    int n_kv_heads;
    int head_dim;
    void *k;
    void *v;
    int batch;
    int max_seq;             /* contiguous: token capacity per request */
    int n_pages;             /* paged */
    int page_size;           /* paged: tokens per page (multiple of 16) */
    int max_pages_per_seq;   /* paged: row length of page_table */
    int32_t *page_table;     /* paged */
} spec_kv_desc;

/*
 * A KV cache in 8 bits, paged: e4m3 codes and one fp32 scale for the keys
 * and one for the values of every (page, KV head); an element stands for
 * code * scale.
 *
 *   kv     : uint8 [n_pages][n_kv_heads][page_size / 8][2][8][head_dim]:
 *            token t of a page has its key at [t / 8][0][t % 8][:] and its
 *            value at [t / 8][1][t % 8][:].  One (page, head) is one
 *            contiguous tile, fetched by one tensor copy, in which both the
 *            key groups and the value groups lie at a fixed stride.
 *            16-byte aligned.
 *   scales : fp32 [n_pages][n_kv_heads][2] (keys, values).
 *   page_table as in spec_kv_desc.  page_size: a multiple of 16, <= 256.
 *
 * The writers (kv8_commit, kv8_append) give a block the scale 2^e with the
 * smallest e, -60 <= e <= 60, for which every value is at most 448 * 2^e: a
 * power of two costs e4m3 (a floating-point format) no precision, and makes
 * the step to a larger scale exact but for e4m3's subnormals.  Larger values
 * saturate.  A non-finite value makes the block's scale NaN, so the block
 * reads as NaN until its page is begun again.  Readers take any finite scale;
 * one below 2^-60 counts as 2^-60, one above 2^60 as 2^60.
 */
typedef struct spec_kv8_desc {
    int n_kv_heads;
    int head_dim;            /* 64 or 128 */
    void *kv;
    float *scales;
    int batch;
    int n_pages;
    int page_size;
    int max_pages_per_seq;
    int32_t *page_table;     /* int32 [batch][max_pages_per_seq] */
} spec_kv8_desc;

/* Shape of one verify-attention call. */
typedef struct spec_attn_desc {
    int batch;         /* B */
    int n_rows;        /* R: padded speculative rows per request (<= 256) */
    int n_q_heads;     /* Hq (multiple of n_kv_heads) */
    int n_kv_heads;    /* Hkv */
    int head_dim;      /* d: 64 or 128 */
    int dtype;         /* SPEC_BF16 or SPEC_F32, for q, kb, vb, soft, o, cache */
    int n_soft;        /* soft-prompt KV entries (0 = none), <= 64 */
    float scale;       /* softmax scale; 0 -> 1/sqrt(head_dim) ([SS] Eq. 1) */
    int split_tokens;  /* prefix tokens per split; 0 = chosen by the library */
} spec_attn_desc;

/* Shape and rule of one acceptance call. */
typedef struct spec_accept_desc {
    int mode;          /* SPEC_ACCEPT_THRESH_CHAIN or SPEC_ACCEPT_GREEDY_TREE */
    float tau;         /* threshold on the proposal probability (chain mode) */
    int batch;         /* B */
    int n_judge_rows;  /* Rj: logits rows per request */
    int vocab;         /* V */
    int logit_dtype;   /* SPEC_BF16 or SPEC_F32 */
    int max_nodes;     /* N: row length of tokens / tree_parent / row_of */
    int path_cap;      /* row length of path */
} spec_accept_desc;

/* Shape of one prefill-form Lookahead Attention call. */
typedef struct spec_prefill_desc {
    int batch;         /* B */
    int n_orig;        /* n: original positions per request (>= 1) */
    int n_look;        /* k: lookahead positions per request (>= 0) */
    int n_q_heads;     /* Hq (multiple of n_kv_heads) */
    int n_kv_heads;    /* Hkv */
    int head_dim;      /* d: 128 */
    int dtype;         /* SPEC_BF16 */
    float scale;       /* softmax scale; 0 -> 1/sqrt(head_dim) */
} spec_prefill_desc;

/* Shape of one soft-matching acceptance call. */
typedef struct spec_soft_desc {
    int batch;          /* B */
    int n_judge_rows;   /* Rj: target logits rows per request */
    int n_draft_rows;   /* Rd: draft logits rows per request (0 = none) */
    int vocab;          /* V (<= 1,048,576) */
    int logit_dtype;    /* SPEC_BF16 or SPEC_F32, target and draft logits */
    int max_nodes;      /* N: row length of tokens / tree_parent / row_of */
    int path_cap;       /* row length of path */
    float temperature;  /* T > 0: p = softmax(z / T), q = softmax(z_d / T) */
} spec_soft_desc;

/* Shape of one draft-tree construction call. */
typedef struct spec_draft_desc {
    int batch;          /* B */
    int n_stream_rows;  /* rows per request in stream_logits */
    int gamma;          /* speculative streams (tree depth) */
    int k;              /* tokens per stream (1..8) */
    int vocab;          /* V (>= k) */
    int logit_dtype;    /* SPEC_BF16 or SPEC_F32 */
    int max_nodes;      /* row length of tokens / tree_parent (>= 1 + sum k^g) */
    int vparent_rows;   /* row length of vparent (>= nodes * (1 + gamma)) */
} spec_draft_desc;

/* Shape and threshold of one tree-pruning call. */
typedef struct spec_prune_desc {
    int batch;          /* B */
    int max_nodes;      /* N (<= 1024): row length of the tree arrays */
    int vocab;          /* V */
    int logit_dtype;    /* SPEC_BF16 or SPEC_F32 (early-exit logits) */
    float threshold;    /* an edge survives iff its probability >= threshold */
    int gamma;          /* stream rows per node in vparent */
    int vparent_rows;   /* row length of vparent (>= N * (1 + gamma)) */
} spec_prune_desc;

/* Shape of one stream value rotation call. */
typedef struct spec_rotate_desc {
    int batch;          /* B */
    int n_rows;         /* R: rows of the block per (request, KV head) */
    int n_kv_heads;     /* Hkv */
    int head_dim;       /* d (multiple of 8) */
    int dtype;          /* SPEC_BF16 or SPEC_F32 */
    int gamma;          /* streams per node (<= 64) */
    float eps;          /* rotation angle per stream index, radians */
} spec_rotate_desc;

/* Shape of one logits adjustment call. */
typedef struct spec_logits_desc {
    int batch;          /* B */
    int n_judge_rows;   /* Rj: logits rows per request */
    int vocab;          /* V */
    int logit_dtype;    /* SPEC_BF16 or SPEC_F32 */
    int max_nodes;      /* N (<= 256): row length of tokens / tree_parent; 0 = no tree */
    int hist_cap;       /* row length of history; 0 = none */
    int n_bias;         /* row length of bias_ids / bias (<= 1024); 0 = none */
    int n_masks;        /* grammar masks; 0 = none */
} spec_logits_desc;

/* Shape of one chunk attention call: a packed batch of new tokens. */
typedef struct spec_chunk_desc {
    int batch;         /* B: requests */
    int n_tokens;      /* rows of q, o and lse; the requests' new tokens fill the first */
    int n_q_heads;     /* Hq (multiple of n_kv_heads, at most 128 times as many) */
    int n_kv_heads;    /* Hkv */
    int head_dim;      /* d: 64 or 128 */
    int dtype;         /* SPEC_BF16 or SPEC_F32, for q, o and a cache of rows */
    float scale;       /* softmax scale; 0 -> 1/sqrt(head_dim) */
} spec_chunk_desc;

/* rotary layouts: which elements of a head make pair i */
#define SPEC_ROPE_PAIRS  0  /* 2i and 2i + 1 */
#define SPEC_ROPE_HALVES 1  /* i and i + rot_dim / 2 */

/* rotary frequencies (spec_rope_freqs) */
#define SPEC_ROPE_PLAIN  0
#define SPEC_ROPE_LINEAR 1
#define SPEC_ROPE_RAMP   2

/* Shape of one rotary position call. */
typedef struct spec_rope_desc {
    int n_tokens;      /* rows of q and k */
    int n_q_heads;     /* query heads; 0 = none */
    int n_k_heads;     /* key heads; 0 = none */
    int head_dim;      /* d: a multiple of 8, <= 256 */
    int rot_dim;       /* even, <= head_dim: the first elements of a head, which turn */
    int layout;        /* SPEC_ROPE_PAIRS or SPEC_ROPE_HALVES */
    int dtype;         /* SPEC_BF16 or SPEC_F32 */
    float attention;   /* factor on what turns; 0 -> 1 */
} spec_rope_desc;

/* Library version (SPECVERIFY_VERSION). */
int spec_version(void);

/* Human-readable name of a return code. */
const char *spec_status_string(spec_status_t status);

/*
 * spec_mask_build -- visibility of the speculative block ([LA] sec. 3.1 in
 * its verify form, [SS] Eq. 2 and Eq. 4 with the following text, [CF] key
 * design 1).
 *
 *   vparent    int32 [batch][n_rows]: SPEC_VP_ROOT (-1): the row sees the
 *              prefix and itself; SPEC_VP_PAD (-2): padding row; p >= 0:
 *              the row sees everything row p sees, plus itself (p must be an
 *              earlier, non-padding row: p < r).
 *   soft_flags uint8 [batch][n_rows] or NULL: nonzero -> the row also sees
 *              the soft-prompt columns (ConFu contemplate tokens).
 *   vis        uint32 [batch][n_rows][ceil(n_rows/32)] out: bit c of word
 *              c/32 of row r is set iff row r sees block column c.
 *   row_flags  uint8 [batch][n_rows] out: SPEC_ROW_VALID | SPEC_ROW_SEES_SOFT.
 *
 * A row whose vparent chain is malformed gets vis = 0 and row_flags = 0
 * and sets SPEC_DEV_BAD_TREE.  n_rows <= SPEC_MAX_ROWS.
 */
spec_status_t spec_mask_build(const int32_t *vparent, const uint8_t *soft_flags,
                              int batch, int n_rows, uint32_t *vis,
                              uint8_t *row_flags, void *stream);

/*
 * Bytes of workspace spec_verify_attn needs for this shape and cache
 * (split partials: per request, KV head and split, the packed rows'
 * running max, sum and unnormalised output in fp32; on the tensor-core
 * paths also the first tile of each CTA's range, which the attention
 * kernel writes and the combine reads, and for the tcgen05 kernel a record
 * per CTA of the split segment its range starts inside of).
 */
spec_status_t spec_verify_attn_workspace_size(const spec_attn_desc *attn,
                                              const spec_kv_desc *cache,
                                              size_t *bytes);

/*
 * spec_verify_attn -- masked attention of the speculative rows
 * ([SS] Eq. 1-2, Eq. 4; [LA] sec. 3.1; [CF] key design 1).
 *
 *   q         [batch][n_rows][n_q_heads][head_dim]
 *   cache     committed prefix (see spec_kv_desc); seq_len int32 [batch]
 *             gives each request's prefix length S_b.
 *   kb, vb    [batch][n_kv_heads][n_rows][head_dim]: the block's own K/V
 *             (never aliases the cache).
 *   soft_k/v  [n_kv_heads][n_soft][head_dim], or NULL when n_soft == 0.
 *   vis, row_flags  from spec_mask_build.
 *   o         out [batch][n_rows][n_q_heads][head_dim] (dtype)
 *   lse       out fp32 [batch][n_q_heads][n_rows]: natural-log
 *             log-sum-exp of the row's scaled scores.
 *   workspace device scratch of >= spec_verify_attn_workspace_size bytes,
 *             256-byte aligned; its contents on entry are ignored.
 *
 * For query head h the K/V head is h / (n_q_heads / n_kv_heads).  A valid
 * row r sees prefix columns 0..S_b-1, the n_soft soft columns iff
 * SPEC_ROW_SEES_SOFT, and block column c iff vis bit c; scores are
 * (q . k) * scale.  Rows without SPEC_ROW_VALID get o = 0, lse = -inf.
 * A seq_len outside [0, capacity] is clamped and sets SPEC_DEV_SEQ_OVERFLOW;
 * a page id outside [0, n_pages) is not read and sets SPEC_DEV_BAD_PAGE (the
 * affected outputs are then unspecified).
 */
spec_status_t spec_verify_attn(const spec_attn_desc *attn, const void *q,
                               const spec_kv_desc *cache, const void *kb,
                               const void *vb, const void *soft_k,
                               const void *soft_v, const int32_t *seq_len,
                               const uint32_t *vis, const uint8_t *row_flags,
                               void *o, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * spec_accept_soft -- acceptance by soft matching ([SS] verification step:
 * a drafted token x is accepted with probability min(1, p(x) / q(x)), the
 * rejection sampling of Leviathan et al.; one correction token is sampled
 * at the rejection point).
 *
 *   logits          [batch][n_judge_rows][vocab]: target (main-stream) logits.
 *   draft_logits    [batch][n_draft_rows][vocab]: the draft distributions.
 *   tokens, tree_parent, row_of, n_nodes: the draft tree as in spec_accept
 *                   (tree mode); row_of NULL = identity.
 *   child_draft_row int32 [batch][max_nodes]: the draft row node c's children
 *                   were drafted from, -1 if none.  May be NULL only when
 *                   n_draft_rows == 0 (every q is then 0).
 *   u_accept        fp32 [batch][max_nodes]: uniform in [0, 1) used when node
 *                   c is tested.
 *   u_sample        fp32 [batch]: uniform in [0, 1) for the correction token.
 *   lse_t, lse_d    fp32 out [batch][n_judge_rows], [batch][n_draft_rows]:
 *                   ln sum exp(z / T) of each row (scratch the call fills).
 *   acc_len, path, next_token, last_node: out, as spec_accept (tree mode).
 *
 * From node 0, the children c of the current node are tried in index
 * order: c (token x) is accepted iff u_accept[c] * q(x) < p(x), with p the
 * softmax(z / T) of the current node's judge row and q that of its
 * child_draft_row; the first accepted child becomes the current node.  When
 * none is accepted, next_token is drawn from max(0, p - q) normalised (from
 * p when the node has no draft row or p <= q everywhere): the smallest v
 * whose cumulative mass exceeds u_sample[b] times the total (fp32 sums); it
 * is -1 where that judge row's logits are all -inf.
 * max_nodes <= SPEC_MAX_ROWS (else SPEC_ERR_UNSUPPORTED).  A malformed index
 * anywhere in the tree (parent, token, judge or draft row) or a path longer
 * than path_cap sets SPEC_DEV_BAD_INDEX; the malformed node is never
 * accepted.  Three launches: two vocab reductions (target, draft) and one
 * test-walk-draw kernel.
 */
spec_status_t spec_accept_soft(const spec_soft_desc *desc, const void *logits,
                               const void *draft_logits, const int32_t *tokens,
                               const int32_t *tree_parent, const int32_t *row_of,
                               const int32_t *child_draft_row, const int32_t *n_nodes,
                               const float *u_accept, const float *u_sample,
                               float *lse_t, float *lse_d, int32_t *acc_len,
                               int32_t *path, int32_t *next_token, int32_t *last_node,
                               void *stream);

/*
 * spec_draft_tree -- the next step's draft tree ([SS] tree draft
 * construction, batching with streams).
 *
 *   stream_logits [batch][n_stream_rows][vocab]: the speculative streams'
 *                 logits; request b's streams 1..gamma are rows
 *                 stream_row[b] .. stream_row[b] + gamma - 1 (stream_row
 *                 NULL: rows 0..gamma-1).
 *   root_token    int32 [batch]: the root's token (the correction token).
 *   tokens, tree_parent  int32 out [batch][max_nodes]; n_nodes int32 out
 *                 [batch] = 1 + sum_{g=1..gamma} k^g.
 *   vparent       int32 out [batch][vparent_rows] or NULL: the flattened
 *                 block for spec_mask_build (see below).
 *
 * The top-k tokens of stream j (largest logit first, ties to the lower
 * token id) are the candidates at depth j; every depth-(j-1) node gets all
 * k of them as children.  The tree is flattened breadth-first: node 0 is
 * the root, depth g holds k^g nodes, node off(g) + m has parent
 * off(g-1) + m / k and the (m % k)-th token of stream g.  vparent: row j < n
 * is node j (SPEC_VP_ROOT for the root, else its parent), row
 * n + j*gamma + (s-1) is stream s of node j (parent: node j for s = 1, the
 * row of stream s-1 otherwise), later rows SPEC_VP_PAD.  Entries past n are
 * -1.  A stream row outside [0, n_stream_rows) sets SPEC_DEV_BAD_INDEX.
 */
spec_status_t spec_draft_tree(const spec_draft_desc *desc, const void *stream_logits,
                              const int32_t *stream_row, const int32_t *root_token,
                              int32_t *tokens, int32_t *tree_parent, int32_t *n_nodes,
                              int32_t *vparent, void *stream);

/*
 * spec_prune_tree -- subtree pruning by early-exit probability ([SS]
 * parallel tree pruning).
 *
 *   tokens, tree_parent, n_nodes  the tree (parents precede children, node 0
 *                 the root), e.g. from spec_draft_tree.
 *   early_logits  [batch][max_nodes][vocab]: early-exit logits at each node.
 *   keep_map      int32 out [batch][max_nodes]: a node's index in the pruned
 *                 tree, or -1.
 *   tokens_out, parent_out  int32 out [batch][max_nodes]: the pruned tree,
 *                 survivors in their original order, parents renumbered;
 *                 entries past n_out are -1.  Must not alias the inputs.
 *   n_out         int32 out [batch].
 *   vparent       int32 out [batch][vparent_rows] or NULL: the pruned tree's
 *                 flattened block (layout as in spec_draft_tree).
 *
 * The edge from node p to its child c survives iff
 * exp(z_p[token c] - ln sum exp z_p) >= threshold (fp32), z_p the early-exit
 * logits at p; c survives iff its edge and its parent survive.  The root
 * always survives.  A parent index that does not precede its node sets
 * SPEC_DEV_BAD_TREE (that node is dropped); a token outside the vocabulary
 * sets SPEC_DEV_BAD_INDEX.  Two launches.
 */
spec_status_t spec_prune_tree(const spec_prune_desc *desc, const int32_t *tokens,
                              const int32_t *tree_parent, const int32_t *n_nodes,
                              const void *early_logits, int32_t *keep_map,
                              int32_t *tokens_out, int32_t *parent_out, int32_t *n_out,
                              int32_t *vparent, void *stream);

/*
 * spec_stream_rotate_values -- stream values by rotation ([SS] Eq. 7,
 * V_tn = V_t e^{i eps n}, 0 <= eps <= pi / (2N) with N the maximum sequence
 * length plus the number of streams).
 *
 *   n_nodes  int32 [batch]: T_b, the nodes of request b's block.
 *   vb       [batch][n_kv_heads][n_rows][head_dim] (dtype), in place: the
 *            block values in the SS layout (rows 0..T_b-1 the nodes, row
 *            T_b + j*gamma + (s-1) stream s of node j).
 *
 * For every node j and stream s = 1..gamma, the stream row's value vector
 * becomes node j's value vector with each pair (v[2i], v[2i+1]), read as
 * v[2i] + i v[2i+1], multiplied by e^{i eps s} (fp32, then the storage
 * type).  Node rows and rows past T_b (1 + gamma) are not touched; the
 * block keys are the caller's.  A request with T_b (1 + gamma) > n_rows is
 * skipped and sets SPEC_DEV_BAD_INDEX.  vb must be 16-byte aligned.  Run it
 * before spec_verify_attn.
 */
spec_status_t spec_stream_rotate_values(const spec_rotate_desc *desc, const int32_t *n_nodes,
                                        void *vb, void *stream);

/*
 * spec_future_gather -- the future-token hand-off ([CF] key design 1: the
 * future prediction of the contemplate token attached to the last accepted
 * node goes to the next round's draft).
 *
 *   o          [batch][n_rows][row_elems] (dtype): e.g. spec_verify_attn's
 *              output with row_elems = n_q_heads * head_dim.
 *   last_node  int32 [batch]: from spec_accept.
 *   out        [batch][row_elems] (dtype) out: row row_offset + last_node[b]
 *              of request b (row_offset = T for the ConFu layout, whose
 *              contemplate token of node j is row T + j).
 *
 * Rows must be whole multiples of 16 bytes and o, out 16-byte aligned.  A
 * row outside [0, n_rows) writes zeros and sets SPEC_DEV_BAD_INDEX.
 */
spec_status_t spec_future_gather(int batch, int n_rows, int row_elems, int dtype,
                                 const void *o, const int32_t *last_node, int row_offset,
                                 void *out, void *stream);

/*
 * spec_la_prefill_attn -- the prefill form of Lookahead Attention ([LA]
 * sec. 3.1): the n original and k lookahead positions of each request attend
 * in one pass under the full (n + k) x (n + k) mask M_LA.
 *
 *   q, o   [batch][n + k][n_q_heads][head_dim] (bf16); positions 0..n-1 are
 *          the originals, n..n+k-1 the lookahead tokens.
 *   k, v   [batch][n + k][n_kv_heads][head_dim] (bf16)
 *   lse    out fp32 [batch][n_q_heads][n + k]: natural-log log-sum-exp of
 *          each position's scaled scores.
 *
 * Position i < n sees keys 0..i (causal attention over the originals);
 * position i >= n sees keys 0..n-1 and itself.  For query head h the K/V
 * head is h / (n_q_heads / n_kv_heads); scores are (q . k) * scale.  q, k
 * and v must be 16-byte aligned.  No workspace: each query tile is finished
 * by one CTA.  Returns SPEC_ERR_UNSUPPORTED unless dtype is SPEC_BF16 and
 * head_dim is 128.
 */
spec_status_t spec_la_prefill_attn(const spec_prefill_desc *desc, const void *q,
                                   const void *k, const void *v, void *o,
                                   float *lse, void *stream);

/* Bytes of the fixed scratch array behind spec_verify_attn_noalloc. */
#define SPEC_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * spec_verify_attn_noalloc -- spec_verify_attn for callers that cannot
 * allocate device memory.  The pages have no counterpart: this is a
 * deployment variant of the same computation.
 *
 * Meant for callers that have no workspace to give: for example an engine
 * that reserved all of the GPU's memory for its own KV-cache pool and allows
 * no later allocation, or a plugin hook whose framework owns the memory and
 * forbids allocating while it runs (cudaMalloc may also synchronise the
 * whole device).  Arguments and results are exactly those of
 * spec_verify_attn without `workspace` / `workspace_bytes`; the split
 * partials go to a fixed array of SPEC_NOALLOC_SCRATCH_BYTES (64 MiB) that
 * is part of the library, held on every GPU that loads the library's kernels
 * until the process exits.
 *
 *   - Returns SPEC_ERR_CAPACITY, before launching anything, when the shape
 *     needs more scratch than that (spec_verify_attn_workspace_size tells);
 *     such shapes must use spec_verify_attn.
 *   - Calls no allocating routine (no cudaMalloc, cudaFree or the like).
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; it is looked up again
 *     only when the device's context has changed (e.g. after
 *     cudaDeviceReset).  Under lazy module loading (the CUDA default) that
 *     first lookup loads the library module holding the array, and that
 *     load is when the 64 MiB are taken from the device.  So make the first
 *     call on each device (any arguments: the lookup comes before every
 *     check) before reserving the rest of the device's memory, and before
 *     any stream capture.
 *   - Every call on a device shares the one array, which keeps the previous
 *     call's contents (nothing needs to start at zero: the kernels write each
 *     partial before reading it).  Calls that can overlap on the GPU (other
 *     streams, other host threads) race on the array and must be serialised
 *     by the caller.
 */
spec_status_t spec_verify_attn_noalloc(const spec_attn_desc *attn, const void *q,
                                       const spec_kv_desc *cache, const void *kb,
                                       const void *vb, const void *soft_k,
                                       const void *soft_v, const int32_t *seq_len,
                                       const uint32_t *vis, const uint8_t *row_flags,
                                       void *o, float *lse, void *stream);

/*
 * spec_vocab_reduce -- per logits row ([LA] sec. 2.4 needs the proposal's
 * probability, [SS] hard matching needs the greedy token):
 *
 *   logits    [n_rows][vocab] (dtype)
 *   proposal  int32 [n_rows] or NULL
 *   argmax    out int32 [n_rows]: index of the maximum, lowest on ties; -1
 *             for a row without a logit above -inf (its mask allows nothing)
 *   lse       out fp32 [n_rows]: ln sum_j exp(z_j)
 *   zprop     out fp32 [n_rows] (may be NULL iff proposal is NULL):
 *             z[proposal[i]]; NaN if the proposal is outside [0, vocab).
 */
spec_status_t spec_vocab_reduce(const void *logits, int dtype, int n_rows,
                                int vocab, const int32_t *proposal,
                                int32_t *argmax, float *lse, float *zprop,
                                void *stream);

/*
 * spec_accept -- the acceptance step.
 *
 * If `logits` ([batch][n_judge_rows][vocab]) is non-NULL, spec_vocab_reduce
 * runs first and writes argmax / lse / zprop ([batch][n_judge_rows]); in
 * chain mode the proposal of judge row i is tokens[b][i].  If `logits` is
 * NULL, argmax / lse / zprop are read as inputs.
 *
 *   tokens      int32 [batch][max_nodes]: chain mode: proposal i of request
 *               b; tree mode: draft token of node j (node 0 = root).
 *   tree_parent int32 [batch][max_nodes] (tree mode): parent node, -1 for
 *               the root; parents precede children.  Ignored in chain mode.
 *   row_of      int32 [batch][max_nodes] or NULL (identity): judge row of
 *               node j (tree mode).  Must be NULL in chain mode.
 *   n_nodes     int32 [batch]: proposals (chain: k_b) or tree nodes.
 *
 * Chain mode ([LA] sec. 2.4): L = the largest l <= n_nodes[b] with
 *   zprop_i - lse_i >= ln(tau) for all i < l (fp32, row i judges proposal i).
 *   acc_len = L, path = 0..L-1, next_token = argmax of row L (or -1 when
 *   L == n_nodes[b]), last_node = L - 1.
 * Tree mode ([SS] verification step): from node 0 move to the child whose
 *   token equals the argmax of the current node's judge row (lowest node
 *   index on duplicate sibling tokens) until none matches.
 *   acc_len = nodes on the path including the root (beta + 1),
 *   path = those nodes, next_token = argmax at the last node (the
 *   correction token), last_node = last node on the path.  Tree mode takes
 *   max_nodes <= SPEC_MAX_ROWS (else SPEC_ERR_UNSUPPORTED).
 * A judge row whose argmax is -1 (no token is allowed there) accepts nothing:
 *   the walk ends at its node or proposal, and next_token is -1.
 * path entries past acc_len are set to -1.  A path longer than path_cap or
 * an index out of range stops the walk and sets SPEC_DEV_BAD_INDEX.
 */
spec_status_t spec_accept(const spec_accept_desc *desc, const void *logits,
                          const int32_t *tokens, const int32_t *tree_parent,
                          const int32_t *row_of, const int32_t *n_nodes,
                          int32_t *argmax, float *lse, float *zprop,
                          int32_t *acc_len, int32_t *path, int32_t *next_token,
                          int32_t *last_node, void *stream);

/*
 * kv_commit -- append each request's accepted block rows to the cache and
 * drop the rest ([LA] sec. 3.2, [SS] lazy removal of pruned KV).
 *
 *   kb, vb    [batch][n_kv_heads][n_rows][head_dim], as for spec_verify_attn
 *   path      int32 [batch][path_cap]: block rows to append, in order
 *   acc_len   int32 [batch]: how many entries of path to append
 *   seq_len   int32 [batch], in/out: += appended rows
 *   free_pages int32 [n_free], free_head int32 [1] in/out (paged only;
 *             NULL / 0 for contiguous caches).
 *
 * Row path[b][i] goes to token position seq_len[b] + i.  Paged caches:
 * requests are served in ascending b; each first fills its partly used last
 * page, then takes pages free_pages[*free_head], free_pages[*free_head+1],
 * ... in order, recording them in page_table.
 * A request that would exceed its capacity (max_seq, or max_pages_per_seq)
 * is skipped and sets SPEC_DEV_CAPACITY; if the free list cannot serve all
 * requests, nothing is written and SPEC_DEV_CAPACITY is set.  Out-of-range
 * path entries are not written (SPEC_DEV_BAD_INDEX).
 */
spec_status_t kv_commit(const spec_kv_desc *cache, int batch, int n_rows,
                        const void *kb, const void *vb, int path_cap,
                        const int32_t *path, const int32_t *acc_len,
                        int32_t *seq_len, const int32_t *free_pages,
                        int n_free, int32_t *free_head, void *stream);

/* Bytes of workspace spec_verify_attn_kv8 needs for this shape and cache. */
spec_status_t spec_verify_attn_kv8_workspace_size(const spec_attn_desc *attn,
                                                  const spec_kv8_desc *cache,
                                                  size_t *bytes);

/*
 * spec_verify_attn_kv8 -- spec_verify_attn over a committed prefix held in
 * 8 bits.  The arguments are those of spec_verify_attn with a spec_kv8_desc
 * cache: q, kb, vb, soft_k, soft_v and o keep attn->dtype (the block and the
 * soft prompt are attended as they are, not as the cache would round them),
 * and one row per request (n_rows = 1 with its own vis bit) is the
 * single-token decoding form.
 *
 * Scores, softmax statistics and sums are held in fp32.  For fp32 rows so is
 * everything else.  bf16 rows reach the tensor cores in 8-bit parts: a query,
 * and a key or value of the block or the soft prompt, is held to 2^-17.8 of
 * its row's largest element (values also to no less than 2^-110); a weight
 * times its block's value scale to 2^-9 of itself, or to 2^-35 of the row's
 * largest such product where it is below 2^-26 of it.  lse takes every weight
 * in fp32, but for products below 2^-138 of the largest.
 *
 * A row that sees a block whose key scale is NaN gets o = lse = NaN, one
 * whose value scale is NaN o = NaN.  For bf16 rows a non-finite query gives o
 * = lse = NaN, and so does a visible block or soft-prompt row with a
 * non-finite key; one with a non-finite value gives o = NaN.  For fp32 rows
 * these are what the arithmetic gives: a score of +inf or NaN makes o = lse =
 * NaN, one of -inf has weight 0, a non-finite value reaches its own dimension
 * of o.  Rows that do not see such a place are not affected, and codes in
 * slots past seq_len are never used.
 *
 * A seq_len outside [0, capacity] is clamped and sets SPEC_DEV_SEQ_OVERFLOW;
 * a page id outside [0, n_pages) is not read and sets SPEC_DEV_BAD_PAGE (the
 * affected outputs are then unspecified).  q, kb, vb, soft_k, soft_v and o
 * must be 16-byte aligned.  Calls that can overlap on the GPU (captured ones
 * too) take workspaces of their own.
 */
spec_status_t spec_verify_attn_kv8(const spec_attn_desc *attn, const void *q,
                                   const spec_kv8_desc *cache, const void *kb,
                                   const void *vb, const void *soft_k,
                                   const void *soft_v, const int32_t *seq_len,
                                   const uint32_t *vis, const uint8_t *row_flags,
                                   void *o, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream);

/*
 * kv8_commit -- kv_commit into a cache held in 8 bits: arguments, page
 * allocation, and what is skipped and reported are kv_commit's; `dtype` is
 * the type of kb and vb (16-byte aligned).
 *
 * A block whose first new row is the page's first row takes its scale from
 * the new rows alone.  In a partly used page the scale is the larger of its
 * present one and that of the new rows; where it grows, the rows before the
 * new ones are rounded to it again (nearest even).  Rows of the page behind
 * the last new one are not touched.  An out-of-range path entry leaves its
 * slot as it was (SPEC_DEV_BAD_INDEX).  Two launches.
 */
spec_status_t kv8_commit(const spec_kv8_desc *cache, int dtype, int batch, int n_rows,
                         const void *kb, const void *vb, int path_cap,
                         const int32_t *path, const int32_t *acc_len,
                         int32_t *seq_len, const int32_t *free_pages,
                         int n_free, int32_t *free_head, void *stream);

/*
 * kv8_append -- writes a packed batch of new tokens (a prompt or a chunk of
 * one, of any number of requests) into the slots that spec_page_plan gave
 * them.
 *
 *   k, v      (dtype) token i's row of KV head h begins at element
 *             i * row_stride + h * head_dim; row_stride >= n_kv_heads *
 *             head_dim (each of k and v may lie inside wider rows, such as a
 *             joint projection's output); rows on 16-byte boundaries.
 *   slot_map  int64 [n_tokens]: page * page_size + offset, or < 0 for a
 *             token that is not written (its slot is left as it was).
 *             Tokens of one page follow one another in consecutive slots,
 *             as spec_page_plan numbers them.
 *
 * Blocks take or raise their scales as in kv8_commit (a run of tokens that
 * begins at offset 0 begins the page).  So the token at offset 0 of a page
 * that is new to its request has to be written: a run that begins behind it
 * goes on with the scales that the page's former owner left (a larger scale
 * stays, NaN stays NaN).  A page named by two separate runs of one call is
 * unspecified.  A slot past the cache is skipped and sets SPEC_DEV_BAD_PAGE.
 * page_table, batch and max_pages_per_seq of the descriptor are not used.
 * One launch.
 */
spec_status_t kv8_append(const spec_kv8_desc *cache, int dtype, int n_tokens,
                         const void *k, long long row_stride_k, const void *v,
                         long long row_stride_v, const int64_t *slot_map,
                         void *stream);

/*
 * spec_page_plan -- block tables and slot maps from request lengths: room
 * for n_new[b] more tokens of every request, before they are computed.
 *
 *   seq_len    int32 [batch]: tokens each request holds.
 *   n_new      int32 [batch]: tokens it is about to get (0 = none).
 *   page_table int32 [batch][max_pages_per_seq], in/out: new entries.
 *   free_pages int32 [n_free], free_head int32 [1] in/out, as in kv_commit.
 *   cu_new     int32 [batch + 1] out: first packed token of each request
 *              (the exclusive sums of n_new).
 *   slot_map   int64 [n_slots] out: packed token cu_new[b] + i is token
 *              seq_len[b] + i of request b and gets page * page_size +
 *              offset; -1 behind the last token.
 *   new_len    int32 [batch] out, or NULL: seq_len + n_new.
 *
 * cu_new, slot_map and new_len overlap none of the other arrays, which other
 * threads still read when they are written (else SPEC_ERR_INVALID_ARG).
 *
 * Pages are taken as kv_commit takes them.  A request that would exceed its
 * table is skipped (its slots are -1, new_len = seq_len; SPEC_DEV_CAPACITY),
 * as is one whose seq_len is out of range (SPEC_DEV_SEQ_OVERFLOW) or whose
 * n_new is negative (counted as 0; SPEC_DEV_BAD_INDEX).  If the free list
 * cannot serve all requests no page is taken, every slot is -1 and
 * SPEC_DEV_CAPACITY is set.  A page id outside [0, n_pages) gives slot -1 and
 * SPEC_DEV_BAD_PAGE; more packed tokens than n_slots set SPEC_DEV_BAD_INDEX
 * (pages are taken, the first n_slots slots written).  The new tokens of all
 * requests number at most 2^31 - 1024 (else SPEC_DEV_BAD_INDEX and nothing is
 * planned); seq_len itself is not changed.  One launch, two for more than
 * 4096 slots.
 */
spec_status_t spec_page_plan(int batch, int page_size, int n_pages,
                             int max_pages_per_seq, const int32_t *seq_len,
                             const int32_t *n_new, int32_t *page_table,
                             const int32_t *free_pages, int n_free,
                             int32_t *free_head, int32_t *cu_new,
                             long long n_slots, int64_t *slot_map,
                             int32_t *new_len, void *stream);

/*
 * spec_logits_adjust -- penalties for repeated tokens, biases and grammar
 * masks on the judged rows, ahead of spec_vocab_reduce / spec_accept /
 * spec_accept_soft.
 *
 *   logits, out  [batch][n_judge_rows][vocab] (logit_dtype); out may be
 *                logits itself, and must not overlap it otherwise.
 *   history      int32 [batch][hist_cap]: committed tokens, hist_len int32
 *                [batch] of them, the first n_prompt[b] (n_prompt NULL: 0)
 *                the prompt.  Negative entries are padding.
 *   tokens, tree_parent  int32 [batch][max_nodes]: the draft, as in
 *                spec_accept (a lookahead chain has tree_parent[i] = i - 1).
 *   row_node     int32 [batch][n_judge_rows], or NULL (row j: node j): the
 *                node that the row follows; -1: the row follows the history
 *                alone.
 *   repetition, presence, frequency  fp32 [batch], each NULL for none
 *                (repetition > 0).
 *   bias_ids, bias  int32 / fp32 [batch][n_bias]: added to those tokens;
 *                negative ids are unused entries, equal ids add up.
 *   mask_bits    uint32 [n_masks][ceil(vocab / 32)]: bit v % 32 of word v /
 *                32 allows token v.  row_mask int32 [batch][n_judge_rows]:
 *                the row's mask, negative for none.
 *
 * With n the number of times token v occurs in the history behind the prompt
 * and on the row's path (its node and the node's ancestors), in fp32:
 *   z = logits[v]
 *   if v is in the history (prompt too) or on the path:
 *       z = z > 0 ? z / repetition : z * repetition
 *   z = z - frequency * n - (n > 0 ? presence : 0) + bias[v]
 *   out[v] = allowed ? z, rounded to nearest : -inf
 * (computed as z * factor + sum, the factor and the sum rounded to fp32).
 * A row whose mask allows nothing is -inf throughout (spec_vocab_reduce then
 * names no token for it, and no acceptance takes one there).  A history,
 * draft or bias token >= vocab, a row_node or row_mask out of range, or a
 * hist_len outside [0, hist_cap] (clamped) is left out and sets
 * SPEC_DEV_BAD_INDEX; a parent that does not precede its node ends the path
 * there and sets SPEC_DEV_BAD_TREE (both for draft nodes only where a row's
 * path meets them).  One launch.
 */
spec_status_t spec_logits_adjust(const spec_logits_desc *desc, const void *logits,
                                 void *out, const int32_t *history,
                                 const int32_t *hist_len, const int32_t *n_prompt,
                                 const int32_t *tokens, const int32_t *tree_parent,
                                 const int32_t *row_node, const float *repetition,
                                 const float *presence, const float *frequency,
                                 const int32_t *bias_ids, const float *bias,
                                 const uint32_t *mask_bits, const int32_t *row_mask,
                                 void *stream);

/*
 * spec_rope_freqs -- rotary frequencies, in radians a position, for spec_rope:
 * freqs (HOST, double [rot_dim / 2]), f_i = base^(-2i / rot_dim), and
 *   SPEC_ROPE_PLAIN   f_i;
 *   SPEC_ROPE_LINEAR  f_i / factor (factor > 0);
 *   SPEC_ROPE_RAMP    f_i (w + (1 - w) / factor), w = (t - low) / (high - low)
 *                     within [0, 1], t = trained_len f_i / 2 pi the turns that
 *                     pair i makes over the trained length: fast pairs stay,
 *                     slow ones are stretched (trained_len > 0, low < high).
 * rot_dim is even, <= 256; arguments that a kind does not name are not looked
 * at.  Runs on the host.
 */
spec_status_t spec_rope_freqs(int rot_dim, double base, int scaling, double factor,
                              double trained_len, double low, double high, double *freqs);

/*
 * spec_rope -- rotary positions of queries and keys, ahead of kv_append /
 * kv8_append and the attention calls, which take rows that have them.
 *
 *   freqs     HOST double [rot_dim / 2], radians a position, finite (from
 *             spec_rope_freqs, or any other); read before the call returns.
 *   q, q_out  (dtype) token i's row of query head h begins at element i *
 *             row_stride + h * head_dim; rows of a stride >= n_q_heads *
 *             head_dim (they may lie inside wider ones, such as a joint
 *             projection's output), on 16-byte boundaries.  q_out may be q
 *             itself, with its stride.  k, k_out likewise.
 *   positions int32 [n_tokens]: each row's position; a row with a negative one
 *             is left as it is (its output not written).  Or NULL, and
 *   seq_len   int32 [batch], cu_new int32 [batch + 1], as in spec_page_plan:
 *             packed token cu_new[b] + i has position seq_len[b] + i; rows that
 *             belong to no request are left as they are.
 *
 * Pair i of a head, (x, y), becomes attention * (x cos t - y sin t, y cos t + x
 * sin t), t = position * freqs[i]; elements from rot_dim on are copied.  The
 * angle is held to 2^-24 of a half turn at any position (a frequency to 2^-52
 * of itself), products and sums are fp32, rounded once to dtype.  What a call
 * writes must not meet anything else that it reads or writes.  Of queries and
 * keys this is checked (SPEC_ERR_INVALID_ARG; rows of unlike strides are told
 * apart by the spans of memory that they reach over); positions, seq_len and
 * cu_new are the caller's to keep apart.  A cu_new that decreases or leaves [0,
 * n_tokens] sets SPEC_DEV_BAD_INDEX (which rows are turned is then
 * unspecified), a negative seq_len SPEC_DEV_SEQ_OVERFLOW (its rows are left as
 * they are).  One launch.
 */
spec_status_t spec_rope(const spec_rope_desc *desc, const double *freqs, const void *q,
                        long long row_stride_q, void *q_out, long long row_stride_q_out,
                        const void *k, long long row_stride_k, void *k_out,
                        long long row_stride_k_out, const int32_t *positions, int batch,
                        const int32_t *seq_len, const int32_t *cu_new, void *stream);

/*
 * kv_append -- kv8_append for a cache of rows: writes a packed batch of new
 * tokens into their slots.
 *
 *   k, v      (the cache's dtype) token i's row of KV head h begins at element
 *             i * row_stride + h * head_dim; row_stride >= n_kv_heads *
 *             head_dim; rows on 16-byte boundaries, as is the cache.
 *   slot_map  int64 [n_tokens]: page * page_size + offset (from
 *             spec_page_plan), or request * max_seq + token for a contiguous
 *             cache; < 0 for a token that is not written.
 *
 * A slot past the cache is skipped and sets SPEC_DEV_BAD_PAGE; of tokens with
 * the same slot, which one is kept is unspecified, element by element.  k and
 * v must not overlap the cache.  page_table and max_pages_per_seq of the
 * descriptor are not used.  One launch.
 */
spec_status_t kv_append(const spec_kv_desc *cache, int n_tokens, const void *k,
                        long long row_stride_k, const void *v, long long row_stride_v,
                        const int64_t *slot_map, void *stream);

/* Bytes of workspace spec_chunk_attn needs for this shape and cache; they do
 * not depend on n_tokens or on the cache's size. */
spec_status_t spec_chunk_attn_workspace_size(const spec_chunk_desc *desc,
                                             const spec_kv_desc *cache, size_t *bytes);

/*
 * spec_chunk_attn -- attention of new tokens that the cache already holds
 * (kv_append): each sees its request's tokens up to itself.  Prompts, chunks of
 * prompts and single tokens, in one call.
 *
 *   q         (dtype) token i's row of query head h begins at element i *
 *             row_stride_q + h * head_dim; row_stride_q >= n_q_heads *
 *             head_dim; rows on 16-byte boundaries.
 *   cache     of the same dtype, paged or contiguous.
 *   seq_len   int32 [batch]: tokens each request held before the new ones.
 *   cu_new    int32 [batch + 1]: first packed token of each request, as
 *             spec_page_plan writes it: request b's new tokens are rows
 *             cu_new[b] .. cu_new[b + 1] - 1 (none, if equal).
 *   o         out (dtype) [n_tokens][n_q_heads][head_dim], 16-byte aligned; it
 *             must not overlap q.
 *   lse       out fp32 [n_tokens][n_q_heads]: natural-log log-sum-exp of the
 *             row's scaled scores.
 *   workspace device scratch of >= spec_chunk_attn_workspace_size bytes,
 *             256-byte aligned; its contents on entry are ignored.
 *
 * New token i of request b sees cache tokens 0 .. seq_len[b] + i; for query
 * head h the K/V head is h / (n_q_heads / n_kv_heads); scores are (q . k) *
 * scale.  Scores, softmax statistics and sums are held in fp32; for bf16 rows a
 * weight is rounded to bf16 (half a step: 2^-8 of itself) before its product
 * with the value.  Rows of o and lse that belong to no request are left as they were.
 *
 * A row that sees a non-finite key or has a non-finite query gets o = lse =
 * NaN where a score is +inf or NaN (-inf has weight 0; a row with no other
 * score gets o = 0, lse = -inf); one that sees a non-finite value gets o
 * non-finite in the value's dimension, and may in all.  Rows that do not see
 * such a place are not affected, and slots past a request's last new token are
 * never used.
 *
 * A request whose cu_new decreases or leaves [0, n_tokens] is skipped and sets
 * SPEC_DEV_BAD_INDEX, one whose seq_len is negative or whose last new token
 * lies past the capacity SPEC_DEV_SEQ_OVERFLOW (their rows are left as they
 * were); a page id outside [0, n_pages) is not read and sets SPEC_DEV_BAD_PAGE
 * (the affected outputs are then unspecified).  Calls that can overlap on the
 * GPU (captured ones too) take workspaces of their own.  Two launches.
 */
spec_status_t spec_chunk_attn(const spec_chunk_desc *desc, const void *q,
                              long long row_stride_q, const spec_kv_desc *cache,
                              const int32_t *seq_len, const int32_t *cu_new, void *o,
                              float *lse, void *workspace, size_t workspace_bytes,
                              void *stream);

/* Bytes of workspace spec_chunk_attn_kv8 needs for this shape and cache. */
spec_status_t spec_chunk_attn_kv8_workspace_size(const spec_chunk_desc *desc,
                                                 const spec_kv8_desc *cache, size_t *bytes);

/*
 * spec_chunk_attn_kv8 -- spec_chunk_attn over a cache held in 8 bits
 * (kv8_append): the new tokens too are attended as the cache holds them.  q and
 * o have desc->dtype.  For bf16 rows an element counts as code * scale rounded
 * to bf16, which is exact for the powers of two that the writers give.  A row
 * that sees a block whose key scale is NaN gets o = lse = NaN, one whose value
 * scale is NaN o = NaN.  (A batch of single tokens alone goes faster through
 * spec_verify_attn_kv8 with one row, before its commit.)
 */
spec_status_t spec_chunk_attn_kv8(const spec_chunk_desc *desc, const void *q,
                                  long long row_stride_q, const spec_kv8_desc *cache,
                                  const int32_t *seq_len, const int32_t *cu_new, void *o,
                                  float *lse, void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * spec_set_wait_limit -- limit, in SM clock cycles, of the internal pipeline
 * waits of the kernels launched from now on (verify and chunk attention over
 * either cache, prefill attention, and the bulk row stream of the vocabulary
 * reduction), process-wide.  The pages have no counterpart: this is the
 * library's guard against a hang.  A wait that runs out sets
 * SPEC_DEV_TIMEOUT; the kernel then stops issuing work, waits (with the
 * default limit) for its own copies and tensor-core operations, frees its
 * tensor memory and returns, and the context stays usable.  cycles < 0
 * restores the default (2e9 cycles, about one second); 0 makes any wait
 * whose condition is not already met fail at once, which is how the tests
 * exercise this path.  Returns the previous limit.  Not for use while other
 * threads launch work of this library.
 */
long long spec_set_wait_limit(long long cycles);

/*
 * spec_get_status -- synchronise `stream`, then read and clear the current
 * device's status word.  *out receives the SPEC_DEV_* bits (0 = none).
 * Returns SPEC_OK if no bit was set, SPEC_ERR_DEVICE otherwise.
 */
spec_status_t spec_get_status(void *stream, int32_t *out);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */
