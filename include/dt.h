/*
 * dt.h -- C ABI of libdt.so: draft-tree construction on AMD Instinct MI355X
 * (gfx950) for diffusion-style speculative decoding.
 *
 * The operation (one call = one batch of B independent requests):
 *
 *   d per-position draft logit rows  --->  pruned draft token tree + mask
 *
 * as the pages define it:
 *   - DART (arXiv 2601.19278), Fig. 3 caption ("Continuity-Aware Tree
 *     Pruning"): the drafter's d logits come from one forward with d-1 mask
 *     tokens ("shifted logits prediction"), the first from the last prefix
 *     position; candidate tokens of each depth are taken from that
 *     position's own logit; an N-gram model keeps only expansions that stay
 *     continuous; the pruned tree is verified with tree attention.
 *   - DARTree (llmdb page, "Tree Construction" and its P_AR equation;
 *     scholarbro abstract): a fixed-width candidate tree of depth K and
 *     width W, every candidate of a depth scored in one batch with a
 *     path-conditioned score, the top-W kept across the whole frontier after
 *     each depth, then best-first pruning selects the verification tree.
 *
 * Concretely, for request b:
 *   1. lse_i = log sum_v exp(logits[b][i][v]) and T_i = the k largest
 *      logits of row i, ordered (value desc, token id asc), i = 0..d-1.
 *   2. The root is the last committed token ctx[b][1] (context ctx[b][0],
 *      ctx[b][1]).  For depth t = 1..d every frontier node p of depth t-1
 *      is paired with every child c in T_{t-1}.  The pair is kept iff
 *      logits[b][t-1][c] > -inf and the N-gram admits c after p's context
 *      (bigram: p's token; trigram: (p's parent's token, p's token), the
 *      root using ctx[b][0]); an admitted entry needs logp > min_logp
 *      (strict), and min_logp = -INFINITY tests membership only.
 *   3. Each kept child gets Rk = (Rk_p + x) + g and S = (S_p + (x - lse)) + g
 *      in double precision, x = its logit, g = E[tok_p] . F[c] in DARTREE
 *      mode (the low-rank parent-conditioned term), g = 0 in DART mode.
 *      The frontier of depth t is the first min(W, #kept) candidates in the
 *      order (Rk desc, token asc, parent's frontier rank asc).  Growth stops
 *      at the first empty frontier.
 *   4. If the candidate tree has more than `budget` nodes, best-first
 *      selection repeatedly takes the available node (parent already taken,
 *      or depth 1) with the best (S desc, depth asc, BFS index asc) until
 *      `budget` nodes are taken.
 *   5. Output in BFS order (depth asc, then frontier rank).
 *
 * DARTREE_FULL mode (DARTree page, "Tree Construction": the drafter proposes
 * W candidate tokens per frontier node): instead of the position's shared
 * top-k, every frontier node p proposes its own W best tokens of the whole
 * vocabulary under its parent-conditioned distribution x[v] + E[tok_p].F[v]
 * (order: Rk desc, token asc), and the frontier is the top-W of all
 * proposals, ranked as in step 3.  This equals the top-W over every
 * (node, token) pair.  k is not used for proposals; the N-gram table must
 * be of kind NONE; W <= 16 and R in {16, 32, 64}.  Keys are exact fp64 (the
 * dense product runs on bf16 matrix cores only to discard tokens that
 * provably cannot be selected).  Best-first selection is replayed literally
 * (g may be positive, so S can rise along a path).
 *
 * Output tree (caller-allocated device memory, n_max = budget,
 * mask_words = ceil(budget / 32)):
 *   n_nodes [B]                     int32, number of draft nodes (0..budget)
 *   tokens  [B][n_max]              int32, token id, -1 in padding rows
 *   parents [B][n_max]              int32, parent node index, -1 = the root
 *   depths  [B][n_max]              int32, 1..d, 0 in padding rows
 *   scores  [B][n_max]              float, S rounded to fp32, -inf padding
 *   mask    [B][n_max][mask_words]  uint32, row i has bit j (word j >> 5,
 *                                   bit j & 31, LSB first) set iff node j
 *                                   is node i or one of its ancestors; the
 *                                   root and prefix are implicit; padding
 *                                   rows are zero.
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers unless stated otherwise; the
 *     structs themselves are host memory read during the call only.
 *   - The caller owns every buffer, including the workspace.  The library
 *     never allocates, frees or synchronises, and keeps no state between
 *     calls (dt_build_tree_noalloc aside: it holds its scratch array per
 *     GPU).  Work is enqueued on `stream` (a hipStream_t; NULL = the null
 *     stream) and the call returns without waiting.  Calls on different
 *     streams need different workspaces.
 *   - Arguments are validated on the host before anything is enqueued; on
 *     an error nothing is enqueued and no output is touched.  A launch
 *     failure returns DT_ERR_HIP.  Faults during execution surface at the
 *     caller's next synchronisation of `stream`.
 *   - Logits are finite or -inf.  NaN or +inf logits give unspecified
 *     (but memory-safe) results.  ctx ids must lie in [0, V); other values
 *     admit no children under bigram tables and add no parent term.  Table
 *     contents (row_ptr ranges, successor ids) are trusted as given.
 *   - Limits: B >= 0; 1 <= d <= 32; 1 <= k <= 32 and k <= V; 1 <= W <= 64;
 *     W * k <= 1024; 1 <= budget <= 1024; 1 <= V < 2^26; the logits
 *     pointer 16-byte aligned; and the tree kernel's shared-memory plan
 *     (which grows with d, k, W, the N-gram kind and the mode) must fit in
 *     the 160 KiB of LDS a gfx950 workgroup may use, else
 *     DT_ERR_UNSUPPORTED.  DARTREE mode needs E and F 16-byte
 *     aligned with R a multiple of 4, 4 <= R <= 256.  A trigram table's
 *     keys array must be 16-byte aligned.
 */
#ifndef DT_H
#define DT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dt_status {
    DT_OK = 0,
    DT_ERR_INVALID_ARG = 1,   /* a null pointer, a value out of range, a misaligned buffer */
    DT_ERR_UNSUPPORTED = 2,   /* valid but outside the library's limits (see above) */
    DT_ERR_WORKSPACE = 3,     /* workspace missing or smaller than dt_workspace_size() */
    DT_ERR_HIP = 4            /* the HIP runtime refused a launch */
} dt_status;

/* F16 is a type of the verification pass's heads (dt_kv_cache) only. */
typedef enum dt_dtype { DT_DTYPE_F32 = 0, DT_DTYPE_BF16 = 1, DT_DTYPE_F16 = 2 } dt_dtype;

typedef enum dt_mode {
    DT_MODE_DART = 0,      /* score = cumulative draft log-probability */
    DT_MODE_DARTREE = 1,   /* + parent-conditioned term E[parent] . F[child] */
    DT_MODE_DARTREE_FULL = 2  /* DARTREE with per-node proposals over the whole vocabulary */
} dt_mode;

typedef enum dt_ngram_kind {
    DT_NGRAM_NONE = 0,          /* every expansion is continuous */
    DT_NGRAM_DENSE_BIGRAM = 1,  /* logp[V][V] indexed [parent token][child] */
    DT_NGRAM_CSR_BIGRAM = 2,    /* successors of a token, ascending ids */
    DT_NGRAM_HASH_TRIGRAM = 3   /* open-addressing table keyed by (t_-2, t_-1) */
} dt_ngram_kind;

/* N-gram continuity table (device arrays; unused fields may be NULL).
 *  dense:  dense_logp[V][V] float.
 *  CSR:    row_ptr[V+1] int32, col[nnz] int32 ascending within a row,
 *          csr_logp[nnz] float (may be NULL when min_logp = -INFINITY);
 *          col and csr_logp may be NULL when nnz = 0 (every row empty).
 *  hash:   keys[cap] uint64 with key = (uint64)t_-2 << 32 | (uint32)t_-1 and
 *          0xFFFFFFFFFFFFFFFF marking a free slot; a key lives in the first
 *          free slot at or after splitmix64(key) & (cap - 1) (the SplitMix64
 *          output function of Steele, Lea and Flood), probing linearly with
 *          wrap-around; succ[cap][S] int32 successor ids, -1 = none;
 *          hash_logp[cap][S] float (may be NULL when min_logp = -INFINITY).
 *          cap is a power of two with at least one free slot, 1 <= S <= 64. */
typedef struct dt_ngram_table {
    int32_t kind;              /* dt_ngram_kind */
    float min_logp;            /* keep iff logp > min_logp; -INFINITY = membership */
    const float* dense_logp;
    const int32_t* row_ptr;
    const int32_t* col;
    const float* csr_logp;
    int64_t nnz;
    const uint64_t* keys;
    const int32_t* succ;
    const float* hash_logp;
    int64_t cap;
    int32_t S;
} dt_ngram_table;

typedef struct dt_params {
    int32_t B;                 /* requests in the batch */
    int32_t V;                 /* vocabulary size (row length) */
    int32_t d;                 /* draft positions = tree depth (K in DARTree) */
    int32_t k;                 /* candidates taken from each position's logit */
    int32_t W;                 /* frontier width kept per depth */
    int32_t budget;            /* verification budget = n_max rows of the output */
    int32_t dtype;             /* dt_dtype of the logits */
    int32_t mode;              /* dt_mode */
    const int32_t* ctx;        /* [B][2] device: (t_-2, t_-1), t_-1 is the root */
    const float* E;            /* [V][R] device, DARTREE only (else may be NULL) */
    const float* F;            /* [V][R] device, DARTREE only */
    int32_t R;                 /* rank of E and F */
    int32_t sweep_chunks;      /* 0 = automatic; else split each row into this many chunks */
    void* workspace;           /* device scratch of at least dt_workspace_size() bytes */
    size_t workspace_bytes;
    void* stream;              /* hipStream_t */
    void* prof_event_start;    /* optional hipEvent_t recorded on `stream` right before */
    void* prof_event_stop;     /* ... and right after the vocabulary-sweep kernel */
} dt_params;

typedef struct dt_tree_out {
    int32_t* n_nodes;          /* [B] */
    int32_t* tokens;           /* [B][budget] */
    int32_t* parents;          /* [B][budget] */
    int32_t* depths;           /* [B][budget] */
    float* scores;             /* [B][budget] */
    uint32_t* mask;            /* [B][budget][ceil(budget/32)] */
} dt_tree_out;

/* The whole path (steps 1-5 above) for B requests.
 * logits: device [B][d][V] of dtype, rows contiguous, 16-byte aligned.
 * Calls on different streams overlap: a sweep of 257 to 512 workgroups
 * (one to two per compute unit, e.g. B=64 at V=151936, d=8) holds 56 KiB
 * of LDS per workgroup when the call's
 * prep and tree workgroups still fit beside two of them, so two calls'
 * sweeps take turns instead of sharing the memory bandwidth, and one call's
 * (latency-bound, raised-priority) prep and tree kernels run beside the next
 * call's sweep. */
dt_status dt_build_tree(const void* logits, const dt_ngram_table* ngram,
                        const dt_params* params, const dt_tree_out* out);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * operation as dt_build_tree, same arguments except that params->workspace
 * and params->workspace_bytes are ignored.  The workspace is instead a
 * scratch array of DT_NOALLOC_SCRATCH_BYTES bytes inside the library, one
 * copy per GPU (the device of params->stream, or the current device for
 * the null stream), held from the first call on that GPU until the process
 * ends.  The call allocates nothing and calls no allocating routine; its
 * first call on a GPU looks the array's address up (hipGetSymbolAddress).
 * Every call on one GPU shares that GPU's array: calls whose executions
 * overlap on the same GPU (different streams, or different host threads)
 * race and give undefined trees, so serialise them (one stream, or events).
 * Errors: as dt_build_tree, and DT_ERR_WORKSPACE when dt_workspace_size()
 * of the parameters exceeds DT_NOALLOC_SCRATCH_BYTES; DT_ERR_HIP when the
 * device or the array's address cannot be obtained. */
#define DT_NOALLOC_SCRATCH_BYTES (32u << 20)
dt_status dt_build_tree_noalloc(const void* logits, const dt_ngram_table* ngram,
                                const dt_params* params, const dt_tree_out* out);

/* Bytes of workspace dt_build_tree / dt_position_topk need for these
 * parameters (depends on B, V, d, k, mode, dtype and sweep_chunks only, and
 * on W and R in DARTREE_FULL mode; the N-gram area is sized for the largest
 * table kind); 0 if the parameters are invalid.  The workspace holds the
 * sweep's per-chunk partials and the per-row normalisers, top-k lists,
 * continuity masks (and DARTree terms) the tree step reads; in DARTREE_FULL
 * mode also the frontier, the candidate tree, the column norms and a bf16
 * copy of F (V * R * 2 bytes) for the matrix-core screen, and every
 * vocabulary chunk's top-W.  Its contents are meaningless between calls. */
size_t dt_workspace_size(const dt_params* params);

/* Static, human-readable name of a status code. */
const char* dt_status_string(dt_status s);

/* Step 1 alone (DART Fig. 3: each position's own logit proposes the tokens
 * of its depth): per row (b, i) the log-softmax normaliser and the top-k.
 * lse: device [B][d] double; topk_tok: device [B][d][k] int32 in order
 * (value desc, id asc); topk_val: device [B][d][k] float (the logits).
 * Uses B, V, d, k, dtype, sweep_chunks, workspace and stream of params. */
dt_status dt_position_topk(const void* logits, const dt_params* params,
                           double* lse, int32_t* topk_tok, float* topk_val);

/* The step after verification: keep a trigram table current with the tokens
 * the target accepted (the N-gram model that keeps DART's expansions
 * continuous, DART Fig. 3).  For request b the stream ctx[b][0], ctx[b][1],
 * tokens[b][0 .. lengths[b]-1] contributes, for every accepted token s_i,
 * the trigram (s_{i-2}, s_{i-1}) -> s_i:
 *   - a missing key takes the first free slot of its probe sequence (the
 *     layout dt_build_tree reads: first free slot at or after
 *     splitmix64(key) & (cap - 1), linear probing); its row starts empty,
 *     so rows of free slots must hold -1 in every entry;
 *   - a missing successor takes the first -1 entry of the key's row and,
 *     when table->hash_logp is not NULL, the log-probability new_logp;
 *   - a trigram whose row is full, whose probe sequence has no free slot, or
 *     whose key equals the free-slot marker is dropped.
 * The trigrams of one call are applied concurrently: the resulting keys and
 * successor sets are those of applying them one by one in any order as long
 * as no row fills up and the table keeps free slots; the slot a new key lands
 * in, and which successors an overflowing row keeps, may vary between runs.
 * table: kind DT_NGRAM_HASH_TRIGRAM; its keys, succ and (if not NULL)
 *   hash_logp arrays are written in place (keys 8-byte, succ and hash_logp
 *   4-byte aligned).
 * ctx: device [B][2] int32; tokens: device [B][L] int32; lengths: device [B]
 *   int32 (entries past lengths[b], or past L, are ignored).
 * counts: device int32[3] or NULL; atomically incremented by keys added,
 *   successors added and trigrams dropped (the caller zeroes it).
 * Must not run concurrently with a dt_build_tree reading the same table.
 * Errors: DT_ERR_INVALID_ARG for a non-trigram table, null or misaligned
 *   arrays, cap not a power of two >= 2, B or L < 0 or a NaN new_logp;
 *   DT_ERR_UNSUPPORTED for S outside 1..64; DT_ERR_HIP if the launch fails. */
dt_status dt_ngram_update(const dt_ngram_table* table, const int32_t* ctx, const int32_t* tokens,
                          const int32_t* lengths, int32_t B, int32_t L, float new_logp,
                          int32_t* counts, void* stream);

/* How many nodes of each built tree to send to verification (LibraSpec,
 * scholarbro listing abstract: the speculative length is chosen for expected
 * speedup and extended only while the acceptance gain outweighs the added
 * verification cost, judged from the drafter's confidence).  Candidate
 * verification sets are the prefixes of the tree's best-first order (a node
 * is available once its parent is taken; the best available by score desc,
 * depth asc, index asc is taken next; every prefix is closed under parents).
 * Node n of that order has confidence c_n = exp(score_n); with
 * A(n) = 1 + sum_{i<n} c_i expected tokens per round and
 * T(n) = cost_fixed + cost_per_token * n its cost (any time unit), node n is
 * added while c_n * T(n) > cost_per_token * A(n), i.e. while A/T strictly
 * grows; n_verify[b] is where that stops (0..n_nodes).  rank[b][i] receives
 * node i's best-first position, -1 for rows i >= n_nodes: verify the nodes
 * with rank < n_verify.
 * tree: the arrays dt_build_tree wrote ([B][budget]; tokens and mask unused).
 * n_verify: device [B] int32; rank: device [B][budget] int32.
 * Errors: DT_ERR_INVALID_ARG for null arrays, B < 0, budget < 1, or a cost
 *   that is not finite, cost_fixed <= 0 or cost_per_token < 0;
 *   DT_ERR_UNSUPPORTED for budget > 1024; DT_ERR_HIP if the launch fails. */
dt_status dt_verify_length(const dt_tree_out* tree, int32_t B, int32_t budget, double cost_fixed,
                           double cost_per_token, int32_t* n_verify, int32_t* rank, void* stream);

/* ------------------------------------------------------------------------
 * The target's verification pass over the built trees: the operators between
 * a tree and the accepted tokens.  With the model's own products between
 * them, one layer is dt_kv_append, then dt_tree_attention; after the last
 * layer dt_process_logits, dt_position_topk with k = 1 (the target's choice
 * for every row) and dt_commit_path, whose outputs dt_ngram_update takes.
 *
 * A batch's new tokens are a CHUNK of `lead + n_max` rows a request: `lead`
 * committed tokens whose keys and values are not in the cache yet (the last
 * of them is the tree's root), then up to n_max tree nodes in the order of
 * dt_build_tree, of which the first n_nodes[b] count.  lead = 1, n_max = 0
 * is a step of plain decoding; lead = 0 with mask = NULL is a (ragged) piece
 * of a prompt.  Row r of request b is position and cache slot
 * ctx_len[b] + r; a node's POSITION is that of the root plus its depth.
 * Rows at or behind lead + n_nodes[b] are neither read nor written, in any
 * buffer.
 *
 * These entry points launch on the device of `stream` (the current device
 * for the null stream), whichever device is current.
 * ------------------------------------------------------------------------ */

/* A paged cache of keys and values.  Element d of head h of the token in
 * slot s of request b in layer l lies at
 *   k + l * layer_stride + page * page_stride + (s % page_size) * slot_stride
 *     + h * head_stride + d,      page = page_table[b * max_pages + s / page_size]
 * and likewise for v.  Strides count elements and are multiples of 8 and not
 * negative (the stride of an axis of length one is not read); k and v are
 * 16-byte aligned.  Calls that write (dt_kv_append, dt_commit_path) need every
 * element at a place of its own, and refuse strides below D.  Tokens whose page lies outside [0, num_pages), or whose
 * slot lies behind the table (max_pages * page_size), are dropped on writing
 * and unseen on reading.  Two tokens written in one call must not share a
 * slot; pages that are only read may be shared by requests. */
typedef struct dt_kv_cache {
    void* k;
    void* v;
    const int32_t* page_table; /* device [B][max_pages] */
    int64_t layer_stride;
    int64_t page_stride;
    int64_t slot_stride;
    int64_t head_stride;
    int32_t layers;            /* >= 1 */
    int32_t num_pages;         /* >= 1 */
    int32_t page_size;         /* >= 1; max_pages * page_size <= 2^30 */
    int32_t max_pages;         /* >= 1 */
    int32_t Hkv;               /* key heads, 1 <= Hkv <= 4096 */
    int32_t D;                 /* elements of a head: 64, 128 or 256 */
    int32_t dtype;             /* DT_DTYPE_BF16 or DT_DTYPE_F16 */
} dt_kv_cache;

/* The new tokens of a batch (see above); every array is on the device. */
typedef struct dt_chunk {
    int32_t B;                 /* requests, 0 <= B <= 65535 */
    int32_t lead;              /* >= 0 */
    int32_t n_max;             /* >= 0; 1 <= lead + n_max <= 65536, B * (lead + n_max) <= 2^24 */
    const int32_t* ctx_len;    /* [B] tokens in the cache; < 0: the request has no rows */
    const int32_t* n_nodes;    /* [B], clamped to 0..n_max; NULL = n_max for all */
    const uint32_t* mask;      /* [B][n_max][ceil(n_max/32)] as dt_tree_out; NULL = every row sees
                                  all slots up to its own */
    const int32_t* depths;     /* [B][n_max] as dt_tree_out; NULL = a row's position is its slot */
} dt_chunk;

/* Frequencies of the rotary positions, on the HOST: freqs[i], 0 <= i <
 * rot_dim / 2, is the angle in radians by which pair i turns from one
 * position to the next, and *scale the factor of dt_append_params.rot_scale.
 *   NONE        f_i = base^(-2i / rot_dim), scale 1;
 *   LINEAR      f_i / factor, scale 1;
 *   WAVELENGTH  with l = 2 pi / f_i: f_i / factor where l > original / low,
 *               f_i where l < original / high, else (1 - s) f_i / factor +
 *               s f_i, s = (original / l - low) / (high - low); scale 1;
 *   YARN        i_low = floor(c(high)), i_high = ceil(c(low)), both clamped
 *               to 0..rot_dim - 1, with c(n) = rot_dim
 *               ln(original / (2 pi n)) / (2 ln base); s = 1 - clamp((i -
 *               i_low) / (i_high - i_low), 0, 1) (a difference of zero counts
 *               as 0.001) in the blend above; scale 0.1 ln(factor) + 1 (1 for
 *               factor <= 1).
 * Errors: DT_ERR_INVALID_ARG for null pointers, rot_dim odd or < 2, base not
 *   finite or <= 1, factor not finite or <= 0, an unknown kind; for WAVELENGTH
 *   and YARN also unless 0 < low < high and original > 0, all finite. */
typedef enum dt_rope_kind {
    DT_ROPE_NONE = 0,
    DT_ROPE_LINEAR = 1,
    DT_ROPE_WAVELENGTH = 2,
    DT_ROPE_YARN = 3
} dt_rope_kind;
dt_status dt_rope_frequencies(int32_t kind, int32_t rot_dim, double base, double factor, double low,
                              double high, double original, double* freqs, float* scale);

typedef struct dt_append_params {
    const void* q;             /* [B][lead + n_max] rows of Hq heads of D, or NULL (keys and values only) */
    const void* k;             /* ... rows of Hkv heads */
    const void* v;
    void* q_out;               /* as q; may be q itself with the same row stride; NULL iff q is */
    int64_t q_stride;          /* elements from row to row; the heads of a row are contiguous */
    int64_t k_stride;
    int64_t v_stride;
    int64_t q_out_stride;
    int32_t Hq;                /* query heads, 1..4096 (not read when q is NULL) */
    const void* q_norm;        /* [D] weights of dtype, or NULL = no norm */
    const void* k_norm;
    float eps;                 /* >= 0 */
    const double* freqs;       /* device [rot_dim / 2] radians a position */
    int32_t rot_dim;           /* the first rot_dim elements of a head turn: 0..D, a multiple of 16 */
    int32_t interleaved;       /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1) */
    float rot_scale;           /* factor of the turned elements (1 without scaling) */
    int32_t layer;             /* layer of the cache, 0 <= layer < layers */
    void* stream;
} dt_append_params;

/* The new tokens' queries, keys and values on their way from the projection:
 * for every row, y = x * rsqrt(mean(x^2) + eps) * w over each head of q (k)
 * if q_norm (k_norm) is given, then pair i of the first rot_dim elements
 * turned by position * freqs[i]: (a, b) -> rot_scale * (a cos - b sin,
 * a sin + b cos); q goes to q_out, k and v (as it is) to their cache slots.
 * All in fp32 (the angle in fp64, reduced before the sine), rounded once.
 * Pointers 16-byte aligned, strides multiples of 8 and, in buffers of more
 * than one row, at least a row's heads; eps finite.
 * Errors: DT_ERR_INVALID_ARG, DT_ERR_UNSUPPORTED (a limit above), DT_ERR_HIP. */
dt_status dt_kv_append(const dt_kv_cache* kv, const dt_chunk* chunk, const dt_append_params* p);

typedef struct dt_attention_params {
    const void* q;             /* [B][lead + n_max] rows of Hq heads of D */
    void* out;                 /* as q, of the cache's dtype */
    int64_t q_stride;          /* elements from row to row; the heads of a row are contiguous */
    int64_t out_stride;
    int32_t Hq;                /* query heads, a multiple of Hkv, 1..4096; head h reads key head h / (Hq / Hkv) */
    float scale;               /* > 0, finite */
    float* lse;                /* [B][lead + n_max][Hq] or NULL: log of the sum of exp(scale * q . k) */
    int32_t layer;
    void* workspace;           /* 16-byte aligned device scratch of dt_attention_workspace() bytes */
    size_t workspace_bytes;
    void* stream;
} dt_attention_params;

/* Attention of the chunk's rows over the paged cache, which already holds the
 * chunk's own keys and values (dt_kv_append):
 *   out = sum_j softmax_j(scale * q . k_j) v_j   over the slots j a row sees:
 *   - row r < lead, or any row when mask is NULL: j <= ctx_len + r;
 *   - node i otherwise: j < ctx_len + lead, and ctx_len + lead + i' for every
 *     i' < n_nodes whose bit is set in mask row i.
 * Scores, the softmax and the sums are fp32; the weights are rounded to the
 * cache's type for the second product, the result once.  A row that sees
 * nothing gives zeros (lse -inf).  Whatever lies in slots that a row does not
 * see, infinities and NaN included, does not reach it; an infinity in v that it
 * sees reaches it times its weight, that is as NaN where the weight has become 0
 * in the cache's type (less than about 2^-31 of the largest in f16).  Finite scores beyond
 * 2^27 in magnitude, whose last bits are many units, give unspecified (but
 * memory-safe) results.
 * The work is split by the lengths on the device, in time that grows with the
 * square of B: meant for some hundred requests (65535 take over a second).
 * q may not overlap out.  Pointers 16-byte aligned (lse 4), strides multiples
 * of 8 and at least Hq * D.
 * Errors: DT_ERR_INVALID_ARG, DT_ERR_UNSUPPORTED (a limit above, or
 *   B * (lead + n_max) * Hq >= 2^31), DT_ERR_WORKSPACE, DT_ERR_HIP. */
dt_status dt_tree_attention(const dt_kv_cache* kv, const dt_chunk* chunk, const dt_attention_params* p);

/* Bytes of workspace dt_tree_attention needs (depends on kv's Hkv and D, on
 * the chunk's B, lead and n_max and on Hq only); 0 if a call would be
 * refused for these.  Its contents are meaningless between calls. */
size_t dt_attention_workspace(const dt_kv_cache* kv, const dt_chunk* chunk, int32_t Hq);

typedef struct dt_logits_params {
    const void* logits;        /* device [B][lead + n_max][V] of dtype, 16-byte aligned */
    void* out;                 /* as logits; may be logits itself */
    int32_t B;                 /* 0 <= B <= 65535 */
    int32_t lead;              /* >= 0 */
    int32_t n_max;             /* >= 0; 1 <= lead + n_max <= 65536 */
    int32_t V;                 /* 1 <= V < 2^26 */
    int32_t dtype;             /* DT_DTYPE_F32 or DT_DTYPE_BF16 */
    const int32_t* n_nodes;    /* [B], clamped to 0..n_max; NULL = n_max */
    const int32_t* history;    /* [B][history_max] token ids, oldest first; NULL = none */
    int32_t history_max;       /* >= 0 */
    const int32_t* history_len;/* [B], clamped to 0..history_max; needed with history */
    const int32_t* prompt_len; /* [B], clamped to 0..history_len; NULL = 0: the first of a
                                  request's history are its prompt, the rest were generated */
    const int32_t* node_tokens;/* [B][n_max] tokens of the tree's nodes (n_max <= 1024), or NULL */
    const uint32_t* node_mask; /* [B][n_max][ceil(n_max/32)] as dt_tree_out; needed with node_tokens */
    const float* repetition;   /* [B] > 0, or NULL = 1 */
    const float* frequency;    /* [B] or NULL = 0 */
    const float* presence;     /* [B] or NULL = 0 */
    const int32_t* bias_ids;   /* [B][n_bias] or NULL */
    const float* bias;         /* [B][n_bias]; needed with bias_ids */
    int32_t n_bias;            /* 0..65534 */
    const uint32_t* allow;     /* [allow_rows][ceil(V/32)] bits of allowed tokens, LSB first, or NULL */
    const int32_t* allow_index;/* [B][lead + n_max] row of allow; outside 0..allow_rows-1: unmasked.
                                  NULL = row number b * (lead + n_max) + r */
    int32_t allow_rows;        /* >= 1 with allow */
    void* stream;
} dt_logits_params;

/* Logits as the sampler should see them; rows are those of a chunk (draft
 * positions: lead = d, n_max = 0).  Token v of row r of request b, with
 *   c    = how often v occurs among the generated tokens of the history and,
 *          for the row of node i, among the nodes whose bit is set in
 *          node_mask row i (its path; nodes at or behind n_nodes do not
 *          count),
 *   seen = c > 0, or v occurs in the prompt:
 *   x = seen ? (x > 0 ? x / repetition : x * repetition) : x
 *   x = x - (frequency * c + presence * [c > 0])
 *   x = x + bias of v (an id listed more than once takes its last entry)
 *   x = -inf where allow's bit of v is 0, whatever x was.
 * In fp32, rounded once; values that no step touches are copied bit by bit.
 * Ids outside [0, V) are skipped, rows behind the last node left as they
 * were.  logits and out must be the same buffer or not overlap.
 * Errors: DT_ERR_INVALID_ARG, DT_ERR_UNSUPPORTED (a limit above), DT_ERR_HIP. */
dt_status dt_process_logits(const dt_logits_params* p);

typedef struct dt_commit_params {
    const int32_t* tokens;     /* [B][n_max] as dt_tree_out */
    const int32_t* parents;    /* [B][n_max] as dt_tree_out */
    const int32_t* target;     /* [B][lead + n_max] the token the target chose after each row */
    int32_t L;                 /* row length of the outputs, >= 1; at most L - 1 nodes are accepted */
    int32_t* accepted;         /* [B][L] the accepted nodes' tokens, the target's next token, then -1 */
    int32_t* lengths;          /* [B] accepted nodes + 1 */
    int32_t* nodes;            /* [B][L] the accepted nodes' indexes, then -1; or NULL */
    void* stream;
} dt_commit_params;

/* After verification: from the root down, the child (lowest index) whose
 * token the target chose after its parent is accepted, until there is none.
 * The accepted nodes' keys and values move, in every layer of the cache, from
 * slot ctx_len + lead + node to slots ctx_len + lead + 0, 1, ..., so the
 * cache holds ctx_len + lead + lengths - 1 committed tokens (the next call's
 * ctx_len).  accepted and lengths are dt_ngram_update's tokens and lengths.
 * The chunk's mask and depths are not used; a node whose parent's index is
 * not below its own is never accepted.  A request with ctx_len < 0 gets
 * lengths 0 and -1 everywhere, and nothing moves.  kv may be NULL (tokens
 * only).  A request's own slots must lie in pages of its own.
 * Errors: DT_ERR_INVALID_ARG (also lead < 1, L < 1), DT_ERR_UNSUPPORTED
 *   (n_max > 1024, or a limit above), DT_ERR_HIP. */
dt_status dt_commit_path(const dt_kv_cache* kv, const dt_chunk* chunk, const dt_commit_params* p);

/* ------------------------------------------------------------------------
 * A target with latent attention, and a target whose tokens are drawn.
 *
 * Latent attention keeps one vector a token for all heads: a latent c of Dc
 * elements, from which each head's keys and values are products, and a part r
 * of Dr rotated elements that every head's key shares.  dt_latent_append,
 * dt_latent_attention or dt_latent_prefill, and dt_latent_commit stand where
 * dt_kv_append, dt_tree_attention and dt_commit_path stand for a cache of
 * keys and values; the chunk is the same.
 *
 * dt_sample_rows stands where dt_position_topk with k = 1 stands for a target
 * that is followed greedily: a token for every row, which dt_commit_path and
 * dt_latent_commit take as `target`.  A node's row is drawn whether or not its
 * node is reached, and the path follows the drawn tokens, so the accepted
 * tokens have the target's own distribution whatever the tree.
 * ------------------------------------------------------------------------ */

/* A paged cache of latents.  Element i of the token in slot s of request b in
 * layer l lies at
 *   c + l * layer_stride + page * page_stride + (s % page_size) * slot_stride + i
 * with page = page_table[b * max_pages + s / page_size]: the latent first
 * (i < Dc), then the rotated part.  Strides, pages and slots as in dt_kv_cache;
 * calls that write refuse strides below Dc + Dr. */
typedef struct dt_latent_cache {
    void* c;
    const int32_t* page_table; /* device [B][max_pages] */
    int64_t layer_stride;
    int64_t page_stride;
    int64_t slot_stride;
    int32_t layers;            /* >= 1 */
    int32_t num_pages;         /* >= 1 */
    int32_t page_size;         /* >= 1; max_pages * page_size <= 2^30 */
    int32_t max_pages;         /* >= 1 */
    int32_t Dc;                /* elements of a latent: 256 or 512 */
    int32_t Dr;                /* elements of the rotated part: 32 or 64 */
    int32_t dtype;             /* DT_DTYPE_BF16 or DT_DTYPE_F16 */
} dt_latent_cache;

typedef struct dt_latent_append_params {
    const void* latent;        /* [B][lead + n_max] rows of Dc */
    const void* k_rot;         /* [B][lead + n_max] rows of Dr: the keys' part before its rotation */
    const void* q_rot;         /* [B][lead + n_max] rows of Hq heads of Dr, or NULL (cache only) */
    void* q_out;               /* as q_rot; may be q_rot itself with the same strides; NULL iff q_rot is */
    int64_t latent_stride;     /* elements from row to row */
    int64_t k_stride;
    int64_t q_stride;
    int64_t q_head_stride;     /* elements from head to head of a row */
    int64_t q_out_stride;
    int64_t q_out_head_stride;
    int32_t Hq;                /* query heads, 1..4096 (not read when q_rot is NULL) */
    const void* norm;          /* [Dc] weights of dtype, or NULL = no norm */
    float eps;                 /* >= 0 */
    const double* freqs;       /* device [Dr / 2] radians a position, or NULL = no rotation */
    int32_t interleaved;       /* as in dt_append_params, with rot_dim = Dr */
    float rot_scale;
    int32_t layer;
    void* stream;
} dt_latent_append_params;

/* The new tokens' latents on their way from the projection: for every row
 *   c = latent * rsqrt(mean(latent^2) + eps) * norm   (norm given; else latent)
 * to the row's cache slot, k_rot turned by the row's position behind it, and
 * the queries' q_rot, every head, turned by it to q_out.  Pairs, angles and
 * roundings as in dt_kv_append; without freqs k_rot and q_rot are copied bit by
 * bit.  Pointers 16-byte aligned, strides multiples of 8; in buffers of
 * more than one row at least what a row covers, heads at least Dr apart.
 * Errors: DT_ERR_INVALID_ARG, DT_ERR_UNSUPPORTED (a limit above), DT_ERR_HIP. */
dt_status dt_latent_append(const dt_latent_cache* cache, const dt_chunk* chunk, const dt_latent_append_params* p);

typedef struct dt_latent_params {
    const void* q;             /* [B][lead + n_max] rows of Hq heads, see below */
    void* out;
    const void* weight;        /* dt_latent_prefill only: [Hq][2 * Dn][Dc] of dtype */
    int64_t q_stride;          /* elements from row to row; the heads of a row are contiguous */
    int64_t out_stride;
    int32_t Hq;                /* query heads, 1..4096 */
    int32_t Dn;                /* dt_latent_prefill only: 64 or 128 */
    int32_t max_keys;          /* dt_latent_prefill only: slots at or behind it are not seen, >= 1 */
    float scale;               /* > 0, finite */
    float* lse;                /* [B][lead + n_max][Hq] or NULL: log of the sum of exp(score) */
    int32_t layer;
    void* workspace;           /* 16-byte aligned device scratch of the size below */
    size_t workspace_bytes;
    void* stream;
} dt_latent_params;

/* Latent attention in its absorbed form: a head's query (q_c, q_r) has Dc + Dr
 * elements (q_c is its unrotated part times the head's key weight), its result
 * Dc (to be multiplied by the head's value weight):
 *   out = sum_j softmax_j(scale * (q_c . c_j + q_r . r_j)) c_j
 * over the slots j that the row sees, as in dt_tree_attention, as are the
 * numerics, rows that see nothing, unseen infinities and NaN, and limits.  An
 * infinity or NaN in a latent that a row sees makes NaN of some or all elements
 * of that row's results.  q may not overlap out.  Pointers 16-byte aligned (lse 4), strides multiples
 * of 8 and at least Hq times a head's elements.
 * Errors: DT_ERR_INVALID_ARG, DT_ERR_UNSUPPORTED (a limit above, or
 *   B * (lead + n_max) * Hq >= 2^31), DT_ERR_WORKSPACE, DT_ERR_HIP. */
dt_status dt_latent_attention(const dt_latent_cache* cache, const dt_chunk* chunk, const dt_latent_params* p);

/* Bytes of workspace dt_latent_attention needs (depends on Dc, on the chunk's
 * B, lead and n_max and on Hq only); 0 if a call would be refused for these.
 * Its contents are meaningless between calls. */
size_t dt_latent_workspace(const dt_latent_cache* cache, const dt_chunk* chunk, int32_t Hq);

/* Latent attention in its expanded form, for many rows (a piece of a prompt):
 * with k_j = weight[h][0..Dn) . c_j and v_j = weight[h][Dn..2 Dn) . c_j, sums in
 * fp32 and rounded to dtype, and q = (q_n, q_r) of Dn + Dr elements,
 *   out = sum_j softmax_j(scale * (q_n . k_j + q_r . r_j)) v_j    (Dn elements)
 * for every head h.  The keys and values are made in the workspace, 4 * Dn bytes
 * a head, request and slot below max_keys: at least the longest request's
 * ctx_len + rows for all to be seen.  Of a request without rows none are made.
 * The rest is as in dt_latent_attention; weight is contiguous, 16-byte aligned.
 * Errors: as dt_latent_attention, and DT_ERR_UNSUPPORTED for another Dn and for
 *   keys and values of 2^63 bytes and more. */
dt_status dt_latent_prefill(const dt_latent_cache* cache, const dt_chunk* chunk, const dt_latent_params* p);

/* Bytes of workspace dt_latent_prefill needs; 0 if a call would be refused for
 * these, but SIZE_MAX where B, Hq, Dn and max_keys ask for 2^63 bytes and more. */
size_t dt_latent_prefill_workspace(const dt_latent_cache* cache, const dt_chunk* chunk, int32_t Hq, int32_t Dn,
                                   int32_t max_keys);

/* dt_commit_path for a cache of latents (which may not be NULL). */
dt_status dt_latent_commit(const dt_latent_cache* cache, const dt_chunk* chunk, const dt_commit_params* p);

typedef struct dt_sample_params {
    const void* logits;        /* device [B][lead + n_max][V] of dtype, 16-byte aligned */
    int32_t B;                 /* 0 <= B <= 65535 */
    int32_t lead;              /* >= 0 */
    int32_t n_max;             /* >= 0; 1 <= lead + n_max <= 65536, B * (lead + n_max) <= 2^24 */
    int32_t V;                 /* 1 <= V < 2^26 */
    int32_t dtype;             /* DT_DTYPE_F32 or DT_DTYPE_BF16 */
    const int32_t* n_nodes;    /* [B], clamped to 0..n_max; NULL = n_max */
    const float* u;            /* [B][lead + n_max] random numbers in [0, 1) */
    const float* temperature;  /* [B] or NULL = 1; not above 0 (or NaN): the largest logit's token */
    const int32_t* top_k;      /* [B] or NULL; not above 0: off */
    const float* top_p;        /* [B] or NULL; 1 and more (or NaN): off */
    const float* min_p;        /* [B] or NULL; not above 0 (or NaN): off */
    int32_t* tokens;           /* [B][lead + n_max] */
    float* logp;               /* [B][lead + n_max] or NULL: log of the probability the token was drawn with */
    void* workspace;           /* not read: no call needs one at present */
    size_t workspace_bytes;
    void* stream;
} dt_sample_params;

/* A token for every row of a chunk, drawn by the row's random number u.  With
 * the tokens in the order (logit desc, id asc) and w = exp((logit - largest
 * logit) / temperature):
 *   top_k   only the first top_k tokens stay;
 *   top_p   of these a token stays iff the w of those before it sum to less
 *           than top_p times the sum of all of these (the first always);
 *   min_p   a token stays iff w >= min_p (the first always).
 * The token drawn is the first BY ID, of those that stay, with which the sum of
 * their w so far exceeds u times the sum of them all.  logp is the logarithm
 * of its w over that sum.  Each w is rounded to a multiple of 2^-s and summed
 * exactly, so no result depends on an order; s is 62 - n, 2^n the power of two
 * from V on, and at most 50 (44 for V = 151936).  A row whose logits are all
 * -inf gives token -1 and logp -inf, and NaN counts as -inf.  +inf gives an
 * unspecified token (but a memory-safe one, in -1..V-1), and u outside [0, 1)
 * the first or the last token that stays.  Rows behind the last node are
 * left as they were.
 * Errors: DT_ERR_INVALID_ARG, DT_ERR_UNSUPPORTED (a limit above), DT_ERR_HIP. */
dt_status dt_sample_rows(const dt_sample_params* p);

/* Bytes of workspace dt_sample_rows needs: 0 for every call at present. */
size_t dt_sample_workspace(const dt_sample_params* p);

#ifdef __cplusplus
}
#endif
#endif /* DT_H */
