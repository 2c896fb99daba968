/*
 * attn.h -- C ABI of the GB300 (sm_103a) online-softmax attention library.
 *
 * Exact scaled dot-product attention, forward and fused backward, computed by
 * the online-softmax block recurrence on one GPU.
 *
 * Definition (TIGA-lang, "注意力与稠密关系" attention examples page, section
 * "全量注意力，无掩码", display equation):
 *     s_hij  = <k_hj, q_hi> * scale
 *     out_hi = sum_j softmax_j(s_hi.) v_hj
 * over a relation that decides which (i, j) pairs exist:
 *   ATTN_FULL    every key of the query's sequence (dense relation);
 *   ATTN_CAUSAL  keys j <= i of the query's sequence (same page, section
 *                "因果稠密关系", triangular relation).
 * With cu_seqlens the tokens form independent sequences back to back and no
 * pair crosses a sequence boundary (same page, section
 * "用图组合表达 varlen 因果注意力": block-diagonal relation, flash-attn's
 * cu_seqlens convention [0, L1, L1+L2, ...]).
 *
 * Algorithm (OCANNL "Module Ir.Online_softmax", fourth bullet): for each
 * query tile a scan over key blocks carries the running row max m and the
 * rescaled row sum l, accumulates the numerator U = sum p*v, and the last
 * block writes O = U / l.  A key block that runs past the end of a sequence
 * is a guarded tail padded with -inf scores.  The row log-sum-exp
 * lse = m + ln l (natural log, of the scaled scores) is written for the
 * backward.
 *
 * Backward (same page, third bullet): Dr_i = sum_d dO_id * O_id per row;
 * per pair recompute p and dp = <dO_i, v_j>; ds = p * (dp - Dr_i);
 * dq = scale * ds . k, dk = scale * ds^T . q, dv = p^T . dO.  In the page's
 * layout each gradient has a nest of its own that owns what it writes
 * (ATTN_DQ_SEPARATE: no atomics, run-to-run deterministic); ATTN_DQ_FUSED
 * instead folds the dq nest into the dk/dv nest with f32 reductions (see
 * attn_dq_mode).
 *
 * Conventions for every entry point:
 *  - Every tensor pointer is a DEVICE pointer on the current CUDA device,
 *    owned by the caller.  The library allocates no memory visible to the
 *    caller; scratch comes from the caller's workspace.
 *  - Tensors are (tokens, heads, D) with element strides given per tensor for
 *    the token and head axes; the D axis must be contiguous (stride 1).
 *    Token and head strides must be multiples of 8 elements for 16-bit types
 *    and of 4 elements for f32 (16-byte rows), and base pointers must be
 *    16-byte aligned.
 *  - lse / Dr are f32 (H, n_q) contiguous.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream).  No call synchronises the host, except
 *    attn_device_status().
 *  - Return value: ATTN_OK (0) or a negative attn_status.  Invalid arguments
 *    are rejected before any launch.  Errors found by kernels (inconsistent
 *    cu_seqlens, a watchdog timeout) are reported by attn_device_status().
 *  - Outputs are fully overwritten; no zero-initialisation is needed.
 *  - A query row that admits no key (only an empty key sequence under
 *    ATTN_FULL) gets O = 0 and lse = -inf.
 *  - Inputs must be finite.
 *  - Token counts are at most 2^31 - 2^16 (ATTN_EUNSUPPORTED), and so are those
 *    of (token, head) query rows of grouped heads and over a cache.
 */
#ifndef ATTN_GB300_ATTN_H
#define ATTN_GB300_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_ABI_VERSION 8

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

typedef enum attn_status {
    ATTN_OK = 0,
    ATTN_EINVAL = -1,        /* bad pointer, stride, size or cu_seqlens */
    ATTN_EUNSUPPORTED = -2,  /* valid but not implemented (dtype, D, relation mix, GPU) */
    ATTN_ECUDA = -3,         /* a CUDA runtime call failed; see attn_last_error_string() */
    ATTN_ETIMEOUT = -4,      /* a kernel's bounded wait expired (device watchdog) */
    ATTN_EWORKSPACE = -5,    /* workspace missing or smaller than *_workspace_bytes() */
    ATTN_ENOPAGES = -6       /* a cache has too few free pages (device status; nothing was changed) */
} attn_status;

typedef enum attn_dtype { ATTN_F16 = 0, ATTN_BF16 = 1, ATTN_F32 = 2 } attn_dtype;

typedef enum attn_relation { ATTN_FULL = 0, ATTN_CAUSAL = 1 } attn_relation;

/* Kernel choice.  AUTO picks the tcgen05 tensor-core kernels for f16/bf16 and
 * the FP32 SIMT kernels for f32.  SIMT forces the CUDA-core kernels (any
 * dtype); TC forces the tensor-core kernels (f16/bf16 only). */
typedef enum attn_kernel { ATTN_KERNEL_AUTO = 0, ATTN_KERNEL_SIMT = 1, ATTN_KERNEL_TC = 2 } attn_kernel;

/* How the backward computes dq.
 * SEPARATE: dk/dv by one kernel (per key block, loop over query blocks) and
 *   dq by another (per query block, loop over key blocks), each writing its
 *   gradient once: deterministic, but the dq kernel recomputes the scores and
 *   dp of every pair (7 contractions per pair in all).
 * FUSED: the dk/dv kernel also forms dq's per-pair contribution ds . k
 *   (5 contractions per pair) and adds it with f32 reductions to partial sums
 *   in the workspace; the dq stage scales and converts the sums.  The order of
 *   the additions varies from run to run, so dq may differ in the last bits
 *   between runs.  Tensor-core kernels only (ATTN_EUNSUPPORTED with SIMT).
 * AUTO: SEPARATE (on the causal training shapes the fused kernel's f32
 *   reduction traffic, 64 KiB per pair of 128-row tiles, costs more than the
 *   recomputation it saves). */
typedef enum attn_dq_mode { ATTN_DQ_AUTO = 0, ATTN_DQ_SEPARATE = 1, ATTN_DQ_FUSED = 2 } attn_dq_mode;

/* A (tokens, heads, D) tensor view: element strides of the token and head axes. */
typedef struct attn_tensor {
    void *ptr;
    int64_t stride_tok;
    int64_t stride_head;
} attn_tensor;

typedef struct attn_fwd_args {
    attn_tensor q;        /* in:  (n_q, H, D), dtype */
    attn_tensor k;        /* in:  (n_k, H, D), dtype */
    attn_tensor v;        /* in:  (n_k, H, D), dtype */
    attn_tensor o;        /* out: (n_q, H, D), o_dtype */
    float *lse;           /* out: (H, n_q) f32, natural-log row log-sum-exp; may be NULL */
    int32_t n_q, n_k;     /* total query / key tokens */
    int32_t H, D;         /* heads; head dim (64 or 128) */
    float scale;          /* score scale, usually D^-1/2: any finite value (0 gives the
                             uniform average of the admitted values, a negative one
                             is accepted); NaN or +-inf: ATTN_EINVAL */
    int32_t relation;     /* attn_relation */
    int32_t dtype;        /* attn_dtype of q, k, v */
    int32_t o_dtype;      /* attn_dtype of o: dtype or ATTN_F32 */
    int32_t n_seq;        /* sequences; 1 when cu_seqlens_* are NULL */
    const int32_t *cu_seqlens_q; /* device, n_seq+1 offsets from 0, or NULL (one sequence of n_q) */
    const int32_t *cu_seqlens_k; /* device, n_seq+1 offsets from 0, or NULL (one sequence of n_k) */
    void *workspace;      /* device scratch, attn_fwd_workspace_bytes() bytes, 256-byte aligned */
    size_t workspace_bytes;
    int32_t kernel;       /* attn_kernel */
    int32_t num_ctas;     /* persistent grid size; 0 = one per SM */
    int32_t num_splits;   /* key splits per query tile (split-K): 0 = chosen by the
                             library (see attn_fwd_num_splits), 1 = none, 2..ATTN_MAX_SPLITS */
    float prune_threshold; /* tile pruning (approximate forward, see below): 0 = off,
                              the exact forward; 0 < rho <= 1 enables it */
    uint64_t *pruned_tiles; /* optional device counter, or NULL: with pruning on, the
                               forward adds the number of pruned tiles to it */
    int32_t qk_fp8;       /* 0: q and k are `dtype`; 1: q and k are fp8 e4m3 (see below) */
    int32_t H_kv;         /* heads of k and v: 0 = H; else a divisor of H (grouped heads, below) */
    int32_t window;       /* sliding window (below): 0 = none; else the last keys a query sees */
    int32_t sinks;        /* with a window: the first keys that every query sees beside it */
} attn_fwd_args;

/* Sliding windows with sinks (window, sinks in the forward, the backward and over a
 * cache; no counterpart on the pages): of the keys that a query would see without a
 * window, in order, it sees the first `sinks` and the last `window` (all of them where
 * they are no more than both together).  So query i of a sequence sees key j <= i if
 * i - j < window or j < sinks, and work and reads go with window + sinks, not with
 * the sequence (attn_cache_weigh of few query rows passes over all of a sequence's weights,
 * though not over the hidden keys).  Causal relation only; window > 0 (or none: both 0, ATTN_EINVAL else); no
 * fp8, no pruning, no ATTN_DQ_FUSED (ATTN_EUNSUPPORTED).  A window as long as all the keys
 * is none.  f16 / bf16 inputs run the kernel that packs grouped heads' rows (for ungrouped
 * heads too, and any number of sequences), which takes neither num_splits > 1 nor
 * num_ctas > 0 (ATTN_EUNSUPPORTED) and whose workspace attn_fwd_noalloc does not have;
 * with ATTN_KERNEL_SIMT, groups of more than 128 or f32 inputs, the CUDA-core kernels.
 * With sinks the backward's workspace holds partial sums of dk and dv (the sinks' key
 * blocks are seen by all queries behind them and cut into items; at most 256 blocks a
 * key head), which are added in a fixed order.  Over a cache whose sequences can be longer
 * than the window, tokens that it hides from every new token of an entry may hold anything,
 * NaN included (with a mask, so may new tokens that none of them sees), and the table's
 * entries may be missing for pages in a run of 256 tokens before the new ones, from a
 * multiple of 256 on, that it hides whole. */

/* Grouped heads (H_kv in the forward and the backward; no counterpart on the
 * pages): k and v hold H_kv heads, each shared by a group of G = H / H_kv
 * query heads: query head h attends to key / value head h / G (integer
 * division).  In the backward dk and dv hold H_kv heads too, each the sum over
 * its group's query heads, added in f32 in a fixed order and rounded once.
 * H_kv must divide H (ATTN_EINVAL).  f16 / bf16 inputs with G > 1 run a
 * tensor-core kernel that packs the (token, head of the group) rows of a key head
 * into its tiles, when the library chooses the schedule (num_splits = 0 and
 * num_ctas = 0, at most 2048 sequences, G <= 128, no fp8 or pruning): two
 * launches, no schedule preparation; key ranges cut between CTAs are merged
 * from the workspace (about 40 MB at D = 128).  With that kernel the rows of other
 * sequences, and rows behind the last one, may hold anything, NaN included.  A
 * row with a score of NaN gets O and lse of NaN from that kernel and from
 * attn_tree_fwd (the other forward kernels leave lse = -inf beside that O). */

/* fp8 queries and keys (qk_fp8 = 1; no counterpart on the pages, a use of the
 * sm_103a tensor cores' 8-bit score contraction): q and k hold e4m3 values,
 * one byte per element (strides in elements = bytes, rows 16-byte aligned);
 * v is `dtype` (f16 or bf16), P is rounded to it and o is o_dtype as usual.
 * The scores are the exact products of the e4m3 values accumulated in f32,
 * times `scale`; a caller with per-tensor dequantisation factors for q and k
 * folds them into `scale`.  Tensor-core kernel only: D = 128 and scale > 0,
 * else ATTN_EUNSUPPORTED (also with ATTN_KERNEL_SIMT).  Backward: none. */

/* Tile pruning (TIGA-lang attention examples page, section
 * "基于 tile 剪枝的稀疏注意力", tile-pruned sparse attention): an explicit,
 * approximate option of the forward.  A tile pairs a query tile with a key
 * tile of the kernel's own sizes (128 x 128 for the tensor-core kernel, 64 x 64
 * for the SIMT kernel).  Per query tile the key tiles are scanned in order;
 * every tile's scores are computed, and a tile whose largest score m_tile
 * satisfies  m_tile < m_run + ln(rho)  -- m_run being the largest score of the
 * tiles admitted so far for that query tile -- is pruned: it adds nothing to
 * the softmax or to O (its value tile is still loaded).  The rule bounds no
 * per-row error.  Only the full relation over one sequence (no cu_seqlens) and
 * no key splits are supported; other combinations, and any backward call with
 * a non-zero prune_threshold, return ATTN_EUNSUPPORTED (fail closed). */

/* Upper bound of attn_fwd_args.num_splits and of attn_merge_args.n_parts. */
#define ATTN_MAX_SPLITS 64

typedef struct attn_bwd_args {
    attn_tensor q, k, v;  /* in: as in the forward */
    attn_tensor o;        /* in: forward output, o_dtype */
    attn_tensor dout;     /* in: dL/dO, (n_q, H, D), dtype */
    const float *lse;     /* in: (H, n_q) f32 from attn_fwd */
    attn_tensor dq;       /* out: (n_q, H, D), grad_dtype */
    attn_tensor dk;       /* out: (n_k, H, D), grad_dtype */
    attn_tensor dv;       /* out: (n_k, H, D), grad_dtype */
    int32_t n_q, n_k, H, D;
    float scale;
    int32_t relation, dtype, o_dtype;
    int32_t grad_dtype;   /* attn_dtype of dq, dk, dv: dtype or ATTN_F32 */
    int32_t n_seq;
    const int32_t *cu_seqlens_q, *cu_seqlens_k;
    void *workspace;      /* attn_bwd_workspace_bytes() bytes, 256-byte aligned */
    size_t workspace_bytes;
    int32_t kernel;
    int32_t num_ctas;
    float prune_threshold; /* must be 0: the backward of a tile-pruned forward is not
                              defined, and a non-zero value returns ATTN_EUNSUPPORTED */
    int32_t dq_mode;      /* attn_dq_mode */
    int32_t H_kv;         /* heads of k, v, dk and dv: 0 = H; else a divisor of H */
    int32_t window, sinks; /* as in the forward */
} attn_bwd_args;

/* Partial attention results over disjoint key sets, to be merged
 * (attn_merge).  Partial c is attention of the same query rows over its own
 * key set: its output O_c (normalised by its own row sum) and its row
 * log-sum-exp lse_c (-inf when it admits no key; O_c is then ignored). */
typedef struct attn_merge_args {
    const float *o_parts;   /* in:  (n_parts, n_q, H, D) f32, contiguous */
    const float *lse_parts; /* in:  (n_parts, H, n_q) f32, contiguous */
    attn_tensor o;          /* out: (n_q, H, D), o_dtype; may not overlap the inputs */
    float *lse;             /* out: (H, n_q) f32, or NULL */
    int32_t n_parts;        /* 1..ATTN_MAX_SPLITS */
    int32_t n_q, H, D;      /* D: a multiple of 4, at most 256 */
    int32_t o_dtype;        /* attn_dtype */
} attn_merge_args;

/* Attention over a general CSR relation (TIGA-lang attention examples page:
 * the varlen section writes a relation as an explicit CSR graph of exactly
 * the admitted edges; the GAT section's display equation is a softmax over
 * each row's incoming edges):
 *     out[i, h] = sum_{e in row i} exp(s[e, h]) / sum_{e' in row i} exp(s[e', h]) * v[col[e], h]
 * Row i's edges are col_idx[row_ptr[i] .. row_ptr[i+1]); an edge listed twice
 * counts twice.  The score is the field edge_scores[e, h] (segment softmax)
 * or, with edge_scores NULL, scale * <q[i, h], k[col[e], h]>.  A row without
 * edges gets O = 0, lse = -inf.  Malformed relations (offsets that decrease
 * or leave [0, n_edges], sources outside [0, n_src)) are not read out of
 * bounds: the row or edge is skipped and attn_device_status() reports
 * ATTN_EINVAL.  One kernel on `stream`; no workspace. */
typedef struct attn_csr_args {
    const int64_t *row_ptr;   /* device, n_dst + 1 nondecreasing offsets in [0, n_edges] */
    const int32_t *col_idx;   /* device, n_edges source indices */
    int64_t n_edges;
    int32_t n_dst, n_src;     /* destination rows; source rows */
    int32_t H, D;             /* heads; D a multiple of 4, at most 256 */
    const float *edge_scores; /* device (n_edges, H) f32 field scores, or NULL */
    attn_tensor q;            /* (n_dst, H, D) dtype, dot-product scores only */
    attn_tensor k;            /* (n_src, H, D) dtype, dot-product scores only */
    attn_tensor v;            /* (n_src, H, D) dtype */
    attn_tensor o;            /* out: (n_dst, H, D) o_dtype */
    float *lse;               /* out: (H, n_dst) f32, or NULL */
    float scale;              /* dot-product scores only */
    int32_t dtype;            /* attn_dtype of q, k, v */
    int32_t o_dtype;          /* dtype or ATTN_F32 */
    /* device, n_dst entries: the order in which the kernel takes the rows (a
     * permutation of [0, n_dst)), or NULL for 0, 1, 2, ...  Results do not
     * depend on it, bit for bit; it only decides which rows are in flight
     * together, and so how often their sources' rows are found in the L2:
     * an order that keeps rows with shared sources close (e.g. points sorted
     * along a space-filling curve) turns most gathers into L2 hits.  An entry
     * outside [0, n_dst) is skipped and reported as ATTN_EINVAL; a row the
     * order omits is not written. */
    const int32_t *row_order;
} attn_csr_args;

/* A paged key / value cache (no counterpart on the pages; what serving needs
 * next to the forward).  All arrays are the caller's device memory.
 *
 * Token t of sequence s, layer y, head h lives in row t % page_size of page
 * table[s * table_stride + t / page_size]; k and v are (n_layers, n_pages,
 * page_size, H_kv, D) with one set of element strides for both, D contiguous,
 * rows 16-byte aligned (strides multiples of 8 elements for 16-bit types, 4
 * for f32).  refs[p] counts the sequences that hold page p (and any references
 * the caller adds); a page with refs[p] == 0 is free, so the counts are the
 * allocator's whole state.  Pages are allocated lowest index first, in list
 * order: the same calls give the same tables.
 *
 * The operations below run on `stream`, read and write only device memory and
 * do not synchronise, so a captured loop can hold them.  They validate on the
 * device, and attn_device_status() reports ATTN_EINVAL.  For attn_cache_extend,
 * _fork, _keep and _evict a list with an entry out of range, a sequence listed twice, or
 * lengths that do not fit leaves the whole cache as it was (so do too few free
 * pages, ATTN_ENOPAGES), and so does a length that does not fit for
 * attn_cache_compact; attn_cache_write and _free leave out the entries that are
 * wrong and do the others.  The tables and counts are the cache's own state: a
 * page index outside the pool is reported and never followed where a call meets
 * it, but fork (among the pages to be shared), keep and free (among those to be
 * released) and compact have then done the rest.  Operations on one cache must be
 * ordered by the caller (one stream); reads of it may overlap. */
typedef struct attn_cache {
    void *k, *v;              /* (n_layers, n_pages, page_size, H_kv, D) dtype */
    int64_t stride_layer, stride_page, stride_tok, stride_head; /* elements, of both k and v */
    int32_t *table;           /* (max_seqs, max_pages) page indices */
    int32_t *lens;            /* (max_seqs) tokens of each sequence; 0 = empty */
    int32_t *refs;            /* (n_pages) reference counts; 0 = free */
    int64_t table_stride;     /* elements between the table's rows, >= max_pages */
    int32_t n_layers, n_pages;
    int32_t page_size;        /* a power of two, 1..1024 */
    int32_t H_kv, D;          /* heads; head dim (64 or 128) */
    int32_t dtype;            /* attn_dtype */
    int32_t max_seqs;         /* rows of table, 1..ATTN_CACHE_MAX_SEQS */
    int32_t max_pages;        /* pages a sequence can hold; max_pages * page_size <= 2^31 - 2^16 */
} attn_cache;

#define ATTN_CACHE_MAX_SEQS 262144

/* Attention of new tokens over the cache: one token (decoding), a chunk, or a
 * tree of drafted tokens per sequence, grouped heads, in one call.
 *
 * Entry i is sequence seqs[i] with L = lens[seqs[i]] cached tokens, whose last
 * T = cu[i + 1] - cu[i] are the query tokens themselves (their rows are in the
 * cache: attn_cache_extend, attn_cache_write).  Query token t of the entry is row
 * cu[i] + t of q, o and lse.  It sees every token before the T new ones, and new
 * token u if bit u % 64 of mask[(cu[i] + t) * mask_words + u / 64] is set, or
 * without a mask if u <= t.  A query that sees nothing gets O = 0, lse = -inf.
 *     o = sum_j softmax_j(scale <q, k_j>) v_j, query head h over cache head h / (H / H_kv)
 * Rows of q from cu[n] on are not read, and their o and lse rows are left as
 * they were; so are those of an entry that does not fit (sequence out of range,
 * T > L, offsets that decrease or leave [0, n_q], more new tokens than the mask
 * has bits), which attn_device_status() reports as ATTN_EINVAL.  Cache slots
 * from token L on are never used, whatever they hold; cached rows below L and q
 * must be finite. */
typedef struct attn_tree_args {
    attn_cache cache;     /* H_kv divides H; dtype also of q */
    int32_t layer;
    int32_t H;            /* query heads */
    attn_tensor q;        /* in:  (n_q, H, D) */
    attn_tensor o;        /* out: (n_q, H, D), o_dtype */
    float *lse;           /* out: (H, n_q) f32, natural log; may be NULL */
    const int32_t *seqs;  /* device, n sequences */
    const int32_t *cu;    /* device, n + 1 offsets from 0 */
    const uint64_t *mask; /* device, (n_q, mask_words), or NULL: new tokens see those up to themselves */
    int32_t n;            /* entries */
    int32_t n_q;          /* query rows */
    int32_t mask_words;   /* 64-bit words of a mask row: new tokens of an entry <= 64 * mask_words */
    float scale;          /* any finite value */
    int32_t o_dtype;      /* the cache's dtype or ATTN_F32 */
    void *workspace;      /* attn_tree_workspace_bytes() bytes, 256-byte aligned */
    size_t workspace_bytes;
    /* sliding window, 0 = none: of the tokens that a new one would see without it -- those
     * before the new ones, then new ones, in the cache's order -- it sees the first `sinks`
     * and the last `window`.  Cached rows that no new token of an entry sees are not read,
     * but for those that share a tile with ones that are. */
    int32_t window, sinks;
} attn_tree_args;

/* The attention that cached tokens get, accumulated: which of them a sequence can do without
 * (attn_cache_evict).  With w the layer's row of the entry's sequence,
 *     w[j] = (j < L - fresh ? w[j] : 0) + sum_{t, h} exp(scale <q_th, k_j> - lse_th)
 * for every token j < L of the sequence, over its query rows (new tokens t, all query heads
 * h) that see j: those of attn_tree_fwd without a mask, whose lse this takes.  The sum is
 * taken in f32 in a fixed order.  A row with an lse of -inf (it saw nothing) adds nothing.
 * Entries from w[L] on are left as they are.  An entry that does not fit (as in
 * attn_tree_args; L > cols; fresh not in [0, L]) is left out, and a list that has a
 * sequence more than once as a whole; both are reported as ATTN_EINVAL. */
typedef struct attn_weigh_args {
    attn_cache cache;       /* k of the layer is read; H_kv divides H; dtype also of q */
    int32_t layer;
    int32_t H;              /* query heads */
    attn_tensor q;          /* in: (n_q, H, D), the query rows of attn_tree_fwd */
    const float *lse;       /* in: (H, n_q) f32, natural log, from attn_tree_fwd */
    float *weights;         /* in, out: the layer's (max_seqs, cols) f32, contiguous rows */
    int64_t weights_stride; /* elements between its rows, >= cols */
    int32_t cols;           /* tokens that a row has room for */
    int32_t n;              /* entries */
    int32_t n_q;            /* query rows */
    float scale;            /* as in attn_tree_fwd */
    int32_t window, sinks;  /* as in attn_tree_fwd */
    const int32_t *seqs;    /* device, n sequences */
    const int32_t *cu;      /* device, n + 1 offsets from 0 */
    const int32_t *fresh;   /* device, n: last tokens whose weight starts anew; NULL: the new ones */
    void *workspace;        /* attn_weigh_workspace_bytes() bytes, 256-byte aligned; NULL where that is 0 */
    size_t workspace_bytes;
} attn_weigh_args;

/* The weights by which attn_cache_evict chooses: (n_layers, max_seqs, cols) f32. */
typedef struct attn_weights {
    float *ptr;
    int64_t stride_layer, stride_seq; /* elements; tokens are contiguous, layers do not overlap */
    int32_t n_layers;                 /* >= 1; need not be the cache's */
    int32_t cols;
} attn_weights;

/* Library ABI version (ATTN_ABI_VERSION) and struct sizes, for bindings to
 * check their mirrors of the structs above. */
ATTN_API int attn_abi_version(void);
ATTN_API size_t attn_fwd_args_size(void);
ATTN_API size_t attn_bwd_args_size(void);
ATTN_API size_t attn_merge_args_size(void);
ATTN_API size_t attn_csr_args_size(void);
ATTN_API size_t attn_cache_size(void);
ATTN_API size_t attn_tree_args_size(void);
ATTN_API size_t attn_weigh_args_size(void);
ATTN_API size_t attn_weights_size(void);

/* Bytes of device workspace the call needs (depends on n_seq, H, n_q, and
 * for the forward on the number of key splits: n_splits > 1 adds the partial
 * results, n_splits * n_q * H * (D + 1) * 4 bytes; for the backward on the dq
 * mode: ATTN_DQ_FUSED adds the dq partial sums, n_q * H * D * 4 bytes; a window
 * with sinks adds the sinks' partial sums).
 * Only sizes, dtypes, the relation, the kernel choice, num_splits and whether
 * cu_seqlens are given are read: the tensor and workspace pointers may still
 * be unset.  Arguments the call would reject give the unsplit size. */
ATTN_API size_t attn_fwd_workspace_bytes(const attn_fwd_args *a);
ATTN_API size_t attn_bwd_workspace_bytes(const attn_bwd_args *a);

/* Forward: writes o and lse.  Launches a schedule-preparation kernel and one
 * persistent attention kernel on `stream`; with key splits (split-K) the
 * attention kernel writes one partial result per split into the workspace
 * and a merge kernel (as attn_merge) combines them into o and lse.  One
 * sequence (no cu_seqlens) whose work items fit in one wave of the default
 * grid (num_ctas = 0) needs no preparation: the attention kernel then runs
 * one item per CTA and is the only launch (plus the merge when split). */
ATTN_API int attn_fwd(const attn_fwd_args *a, void *stream);

/* Key splits a forward with these arguments runs (>= 1), resolving
 * num_splits = 0, or a negative attn_status.  Host-only; launches nothing.
 *
 * Split-K (Vx issue "Chunked-dot Reduce lowering: shorten the reduction
 * dependency chain", measurement section: the record FP32 kernel splits the
 * keys in C = 8 chunks): each query tile's key tiles are cut into n_splits
 * contiguous chunks that run as separate work items, so shapes with few
 * query tiles still fill the GPU.  The automatic choice splits only when the
 * query tiles alone leave most SMs idle and every chunk keeps at least two
 * key tiles. */
ATTN_API int attn_fwd_num_splits(const attn_fwd_args *a);

/* Merge of partial results over disjoint key sets into attention over their
 * union (the split-K merge; with each partial's online-softmax state written
 * as m_c = lse_c, l_c = 1, U_c = O_c, this is the (m, l, U) combination of the
 * OCANNL "Module Ir.Online_softmax" page, fourth bullet):
 *     lse = ln sum_c exp(lse_c),   O = sum_c exp(lse_c - lse) O_c.
 * A row whose partials are all -inf gets O = 0, lse = -inf.  One kernel on
 * `stream`; no workspace. */
ATTN_API int attn_merge(const attn_merge_args *a, void *stream);

/* Backward: writes dq, dk, dv.  Equivalent to attn_bwd_preprocess, then
 * attn_bwd_dkdv, then attn_bwd_dq on the same stream and workspace. */
ATTN_API int attn_bwd(const attn_bwd_args *a, void *stream);

/* The three stages of attn_bwd, callable one by one (e.g. to time each):
 *  preprocess: Dr = rowsum(dO * O) into the workspace, and the schedules
 *              (FUSED: also zeroes the dq partial sums);
 *  dkdv:       per key block, loop over query blocks, write dk and dv
 *              (FUSED: also add each pair's dq contribution to the sums);
 *  dq:         SEPARATE: per query block, loop over key blocks, write dq;
 *              FUSED: dq = scale * partial sums, converted to grad_dtype.
 * dkdv and dq read what preprocess wrote into the same workspace. */
ATTN_API int attn_bwd_preprocess(const attn_bwd_args *a, void *stream);
ATTN_API int attn_bwd_dkdv(const attn_bwd_args *a, void *stream);
ATTN_API int attn_bwd_dq(const attn_bwd_args *a, void *stream);

/* Flat form for contiguous (N, H, D) self-attention tensors (token stride
 * H*D, head stride D), o in the input dtype, AUTO kernel choice and AUTO key
 * splits (the same schedule attn_fwd picks for these arguments).
 * cu_seqlens: device, n_seq+1 entries, or NULL for one sequence (n_seq is
 * then ignored).  workspace: device, 256-byte aligned, at least
 * attn_fwd_simple_workspace_bytes(N, H, D, relation, n_seq, dtype) bytes
 * (ATTN_EWORKSPACE otherwise).  Defined as in attn_fwd (TIGA-lang attention
 * examples page, section "全量注意力，无掩码", and its causal and varlen
 * sections). */
ATTN_API int attn_fwd_simple(const void *q, const void *k, const void *v, void *out, float *lse,
                    int32_t N, int32_t H, int32_t D, float scale, int32_t relation,
                    const int32_t *cu_seqlens, int32_t n_seq, int32_t dtype,
                    void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes attn_fwd_simple needs for these sizes (n_seq: the number of
 * sequences cu_seqlens will describe, 1 without cu_seqlens); host-only.  Large
 * enough for any key-split count the library may choose on the current device;
 * 0 for n_seq < 1. */
ATTN_API size_t attn_fwd_simple_workspace_bytes(int32_t N, int32_t H, int32_t D, int32_t relation,
                                                int32_t n_seq, int32_t dtype);

/* The kernel family a call with these arguments runs (ATTN_KERNEL_SIMT or
 * ATTN_KERNEL_TC, resolving AUTO), or a negative attn_status if the call
 * would be rejected.  Host-only; launches nothing. */
ATTN_API int attn_fwd_selected_kernel(const attn_fwd_args *a);
ATTN_API int attn_bwd_selected_kernel(const attn_bwd_args *a);

/* The dq mode a backward with these arguments runs (ATTN_DQ_SEPARATE or
 * ATTN_DQ_FUSED, resolving AUTO), or a negative attn_status.  Host-only. */
ATTN_API int attn_bwd_selected_dq_mode(const attn_bwd_args *a);

/* Attention over the CSR relation of `a` (see attn_csr_args). */
ATTN_API int attn_csr_fwd(const attn_csr_args *a, void *stream);

/* Attention of new tokens over the cache (see attn_tree_args): an attention
 * kernel over equal shares of all (sequence, head, keys) work, and a kernel that
 * merges the shares of a split sequence.  The workspace depends on sizes only
 * (not on lengths); calls that may overlap need one each. */
ATTN_API int attn_tree_fwd(const attn_tree_args *a, void *stream);
ATTN_API size_t attn_tree_workspace_bytes(const attn_tree_args *a);

/* Bytes of workspace attn_cache_extend, _fork, _keep and _compact need for
 * lists of n entries (256-byte aligned device memory); 0 for bad arguments. */
ATTN_API size_t attn_cache_workspace_bytes(const attn_cache *c, int32_t n);

/* Room for counts[i] >= 0 more tokens of sequence seqs[i]: allocates the pages
 * they need and adds counts[i] to lens.  The new rows hold whatever the pages
 * held until attn_cache_write fills them.  A partial last page that other
 * sequences hold too is replaced by a copy first (all layers). */
ATTN_API int attn_cache_extend(const attn_cache *c, const int32_t *seqs, const int32_t *counts,
                               int32_t n, void *workspace, size_t workspace_bytes, void *stream);

/* Writes new k and v rows (n_rows, H_kv, D) of one layer: rows
 * [cu[i], cu[i + 1]) become the last cu[i + 1] - cu[i] tokens of sequence
 * seqs[i] (cu: n + 1 offsets from 0; rows from cu[n] on are left out).  An
 * entry that does not fit, that repeats an earlier entry's sequence, or a row
 * whose page other sequences hold too is skipped and reported as ATTN_EINVAL;
 * the others are written. */
ATTN_API int attn_cache_write(const attn_cache *c, int32_t layer, const int32_t *seqs,
                              const int32_t *cu, int32_t n, const attn_tensor *k, const attn_tensor *v,
                              int32_t n_rows, void *stream);

/* children[i] becomes a copy of parents[i]: it shares the parent's full pages
 * and gets a page of its own for the rows of a partial last one (all layers;
 * the rest of that page is left as it was).  Children must be empty and
 * listed once; a parent may be listed many times. */
ATTN_API int attn_cache_fork(const attn_cache *c, const int32_t *parents, const int32_t *children,
                             int32_t n, void *workspace, size_t workspace_bytes, void *stream);

/* Of the last n_draft[i] tokens of sequence seqs[i] keeps the n_keep[i] whose
 * offsets (in [0, n_draft[i]), strictly ascending) stand at
 * keep[i * keep_stride]: their rows move down, in all layers, to follow the
 * tokens before the drafts; the sequence ends behind them and the pages it no
 * longer needs are released.  Rows behind the new end keep what they hold.  A
 * row that would move into a page that other sequences hold too: ATTN_EINVAL. */
ATTN_API int attn_cache_keep(const attn_cache *c, const int32_t *seqs, const int32_t *n_draft,
                             const int32_t *keep, int64_t keep_stride, const int32_t *n_keep, int32_t n,
                             void *workspace, size_t workspace_bytes, void *stream);

/* Releases the pages of the sequences and empties them.  A sequence listed
 * twice is released once; entries out of range, and sequences whose length is
 * not in [0, max_pages * page_size], are left as they are and reported. */
ATTN_API int attn_cache_free(const attn_cache *c, const int32_t *seqs, int32_t n, void *stream);

/* Moves the live pages to the front: with L live pages, those at or above L
 * move, in ascending order, to the free pages below L (all layers, k and v);
 * the tables and counts follow.  remap (n_pages entries, or NULL) gets every
 * page's new index, for references that the caller holds.  With a length among
 * all of lens that does not fit, nothing moves, and it is reported. */
ATTN_API int attn_cache_compact(const attn_cache *c, int32_t *remap, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Adds the attention that cached tokens get from new ones to their weights (see
 * attn_weigh_args).  Calls on the same rows of weights must be ordered by the caller, and
 * calls that may overlap need a workspace each; its size depends on sizes only (0 for few
 * query rows an entry, f32, pages below 8 rows, and arguments that are refused). */
ATTN_API int attn_cache_weigh(const attn_weigh_args *a, void *stream);
ATTN_API size_t attn_weigh_workspace_bytes(const attn_weigh_args *a);

/* Cuts every listed sequence of more than budgets[i] tokens to that many: its first `sinks`,
 * its last `recent`, and the heaviest of the others by the sum of their weights over the
 * layers (taken in twice f32's precision, rounded to f32; equal weights: the lower token
 * first; NaN is lighter than every number).  The kept rows move down in order, in all layers of the cache,
 * and their weights in all layers of w; the pages behind the new end are released.  Rows
 * and weights behind the new end keep what they hold.  Shorter sequences stay as they are.
 * sinks >= 0, recent >= 0.  A list is done as a whole or not at all: an entry out of
 * range, a sequence listed twice, a negative budget, sinks + recent above the budget of a
 * sequence that is cut, a length above cols, a page index outside the pool, or a row that
 * would move into a page that other sequences hold too: ATTN_EINVAL. */
ATTN_API int attn_cache_evict(const attn_cache *c, const int32_t *seqs, const int32_t *budgets, int32_t n,
                              const attn_weights *w, int32_t sinks, int32_t recent, void *workspace,
                              size_t workspace_bytes, void *stream);

/* Bytes of workspace attn_cache_evict needs for a list of n entries and weights of `cols`
 * tokens (256-byte aligned device memory); 0 for bad arguments. */
ATTN_API size_t attn_cache_evict_workspace_bytes(const attn_cache *c, int32_t n, int32_t cols);

/* Forward for callers that cannot allocate device memory (no counterpart on
 * the pages; a deployment convenience).  Same arguments and results as
 * attn_fwd, except that `num_splits` is taken as 1 (no key splits) and
 * `workspace` / `workspace_bytes` are ignored: the
 * scheduler's scratch lives in a fixed 64 KiB array inside this library's
 * device memory, which every GPU that loads the library keeps until the
 * process exits.  No call allocates anything.
 *  - n_seq must be at most ATTN_NOALLOC_MAX_SEQ; larger inputs return
 *    ATTN_EUNSUPPORTED before any launch.
 *  - The first call on a device looks up the array's device address (with
 *    that device current); make that first call before any stream capture.
 *    The address is kept per device ordinal, so calls must run in the
 *    device's primary context (the CUDA runtime's default context).
 *  - All calls share the one array and each call rewrites the part it reads,
 *    so calls whose kernels overlap on the GPU (concurrent streams, or
 *    threads on one device) race: serialise them on one stream. */
#define ATTN_NOALLOC_MAX_SEQ 16367
ATTN_API int attn_fwd_noalloc(const attn_fwd_args *a, void *stream);

/* Bounded-wait budget, in SM clock cycles, of every mbarrier wait in the
 * tensor-core kernels launched after this call (default 4e9, or the
 * ATTN_WATCHDOG_CYCLES environment variable; cycles <= 0 restores that).  When
 * a wait runs out the kernel stops, drains its loads in flight, frees its
 * tensor memory and exits; attn_device_status() then returns ATTN_ETIMEOUT.
 * Budgets below 2^20 cycles (meant for failure-detection tests) make every
 * wait poll without suspending, so that they run out reliably; larger ones let
 * a wait suspend in hardware first.  Returns the previous budget. */
ATTN_API long long attn_set_watchdog_cycles(long long cycles);

/* Synchronises `stream`, then returns and clears the device-side status word
 * of the current device: ATTN_OK, ATTN_EINVAL (a kernel found inconsistent
 * cu_seqlens and skipped the work) or ATTN_ETIMEOUT (a bounded wait expired
 * and the kernel exited early; outputs are then incomplete). */
ATTN_API int attn_device_status(void *stream);

/* Diagnostic: y[i] = 2^x[i] computed by the polynomial exp2 that the
 * tensor-core kernels run on the FMA pipe for part of the softmax (Cody-Waite
 * range reduction, degree-4 polynomial; max relative error 2.9e-6 for
 * -126 <= x <= 127; x is clamped to that range first, so larger arguments
 * give about 2^127 and smaller ones about 2^-126).  x, y: device arrays of n
 * floats. */
ATTN_API int attn_selftest_exp2(const float *x, float *y, int32_t n, void *stream);

/* Number of kernels the library has launched in this process (all devices). */
ATTN_API uint64_t attn_launch_count(void);

/* Static text for a status code, and the last CUDA error text of this thread. */
ATTN_API const char *attn_strerror(int code);
ATTN_API const char *attn_last_error_string(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_ATTN_H */
