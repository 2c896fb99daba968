// Internal (not exported) parameter blocks and launchers of the attention
// library.  The C ABI in attn_api.cu validates the public argument structs and
// translates them into these plain-old-data blocks, which kernels take by value.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "heads.h"

namespace attn {

// Schedule block in the workspace: [0] dynamic work counter, [1] item count,
// then the per-sequence prefix of item counts (n_seq + 1 ints), and for the
// backward of up to kSortedSeqs sequences the sequences longest-first (n_seq ints),
// to which the prefix then refers by position.
constexpr int kSchedHeaderInts = 16;
constexpr int kSortedSeqs = 1024;

struct Sched {
    int *hdr;          // counter, total
    const int *prefix; // n_seq + 1 entries
    int *order;        // n_seq entries, or null: sequences as they are
};

struct FwdParams {
    const void *q, *k, *v;
    void *o;
    float *lse;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;
    int n_q, n_k, H, D;
    int Hkv, group;    // key / value heads; query heads that share one (H = Hkv * group)
    unsigned long long group_inv;  // group_inverse(group)
    float scale;       // score scale
    float scale_log2;  // scale * log2(e)
    int causal;
    int dtype, o_dtype;
    int qk_fp8;        // q and k are e4m3 (one byte per element); v is `dtype`
    int n_seq;
    const int32_t *cu_q, *cu_k;  // null => one sequence
    Sched sched;
    // > 0: static schedule of one sequence (cu_q, cu_k null) with this many
    // work items, one per CTA of a grid of exactly this size; the workspace's
    // schedule block is neither written nor read.  0: dynamic schedule.
    int static_items;
    int *status;
    long long watchdog_cycles;
    // split-K: key tiles of every query tile cut into n_splits chunks; chunk c
    // writes its partial (O_c f32, lse_c) at o + c * o_split_st, lse + c * lse_split_st
    int n_splits;
    int64_t o_split_st, lse_split_st;
    // tile pruning: prune a key tile when its largest score (log2 units) is
    // below the query tile's rolling max + prune_log2; count pruned tiles
    int prune;
    float prune_log2;  // log2(rho)
    unsigned long long *pruned_tiles;
    // f32 inputs on the tensor cores: workspace region for the bf16 parts of
    // q, k and v (see fwd_x3.cu), else null
    void *split_ws;
    // grouped heads with packed query rows (group_tc.cu)
    int packed;
};

// Key-tile range [begin, end) of chunk c when n_tiles key tiles are cut into
// n_splits contiguous chunks of ceil(n_tiles / n_splits) tiles (the last ones
// may be shorter or empty).
struct KeyChunk {
    int begin, end;
};
#ifdef __CUDACC__
__host__ __device__
#endif
inline KeyChunk key_chunk(int n_tiles, int n_splits, int c) {
    const int per = (n_tiles + n_splits - 1) / n_splits;
    int b = c * per, e = b + per;
    if (b > n_tiles) b = n_tiles;
    if (e > n_tiles) e = n_tiles;
    return KeyChunk{b, e};
}

struct MergeParams {
    const float *o_parts, *lse_parts;
    void *o;
    float *lse;
    int64_t o_st, o_sh;        // output strides (elements)
    int64_t part_st;           // elements between partials of o_parts (n_q * H * D)
    int n_parts, n_q, H, D, o_dtype;
};

// Attention over a CSR relation (row_ptr over destination rows, col = sources).
struct CsrParams {
    const int64_t *row_ptr;
    const int32_t *col;
    int64_t n_edges;
    int n_dst, n_src, H, D;
    const float *scores;  // (n_edges, H) field scores, or null: dot-product scores
    const void *q, *k, *v;
    void *o;
    float *lse;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;
    float scale_log2;
    int dtype, o_dtype;
    const int32_t *row_order;  // n_dst rows in processing order, or null: identity
    int *status;
};

cudaError_t launch_csr_fwd(const CsrParams &p, cudaStream_t s);

// A paged key / value cache (attn_cache with byte strides and its page size as
// a shift), and the list arguments of its operations.
struct CacheParams {
    char *k, *v;
    int64_t b_layer, b_page, b_tok, b_head;  // byte strides
    int *table, *lens, *refs;
    int64_t table_stride;
    int n_layers, n_pages, page_shift, H, row_bytes;
    int max_seqs, max_pages;
    int *status;
};

// Workspace of the cache operations: what the one-block plan kernels hand to
// the kernels that carry the plan out.
struct CachePlan {
    int *hdr;    // [0] 1: carry out, 0: refused; [1] compact: live pages; [2] compact: moves
    int *first;  // n + 1: prefix of the entries' new pages
    int *len;    // n: extend, keep: length before the call (keep: before the drafts); fork: the parent's
    int *src;    // n: page whose rows are copied to the entry's first new page, or -1
    int *pages;  // n_pages: the new pages in order; compact: the pages moved to
    int *from;   // n_pages: compact: the pages moved from
    int *remap;  // n_pages: compact: every page's new index
};
constexpr int kPlanHdr = 64;

// Partial results of units that are cut between blocks (stretch.cuh): two slots
// for each block of the grid, and the blocks' notes for the merge.
struct CutUnit {
    int last;     // block that holds the unit's last part; <= the writing block: nothing to merge
    int q0, hk;   // first query row (token) of the entry; key head
    int base;     // first (token, head of the group) row of the unit
    int rows;     // such rows of the whole entry
    int pad[3];
};
struct Parts {
    float *o;       // (2 blocks, rows, D) f32 sums relative to the row's max
    float2 *ml;     // (2 blocks, rows): max in log2 units, sum
    CutUnit *cut;   // (blocks)
};

// Merge of cut units.  Row r of a slot is row base + (r / tile_rows) * tile_live +
// r % tile_rows of the entry (r % tile_rows < tile_live; the others do not exist).
struct PartsMergeParams {
    Parts parts;
    void *o;
    float *lse;
    int64_t o_st, o_sh;
    int n_q, group, D, o_dtype;
    int rows, tile_rows, tile_live, blocks;
};
cudaError_t launch_parts_merge(const PartsMergeParams &p, cudaStream_t s);

// Attention of new tokens over the cache (attn_tree_args).
struct TreeParams {
    CacheParams c;          // k, v: the layer's
    const void *q;
    void *o;
    float *lse;
    int64_t q_st, q_sh, o_st, o_sh;  // elements
    const int *seqs, *cu;
    const unsigned long long *mask;
    int n, n_q, mask_words;
    int H, group, D;
    float scale_log2;
    int dtype, o_dtype;
    Parts parts;
    long long watchdog_cycles;
};
// Query rows (token, head of the group) of a work unit (kGroupRows: the
// tensor-core kernel of group_tc.cu), and the grid.
int tree_rows(const TreeParams &p);
int tree_blocks();

// Grouped attention on the tensor cores with packed query rows (group_tc.cu):
// over contiguous keys (prompts) or a cache.
struct GroupParams {
    const void *q;
    void *o;
    float *lse;
    int64_t q_st, q_sh, o_st, o_sh;  // elements
    int n, n_q, H, Hkv, group, D;
    const int *cu_q;                 // n + 1 offsets, or null: one entry of n_q
    int causal;                      // contiguous keys: query i sees keys up to i; else all
    // contiguous keys: k, v views and their offsets (null: one entry of n_k)
    const void *k, *v;
    int64_t k_st, k_sh, v_st, v_sh;
    int n_k;
    const int *cu_k;
    // cached keys: the layer's pools, the entries' sequences, the new tokens' mask
    int paged;
    CacheParams c;
    const int *seqs;
    const unsigned long long *mask;
    int mask_words;
    float scale_log2;
    int dtype, o_dtype;
    Parts parts;
    int *status;
    long long watchdog_cycles;
};
constexpr int kGroupRows = 256;  // query rows of a unit (two 128-row tiles)
bool group_supported(int dtype, int D, int group);
cudaError_t launch_group(const GroupParams &p, cudaStream_t s);
cudaError_t launch_tree_fwd(const TreeParams &p, cudaStream_t s);

cudaError_t launch_cache_extend(const CacheParams &c, const CachePlan &w, const int *seqs, const int *counts, int n,
                                cudaStream_t s);
cudaError_t launch_cache_fork(const CacheParams &c, const CachePlan &w, const int *parents, const int *children, int n,
                              cudaStream_t s);
cudaError_t launch_cache_keep(const CacheParams &c, const CachePlan &w, const int *seqs, const int *n_draft,
                              const int *keep, int64_t keep_stride, const int *n_keep, int n, cudaStream_t s);
cudaError_t launch_cache_free(const CacheParams &c, const int *seqs, int n, cudaStream_t s);
cudaError_t launch_cache_compact(const CacheParams &c, const CachePlan &w, cudaStream_t s);
// kb / vb, ks_* / vs_*: the new rows and their byte strides (token, head)
cudaError_t launch_cache_write(const CacheParams &c, int layer, const int *seqs, const int *cu, int n, const char *kb,
                               const char *vb, int64_t ks_tok, int64_t ks_head, int64_t vs_tok, int64_t vs_head,
                               int n_rows, cudaStream_t s);

struct BwdParams {
    const void *q, *k, *v, *o, *dout;
    const float *lse;
    void *dq, *dk, *dv;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh, do_st, do_sh;
    int64_t dq_st, dq_sh, dk_st, dk_sh, dv_st, dv_sh;
    int n_q, n_k, H, D;
    int Hkv, group;     // key / value heads; query heads that share one (H = Hkv * group)
    unsigned long long group_inv;  // group_inverse(group)
    float scale, scale_log2;
    int causal;
    int dtype, o_dtype, grad_dtype;
    int n_seq;
    const int32_t *cu_q, *cu_k;
    float *dr;          // (H, n_q) rowsum(dO * O), in the workspace
    float *lse2;        // (H, n_q) lse * log2(e), +inf where lse = -inf, in the workspace
    // fused dQ (tensor-core dK/dV kernel also accumulates dQ): f32 partial sums
    // laid out (H, D/4, n_q, 4) in the workspace, so that 32 consecutive query
    // rows of one 4-column group are 512 contiguous bytes; null = separate dQ kernel
    float *dq_accum;
    Sched sched_kv;     // items over key blocks (dk, dv)
    Sched sched_q;      // items over query blocks (dq)
    int *status;
    long long watchdog_cycles;
};

// Schedule preparation: validates cu_seqlens on the device and writes the
// prefix of item counts for tiles of `block` rows of the query or key side, of H
// heads.  Each tile counts as `splits` work items (split-K), numbered tile-major.
// One launch prepares one or two schedules.
struct PrepJob {
    int H, block, rows_are_keys, splits;
    Sched sched;
};
struct PrepJobs {
    PrepJob job[2];
};
cudaError_t launch_prep(const int32_t *cu_q, const int32_t *cu_k, int n_seq, int n_q, int n_k, int causal,
                        const PrepJobs &jobs, int n_jobs, int *status, cudaStream_t s);

// Merge of partial results (split-K): one warp per (query row, head).
cudaError_t launch_merge(const MergeParams &p, cudaStream_t s);

// SIMT (CUDA-core) kernels: any dtype, D in {64, 128}.
constexpr int kSimtBlock = 64;
cudaError_t launch_fwd_simt(const FwdParams &p, int num_ctas, cudaStream_t s);
int fwd_simt_ctas_per_sm(const FwdParams &p);  // resident CTAs per SM of the kernel p selects
cudaError_t launch_bwd_preprocess(const BwdParams &p, cudaStream_t s);
cudaError_t launch_bwd_dkdv_simt(const BwdParams &p, int num_ctas, cudaStream_t s);
cudaError_t launch_bwd_dq_simt(const BwdParams &p, int num_ctas, cudaStream_t s);
// fused dQ: zero the partial sums (before the dK/dV kernel); dq = scale * sums
// converted to grad_dtype with dq's strides (after it)
cudaError_t launch_dq_accum_zero(const BwdParams &p, cudaStream_t s);
cudaError_t launch_dq_accum_convert(const BwdParams &p, cudaStream_t s);

// Number of multiprocessors of the current device.
int sm_count();

#ifdef __CUDACC__
// Launch with programmatic stream serialization: the kernel may start while the
// kernel before it on the stream is still running (once every CTA of that one
// has started and executed pdl_trigger).  Every kernel launched this way
// executes pdl_wait -- which returns once the previous grid has completed and
// its writes are visible -- before it reads global memory, so it sees that
// kernel's results; what it overlaps is its launch and set-up.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Args &&>(args)...);
}
#endif

// Kernel-launch accounting (attn_launch_count).
void count_launch(int n = 1);

}  // namespace attn
