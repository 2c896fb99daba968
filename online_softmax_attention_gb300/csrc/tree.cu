// Attention of new tokens over the cache: the choice between the kernels of tree.cuh and group_tc.cuh, and those of tree.cuh
// without a window and with one, but for masks over a window (tree_masks.cu).
#include "tree.cuh"

namespace attn {

int tree_blocks(const TreeParams &p) { return tree_rows(p) == kGroupRows ? sm_count() : sm_count() * per_sm(p.window > 0, p.dtype == ATTN_F32); }

// Entries of more than 16 rows on average take the tensor-core kernel's units: the
// keys are read once for up to 256 rows (32 sequences of 2000-4000 tokens, 32 key heads'
// rows each, D = 128: 84 us; two 16-row units here: 102).  With 16 rows it is this
// kernel that is faster (75 against 84 us; 4 rows: 71 against 82), without a 128-row
// tile's latency per key tile.  Pages of fewer than 8 rows have no TMA box.
int tree_rows(const TreeParams &p) {
    const bool many = (int64_t)p.n_q * p.group > (int64_t)16 * p.n;
    return many && p.c.page_shift >= 3 && group_supported(p.dtype, p.D, p.group) ? kGroupRows : 16;
}

cudaError_t launch_tree_fwd(const TreeParams &p, cudaStream_t s) {
    if (tree_rows(p) == kGroupRows) {
        GroupParams g = {};
        g.q = p.q; g.o = p.o; g.lse = p.lse;
        g.q_st = p.q_st; g.q_sh = p.q_sh; g.o_st = p.o_st; g.o_sh = p.o_sh;
        g.n = p.n; g.n_q = p.n_q; g.H = p.H; g.Hkv = p.c.H; g.group = p.group; g.D = p.D;
        g.cu_q = p.cu;
        g.paged = 1;
        g.c = p.c;
        g.seqs = p.seqs;
        g.mask = p.mask;
        g.mask_words = p.mask_words;
        g.scale_log2 = p.scale_log2;
        g.dtype = p.dtype; g.o_dtype = p.o_dtype;
        g.parts = p.parts;
        g.status = p.c.status;
        g.watchdog_cycles = p.watchdog_cycles;
        g.window = p.window;
        g.sinks = p.sinks;
        return p.window ? launch_group_window(g, s) : launch_group(g, s);
    }
    if (!p.window) return launch_tree<false, false>(p, s);
    return p.mask ? launch_tree_masks(p, s) : launch_tree<true, false>(p, s);
}

}  // namespace attn
