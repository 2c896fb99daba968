// Eviction from the cache by accumulated attention weight (attn_cache_evict).
//
// Three kernels, the later ones launched dependently.  The check of the list (one block); a
// block an entry that chooses the kept tokens; and the kernel that moves the kept rows, in all
// layers, and their weights, and releases the pages behind.  The list is done as a whole or not
// at all: what the first two find wrong clears hdr[0], and the third then changes nothing.
//
// Choice.  A token's weight, summed over the layers in f64 and rounded to f32, becomes a whole
// number in the same order; four passes over 8 bits each, a histogram a pass, find the
// smallest number that is kept and how many of the tokens that have it are (the first ones).
// A scan in token order then numbers the kept ones.  Every result is a function of the inputs.
//
// Move.  Kept token number j comes from source[j] >= j, ascending.  A block owns 512 bytes of
// every row (32 columns of 16 bytes, one a lane) of a layer of k or v, and takes batches of
// rows, one a warp and pass: all of a batch's rows are loaded before any is stored (a
// barrier), and the next batch's are loaded ahead of the stores, which cannot meet
// them: its sources lie at or behind its own places, which follow this batch's.
//
// Bound: HBM, the moved rows read and written once; few rows: the chain of batches.
#include "../../include/attn.h"
#include "common.cuh"
#include "pages.h"

namespace attn {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kHeld = 40960;  // tokens whose numbers fit shared memory; more are summed anew each pass

__device__ __forceinline__ bool in_range(int x, int n) { return (unsigned)x < (unsigned)n; }

__device__ __forceinline__ int table_at(const CacheParams &c, int s, int slot) {
    return c.table[(int64_t)s * c.table_stride + slot];
}

__global__ void __launch_bounds__(kPlanThreads) evict_check_kernel(const CacheParams c, const EvictParams p) {
    __shared__ uint32_t seen[ATTN_CACHE_MAX_SEQS / 32];
    pdl_trigger();
    pdl_wait();
    for (int i = threadIdx.x; i < (c.max_seqs + 31) / 32; i += kPlanThreads) seen[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
        const int s = p.seqs[i], budget = p.budgets[i];
        if (!in_range(s, c.max_seqs) || budget < 0) {
            bad = true;
            continue;
        }
        const uint32_t bit = 1u << (s & 31);
        const int len = c.lens[s];
        bad = bad || (atomicOr(&seen[s >> 5], bit) & bit) || !length_fits(len, c.max_pages, c.page_shift) || len > p.cols ||
              (len > budget && (long long)p.sinks + p.recent > budget);
        p.len[i] = len;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        p.hdr[0] = !bad;
        if (bad) report_status(c.status, ATTN_EINVAL);
    }
}

// A weight as a whole number in the same order: NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive prefix of x over the block; `total` gets the sum.
__device__ __forceinline__ int block_prefix(int x, int *s_warp, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) s_warp[warp] = y;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    __syncthreads();  // s_warp may be reused
    return before + y - x;
}

__global__ void __launch_bounds__(kPlanThreads) evict_choose_kernel(const CacheParams c, const EvictParams p) {
    extern __shared__ uint32_t held[];
    __shared__ int bins[256], s_warp[32], s_first, s_digit, s_above;
    pdl_trigger();
    pdl_wait();
    // (read by one thread: another block may clear it meanwhile, and nothing of this is used then)
    if (__syncthreads_or(threadIdx.x == 0 && !p.hdr[0])) return;
    const int i = blockIdx.x, tid = threadIdx.x, s = p.seqs[i], budget = p.budgets[i], len = p.len[i];
    if (len <= budget) return;
    const int sinks = p.sinks, last = len - p.recent;  // the tokens [sinks, last) are chosen from
    const int want = budget - sinks - p.recent, n = last - sinks;
    const float *w = p.weights + (int64_t)s * p.w_seq + sinks;
    auto sum_of = [&](int t) {
        double x = w[t];
        for (int y = 1; y < p.w_layers; ++y) x += (double)w[(int64_t)y * p.w_layer + t];
        return order_of((float)x);
    };
    const bool keep = n <= kHeld;
    if (keep)
        for (int t = tid; t < n; t += kPlanThreads) held[t] = sum_of(t);
    auto number_of = [&](int t) { return keep ? held[t] : sum_of(t); };
    if (tid == 0) s_first = len;

    // the smallest number that is kept: its digits from the top; `left` of those that share them so far
    uint32_t found = 0;
    int left = want;
    for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
        if (tid < 256) bins[tid] = 0;
        __syncthreads();
        for (int t0 = 0; t0 < n; t0 += kPlanThreads) {
            const int t = t0 + tid;
            const uint32_t x = t < n ? number_of(t) : 0u;
            const bool in = t < n && (shift == 24 || (x >> (shift + 8)) == (found >> (shift + 8)));
            // equal digits of a warp are counted together: weights of the same size share them
            const uint32_t digit = (x >> shift) & 255u;
            const uint32_t same = __match_any_sync(0xffffffffu, in ? digit : 256u);
            if (in && (tid & 31) == __ffs(same) - 1) atomicAdd(&bins[digit], __popc(same));
        }
        __syncthreads();
        if (tid < 32) {  // the largest digit with at least `left` numbers from it on; lane l has digits 8 l ..
            int mine = 0;
#pragma unroll
            for (int b = 0; b < 8; ++b) mine += bins[8 * tid + b];
            int from = mine;  // of this lane's digits and larger ones
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_down_sync(0xffffffffu, from, o);
                if (tid + o < 32) from += y;
            }
            int above = from - mine;
            if (above < left && from >= left) {
                int b = 7;
                while (above + bins[8 * tid + b] < left) above += bins[8 * tid + b--];
                s_digit = 8 * tid + b;
                s_above = above;
            }
        }
        __syncthreads();
        found |= (uint32_t)s_digit << shift;
        left -= s_above;
        __syncthreads();
    }

    // number the kept ones in order
    int *source = p.source + (int64_t)i * p.cols;
    int kept = 0, equal = 0;  // before the tokens of this pass
    int first = len;          // token that goes
    for (int t0 = 0; t0 < len; t0 += kPlanThreads) {
        const int t = t0 + tid;
        const bool chosen = t >= sinks && t < last;
        const uint32_t x = chosen && want > 0 ? number_of(t - sinks) : 0u;
        const bool tie = chosen && want > 0 && x == found;
        int ties;
        const int rank = equal + block_prefix(tie, s_warp, ties);
        equal += ties;
        const bool stays = t < len && (!chosen || (want > 0 && (x > found || (tie && rank < left))));
        int count;
        const int to = kept + block_prefix(stays, s_warp, count);
        kept += count;
        if (stays) source[to] = t;
        else if (t < len) first = min(first, t);
    }
    atomicMin(&s_first, first);
    __syncthreads();
    first = s_first;
    if (tid == 0) p.first[i] = min(first, budget);
    // every page from the first row that moves on exists, and those that rows move into are the sequence's own
    bool bad = false;
    if (first < budget) {
        const int end = pages_of(budget, c.page_shift);
        for (int k = (first >> c.page_shift) + tid; k < end; k += kPlanThreads) {
            const int page = table_at(c, s, k);
            bad = bad || !in_range(page, c.n_pages) || c.refs[page] > 1;
        }
    }
    for (int k = (min(first, budget) >> c.page_shift) + tid; k < pages_of(len, c.page_shift); k += kPlanThreads)
        bad = bad || !in_range(table_at(c, s, k), c.n_pages);
    if (__syncthreads_or(bad) && tid == 0) {
        p.hdr[0] = 0;
        report_status(c.status, ATTN_EINVAL);
    }
}

// Moves what a warp's lanes hold of rows [first, count) to their places; load(token), store(row, value).
// kRows rows a warp and batch.
template <int kRows, typename V, typename L, typename S>
__device__ __forceinline__ void move_rows(const int *source, int first, int count, L load, S store) {
    constexpr int kWarps = kMoveThreads / 32, kBatch = kRows * kWarps;
    const int warp = threadIdx.x >> 5;
    V now[kRows], next[kRows];
    auto fetch = [&](int j0, V (&v)[kRows]) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int j = j0 + r * kWarps + warp;
            if (j < count) v[r] = load(source[j]);
        }
    };
    fetch(first, now);
    for (int j0 = first; j0 < count; j0 += kBatch) {
        __syncthreads();  // every warp has its rows of this batch
        fetch(j0 + kBatch, next);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int j = j0 + r * kWarps + warp;
            if (j < count) store(j, now[r]);
            now[r] = next[r];
        }
    }
}

// Block (i, y): entry i; y walks the 512-byte columns of the layers of k and v, then the layers of weights.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const CacheParams c, const EvictParams p) {
    pdl_trigger();
    pdl_wait();
    if (!p.hdr[0]) return;
    const int i = blockIdx.x, lane = threadIdx.x & 31, s = p.seqs[i], count = p.budgets[i], len = p.len[i];
    if (len <= count) return;
    const int first = p.first[i];
    const int *source = p.source + (int64_t)i * p.cols;
    const int per_row = c.row_bytes >> 4, per_tok = c.H * per_row, strips = (per_tok + 31) / 32;
    const int mask = (1 << c.page_shift) - 1, pools = 2 * c.n_layers * strips;
    for (int y = blockIdx.y; y < pools + p.w_layers; y += gridDim.y) {
        if (y < pools) {
            const int layer = y / (2 * strips), rest = y - layer * 2 * strips, x = (rest >> 1) * 32 + lane, h = x / per_row;
            char *col = (rest & 1 ? c.v : c.k) + layer * c.b_layer + h * c.b_head + 16 * (x - h * per_row);
            const bool mine = x < per_tok;
            auto row = [&](int t) {
                return reinterpret_cast<uint4 *>(col + table_at(c, s, t >> c.page_shift) * c.b_page + (t & mask) * c.b_tok);
            };
            move_rows<8, uint4>(
                source, first, count, [&](int t) { return mine ? *row(t) : make_uint4(0, 0, 0, 0); },
                [&](int j, uint4 v) { if (mine) *row(j) = v; });
        } else {
            // a token a thread: warps take 32 tokens at a time
            float *w = p.weights + (int64_t)(y - pools) * p.w_layer + (int64_t)s * p.w_seq;
            for (int j0 = first; j0 < count; j0 += kMoveThreads * 4) {
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = j0 + r * kMoveThreads + threadIdx.x;
                    if (j < count) v[r] = w[source[j]];
                }
                __syncthreads();
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = j0 + r * kMoveThreads + threadIdx.x;
                    if (j < count) w[j] = v[r];
                }
                __syncthreads();
            }
        }
    }
    if (blockIdx.y == 0) {  // the pages behind the new end
        for (int k = pages_of(count, c.page_shift) + threadIdx.x; k < pages_of(len, c.page_shift); k += kMoveThreads) {
            const int page = table_at(c, s, k);
            if (atomicSub(&c.refs[page], 1) > 0) continue;
            report_status(c.status, ATTN_EINVAL);
            atomicAdd(&c.refs[page], 1);
        }
        if (threadIdx.x == 0) c.lens[s] = count;
    }
}

}  // namespace

cudaError_t launch_cache_evict(const CacheParams &c, const EvictParams &p, cudaStream_t s) {
    cudaError_t e = launch_pdl(evict_check_kernel, dim3(1), dim3(kPlanThreads), 0, s, c, p);
    count_launch();
    if (e != cudaSuccess) return e;
    const int smem = 4 * (p.cols < kHeld ? p.cols : kHeld);
    e = cudaFuncSetAttribute(evict_choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(evict_choose_kernel, dim3(p.n), dim3(kPlanThreads), smem, s, c, p);
    count_launch();
    if (e != cudaSuccess) return e;
    const int64_t per_tok = (int64_t)c.H * (c.row_bytes >> 4), columns = 2 * c.n_layers * ((per_tok + 31) / 32) + p.w_layers;
    e = launch_pdl(evict_move_kernel, dim3(p.n, (unsigned)(columns < 65535 ? columns : 65535)), dim3(kMoveThreads), 0, s, c, p);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace attn
