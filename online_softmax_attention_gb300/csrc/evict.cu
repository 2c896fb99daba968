// Eviction from the cache by accumulated attention weight (attn_cache_evict).
//
// Two kernels.  A block an entry checks it and chooses the kept tokens; the other kernel, launched
// dependently, moves the kept rows, in all layers, and their weights, and releases the pages
// behind.  The list is done as a whole or not at all: every entry leaves a mark, and the
// second kernel does nothing unless all of them are good.
//
// Choice.  A token's weight, summed over the layers and rounded to f32, becomes a whole
// number in the same order; three passes over 11, 11 and 10 bits, a histogram a pass, find the
// smallest number that is kept and how many of the tokens that have it are (the first ones).
// A thread then numbers a run of tokens, behind two scans over the block.  Every result is a
// function of the inputs.
//
// Move.  Kept token number j comes from source[j] >= j, ascending.  A block, or a cluster of them, owns
// up to 512 bytes of every row of a layer of k or v, and moves 64 rows a block and more at a time:
// all of a batch's rows are in shared memory before any is stored (a barrier over the
// cluster), and the next batch's loads are in flight meanwhile, which the stores cannot meet:
// their sources lie at or behind their own places, which follow this batch's.  So a sequence's
// rows move in place, many at once, without a copy.
//
// Bound: HBM, the moved rows read and written once; few rows: the chain of the two kernels.
#include <cfloat>

#include "../../include/attn.h"
#include "common.cuh"
#include "pages.h"

namespace attn {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kHeld = 40960;  // tokens whose numbers fit shared memory; more have them in the workspace

__device__ __forceinline__ bool in_range(int x, int n) { return (unsigned)x < (unsigned)n; }

__device__ __forceinline__ int table_at(const CacheParams &c, int s, int slot) {
    return c.table[(int64_t)s * c.table_stride + slot];
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
    int sums = s_warp[lane];  // (every warp adds them up: there are as many as lanes)
    __syncthreads();          // s_warp may be reused
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += z;
    }
    total = __shfl_sync(0xffffffffu, sums, 31);
    const int before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + y - x;
}

// Bins of a pass's histogram: 11 bits of the weights' numbers (the last pass has 10).
constexpr int kBins = 2048;

__global__ void __launch_bounds__(kPlanThreads) evict_choose_kernel(const CacheParams c, const EvictParams p) {
    extern __shared__ uint32_t s_held[];
    __shared__ int bins[kBins], s_warp[32], s_first, s_digit, s_above;
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x, tid = threadIdx.x, s = p.seqs[i], budget = p.budgets[i];
    bool bad = !in_range(s, c.max_seqs) || budget < 0;
    const int len = bad ? 0 : c.lens[s];
    bad = bad || !length_fits(len, c.max_pages, c.page_shift) || len > p.cols ||
          (len > budget && (long long)p.sinks + p.recent > budget);
    for (int j = tid; j < p.n; j += kPlanThreads) bad = bad || (j != i && p.seqs[j] == s);
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        p.good[i] = !bad;
        p.len[i] = len;
        s_first = len;
        if (bad) report_status(c.status, ATTN_EINVAL);
    }
    if (bad || len <= budget) return;
    // this thread's page of the sequence, for the check at the end
    const int pages = pages_of(len, c.page_shift), my_page = tid < pages ? table_at(c, s, tid) : 0;
    const int my_refs = in_range(my_page, c.n_pages) ? c.refs[my_page] : 0;
    const int sinks = p.sinks, last = len - p.recent;  // the tokens [sinks, last) are chosen from
    const int want = budget - sinks - p.recent, n = last - sinks;
    const float *w = p.weights + (int64_t)s * p.w_seq + sinks;
    // kTokens tokens' sums over the layers, t + kPlanThreads k (those below n): each with the
    // additions' errors beside it, twice f32's precision.  (The GPU adds few f64 numbers at a time:
    // 25 us of them for 32 sequences of 6000 tokens in 8 layers.)
    constexpr int kTokens = 4;
    auto sums_of = [&](int t, uint32_t (&r)[kTokens]) {
        float hi[kTokens], lo[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) hi[k] = lo[k] = 0.f;
#pragma unroll 4
        for (int y = 0; y < p.w_layers; ++y)
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                const float x = t + kPlanThreads * k < n ? w[(int64_t)y * p.w_layer + t + kPlanThreads * k] : 0.f;
                const float sum = __fadd_rn(hi[k], x), was = __fsub_rn(sum, x);
                lo[k] = __fadd_rn(lo[k], __fadd_rn(__fsub_rn(hi[k], was), __fsub_rn(x, __fsub_rn(sum, was))));
                hi[k] = sum;
            }
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            float x = __fadd_rn(hi[k], lo[k]);
            if (!(fabsf(x) <= FLT_MAX) && t + kPlanThreads * k < n) {  // infinities, NaN, or a sum on the way past f32
                double s = 0.;
                for (int y = 0; y < p.w_layers; ++y) s += (double)w[(int64_t)y * p.w_layer + t + kPlanThreads * k];
                x = (float)s;
            }
            r[k] = order_of(x);
        }
    };
    uint32_t *const held = n <= kHeld ? s_held : p.numbers + (int64_t)i * p.cols;

    // the smallest number that is kept: its digits from the top; `left` of those that share them so far
    uint32_t found = 0;
    int left = want;
#pragma unroll 1
    for (int pass = 0; pass < 3 && want > 0; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 0 : pass == 1 ? 21 : 10;
        for (int b = tid; b < kBins; b += kPlanThreads) bins[b] = 0;
        __syncthreads();
        for (int t = tid; t < n; t += kTokens * kPlanThreads) {
            uint32_t x[kTokens];
            if (pass == 0) sums_of(t, x);
#pragma unroll
            for (int k = 0; k < kTokens; ++k) {
                const int at = t + kPlanThreads * k;
                if (at >= n) break;
                if (pass > 0) x[k] = held[at];
                else held[at] = x[k];
                if (pass == 0 || x[k] >> above == found >> above)
                    atomicAdd(&bins[(x[k] >> shift) & (pass == 2 ? 1023u : 2047u)], 1);
            }
        }
        __syncthreads();
        // the largest digit with at least `left` numbers from it on; a thread has two digits, the largest first
        const int hi = kBins - 1 - 2 * tid, at_hi = bins[hi], mine = at_hi + bins[hi - 1];
        int all;
        const int before = block_prefix(mine, s_warp, all);
        if (before < left && before + mine >= left) {
            const bool first = before + at_hi >= left;
            s_digit = first ? hi : hi - 1;
            s_above = first ? before : before + at_hi;
        }
        __syncthreads();
        found |= (uint32_t)s_digit << shift;
        left -= s_above;
        __syncthreads();
    }

    // number the kept ones in order, a run of tokens a thread (an odd run: its words lie in other banks)
    int *source = p.source + (int64_t)i * p.cols;
    for (int t = tid; t < sinks; t += kPlanThreads) source[t] = t;
    for (int t = tid; t < p.recent; t += kPlanThreads) source[budget - p.recent + t] = last + t;
    const int run = ((n + kPlanThreads - 1) / kPlanThreads) | 1, t0 = min(n, tid * run), t1 = min(n, t0 + run);
    int more = 0, equal = 0;
    if (want > 0)
        for (int t = t0; t < t1; ++t) {
            const uint32_t x = held[t];
            more += x > found;
            equal += x == found;
        }
    int all;
    const int ties = max(0, min(equal, left - block_prefix(equal, s_warp, all)));  // of this run that are kept
    int to = sinks + block_prefix(more + ties, s_warp, all), taken = 0, first = len;
    for (int t = t0; t < t1; ++t) {
        const uint32_t x = want > 0 ? held[t] : 0u;
        if (want > 0 && (x > found || (x == found && taken < ties))) {
            taken += x == found;
            source[to++] = sinks + t;
        } else {
            first = min(first, sinks + t);
        }
    }
    if (first < len) atomicMin(&s_first, first);
    __syncthreads();
    first = min(s_first, budget);
    if (tid == 0) p.first[i] = first;
    // every page from the first row that moves on exists, and those that rows move into are the sequence's own
    const int end = first < budget ? pages_of(budget, c.page_shift) : 0;
    if (tid >= first >> c.page_shift && tid < pages) bad = !in_range(my_page, c.n_pages) || (tid < end && my_refs > 1);
    for (int k = max(first >> c.page_shift, kPlanThreads) + tid; k < pages; k += kPlanThreads) {
        const int page = table_at(c, s, k);
        bad = bad || !in_range(page, c.n_pages) || (k < end && c.refs[page] > 1);
    }
    if (__syncthreads_or(bad) && tid == 0) {
        p.good[i] = 0;
        report_status(c.status, ATTN_EINVAL);
    }
}

template <int kCluster>
__device__ __forceinline__ void cluster_barrier() {
    if constexpr (kCluster == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

constexpr int kMoveRows = 8;  // of a warp and batch, in instructions of 32 chunks of 16 bytes
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kMoveBytes = kMoveWarps * kMoveRows * 512;  // of a batch

// Cluster (i, y): entry i; y walks the strips of the layers of k and v, then the layers of weights.
template <int kCluster>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kMoveThreads)
    evict_move_kernel(const CacheParams c, const EvictParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x / kCluster, rank = blockIdx.x % kCluster, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // (one round of loads; `first` is there for those that are cut)
    const int s = p.seqs[i], count = p.budgets[i], len = p.len[i], first = p.first[i];
    bool good = true;
    for (int j = threadIdx.x; j < p.n; j += kMoveThreads) good = good && p.good[j];
    if (!__syncthreads_and(good) || len <= count) return;  // (the whole cluster)
    const int *source = p.source + (int64_t)i * p.cols;
    const int per_row = c.row_bytes >> 4, per_tok = c.H * per_row, strips = (per_tok + 31) / 32;
    const int mask = (1 << c.page_shift) - 1, pools = 2 * c.n_layers * strips;
    // rows of fewer than 32 chunks: several an instruction
    const int width = min(32, per_tok), sub = 32 / width, mine = lane / width, chunk = lane - mine * width;
    const int rows = kMoveRows * sub, step = kCluster * kMoveWarps * rows;  // of a warp; of the cluster's batch
    const int warp0 = (rank * kMoveWarps + warp) * rows;
    const uint32_t buffers = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
    auto offset = [&](int t) -> long long {
        return table_at(c, s, t >> c.page_shift) * c.b_page + (t & mask) * c.b_tok;
    };
    for (int y = blockIdx.y; y < pools + p.w_layers; y += gridDim.y) {
        if (y < pools) {
            const int layer = y / (2 * strips), rest = y - layer * 2 * strips, x = (rest >> 1) * 32 + chunk, h = x / per_row;
            char *col = (rest & 1 ? c.v : c.k) + layer * c.b_layer + h * c.b_head + 16 * (x - h * per_row);
            const bool live = mine < sub && x < per_tok;
            auto load = [&](int j0, int buffer) {  // the batch that begins at row j0
                const int j = j0 + warp0 + lane;   // lane r has the warp's row r
                const long long from = lane < rows && j < count ? offset(source[j]) : 0;
#pragma unroll
                for (int r = 0; r < kMoveRows; ++r) {
                    const int k = r * sub + mine;
                    const long long o = __shfl_sync(0xffffffffu, from, k & 31);
                    if (live && j0 + warp0 + k < count)
                        cp_async16(buffers + buffer * kMoveBytes + r * kMoveThreads * 16, col + o);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            int buffer = 0;
            load(first, 0);
            for (int j0 = first; j0 < count; j0 += step) {
                const int j = j0 + warp0 + lane;
                const long long to = lane < rows && j < count ? offset(j) : 0;
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                cluster_barrier<kCluster>();  // the batch is in shared memory
                if (j0 + step < count) load(j0 + step, buffer ^ 1);
#pragma unroll
                for (int r = 0; r < kMoveRows; ++r) {
                    const int k = r * sub + mine;
                    const long long o = __shfl_sync(0xffffffffu, to, k & 31);
                    if (live && j0 + warp0 + k < count)
                        *reinterpret_cast<uint4 *>(col + o) =
                            *reinterpret_cast<const uint4 *>(smem + buffer * kMoveBytes + (r * kMoveThreads + threadIdx.x) * 16);
                }
                buffer ^= 1;
            }
        } else {
            float *w = p.weights + (int64_t)(y - pools) * p.w_layer + (int64_t)s * p.w_seq;
            constexpr int kTokens = 8, kStep = kCluster * kMoveThreads;
            for (int j0 = first + rank * kMoveThreads + threadIdx.x; j0 - rank * kMoveThreads - (int)threadIdx.x < count;
                 j0 += kTokens * kStep) {
                float v[kTokens];
#pragma unroll
                for (int r = 0; r < kTokens; ++r)
                    if (j0 + r * kStep < count) v[r] = w[source[j0 + r * kStep]];
                cluster_barrier<kCluster>();
#pragma unroll
                for (int r = 0; r < kTokens; ++r)
                    if (j0 + r * kStep < count) w[j0 + r * kStep] = v[r];
            }
        }
    }
    if (blockIdx.y == 0 && rank == 0) {  // the pages behind the new end
        for (int k = pages_of(count, c.page_shift) + threadIdx.x; k < pages_of(len, c.page_shift); k += kMoveThreads) {
            const int page = table_at(c, s, k);
            if (atomicSub(&c.refs[page], 1) > 0) continue;
            report_status(c.status, ATTN_EINVAL);
            atomicAdd(&c.refs[page], 1);
        }
        if (threadIdx.x == 0) c.lens[s] = count;
    }
}

template <int kCluster>
cudaError_t launch_move(const CacheParams &c, const EvictParams &p, unsigned y, cudaStream_t s) {
    auto kern = evict_move_kernel<kCluster>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kMoveBytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(kCluster * p.n, y), dim3(kMoveThreads), 2 * kMoveBytes, s, c, p);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool evict_needs_numbers(int cols) { return cols > kHeld; }

cudaError_t launch_cache_evict(const CacheParams &c, const EvictParams &p, cudaStream_t s) {
    const int held = 4 * (p.cols < kHeld ? p.cols : kHeld);  // bytes
    cudaError_t e = cudaFuncSetAttribute(evict_choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, held);
    if (e != cudaSuccess) return e;
    e = launch_pdl(evict_choose_kernel, dim3(p.n), dim3(kPlanThreads), held, s, c, p);
    count_launch();
    if (e != cudaSuccess) return e;
    const int64_t per_tok = (int64_t)c.H * (c.row_bytes >> 4), columns = 2 * c.n_layers * ((per_tok + 31) / 32) + p.w_layers;
    // Few clusters are wide ones, which move a strip in few batches; many need no width to fill the GPU, and
    // single blocks wait for no others.  (Clusters of 8 and of 1: one sequence of 4 layers, 36 clusters:
    // 24.7 and 36.6 us; 4 sequences of 4000 kept tokens, 144: 122 and 146; 8 sequences, 288: 70 and
    // 64; 32 sequences of 8 layers, 2304: 413 and 351.)
    const int64_t clusters = p.n * columns;
    const unsigned y = (unsigned)(columns < 65535 ? columns : 65535);
    return clusters < 256 ? launch_move<8>(c, p, y, s) : launch_move<1>(c, p, y, s);
}

}  // namespace attn
