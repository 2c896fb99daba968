// Operations of the paged key / value cache: room for new tokens, writing
// their rows, forking, keeping accepted drafts, freeing, compacting.
//
// The reference counts are the allocator's whole state (0 = free), and
// allocation takes the lowest free pages in list order, so every result is a
// function of the inputs: the only atomics are integer additions on counts.
//
// An operation is a plan and its execution.  The plan kernel (one block)
// validates the whole list, takes the free pages' ranks by a block-wide scan of
// the counts, and writes the plan into the workspace; the kernel behind it
// (programmatic dependent launch) applies it over the whole GPU: tables, counts,
// lengths and the copied rows.  A list that does not pass leaves hdr[0] = 0, and
// the second kernel then changes nothing.
//
// What bounds them: the rows that have to be copied, at HBM rate (16-byte
// loads and stores, whole rows of D elements), above two launches and, for the
// plans, one block's read of the counts (4 bytes a page).
#include "../../include/attn.h"
#include "common.cuh"
#include "pages.h"

namespace attn {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kSeenWords = ATTN_CACHE_MAX_SEQS / 32;  // bitmap of listed sequences (32 KiB)

__device__ __forceinline__ int pages_of(const CacheParams &c, int tokens) { return attn::pages_of(tokens, c.page_shift); }

// Every length read from `lens` is checked before it places anything.
__device__ __forceinline__ bool length_fits(const CacheParams &c, int len) {
    return attn::length_fits(len, c.max_pages, c.page_shift);
}

__device__ __forceinline__ bool in_range(int x, int n) { return (unsigned)x < (unsigned)n; }

__device__ __forceinline__ int table_at(const CacheParams &c, int s, int slot) {
    return c.table[(int64_t)s * c.table_stride + slot];
}

// Inclusive scan over the block's kPlanThreads threads; `total` gets the sum.
template <typename I>
__device__ __forceinline__ I block_scan(I x, I *s_warp, I &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const I y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        I w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const I r = x + (warp ? s_warp[warp - 1] : 0);
    total = s_warp[kPlanThreads / 32 - 1];
    __syncthreads();  // s_warp may be reused
    return r;
}

// 32 consecutive counts from `at` on as a bit mask of those that are zero
// (pages past the pool count as held).
__device__ __forceinline__ uint32_t free_mask(const CacheParams &c, int64_t at) {
    uint32_t m = 0;
    if (at + 32 <= c.n_pages && (reinterpret_cast<uintptr_t>(c.refs) & 15) == 0) {
        int4 r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = *reinterpret_cast<const int4 *>(c.refs + at + 4 * i);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m |= ((r[i].x == 0) | (r[i].y == 0) << 1 | (r[i].z == 0) << 2 | (r[i].w == 0) << 3) << (4 * i);
    } else {
        for (int i = 0; i < 32; ++i)
            if (at + i < c.n_pages && c.refs[at + i] == 0) m |= 1u << i;
    }
    return m;
}

// Marks the sequence as listed; false if it was listed before.
__device__ __forceinline__ bool list_once(uint32_t *seen, int s) {
    const uint32_t bit = 1u << (s & 31);
    return (atomicOr(&seen[s >> 5], bit) & bit) == 0;
}

__device__ __forceinline__ void clear_seen(const CacheParams &c, uint32_t *seen) {
    for (int i = threadIdx.x; i < (c.max_seqs + 31) / 32; i += kPlanThreads) seen[i] = 0;
}

// ---- extend, fork -------------------------------------------------------------------

// Plan: every entry's new pages (first: their prefix; pages: the lowest free
// ones, in order), the length it starts from and the page whose rows it copies.
//   extend: a = sequences, b = token counts;  fork: a = parents, b = children
template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads) alloc_plan_kernel(const CacheParams c, const CachePlan w,
                                                                  const int *a,
                                                                  const int *b, int n) {
    __shared__ uint32_t seen[kSeenWords];
    __shared__ long long s_need[32];
    __shared__ int s_warp[32];
    __shared__ int s_bad;
    pdl_trigger();
    pdl_wait();
    clear_seen(c, seen);
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();

    const int page = 1 << c.page_shift;
    long long carry = 0;  // the same for every thread
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int need = 0;
        bool bad = false;
        if (i < n) {
            const int s = a[i], other = b[i];
            int len = 0, src = -1;
            bad = !in_range(s, c.max_seqs) || (kFork ? !in_range(other, c.max_seqs) : other < 0);
            if (!bad) {
                len = c.lens[s];
                bad = !length_fits(c, len) || !list_once(seen, kFork ? other : s);
            }
            if (!bad) {
                const int tail = len & (page - 1);
                if (tail) {
                    src = table_at(c, s, len >> c.page_shift);
                    bad = !in_range(src, c.n_pages);
                }
                if (kFork) {
                    bad = bad || c.lens[other] != 0;
                    need = tail != 0;
                } else if (!bad) {
                    bad = (long long)len + other > (long long)c.max_pages << c.page_shift;
                    // a partial last page that is not the sequence's own: copied before it grows
                    if (src >= 0 && (other == 0 || c.refs[src] <= 1)) src = -1;
                    if (!bad) need = pages_of(c, len + other) - pages_of(c, len) + (src >= 0);
                }
            }
            if (bad) need = 0;
            w.len[i] = len;
            w.src[i] = src;
        }
        if (bad) s_bad = 1;
        long long total;
        const long long incl = block_scan((long long)need, s_need, total);
        if (i < n) w.first[i] = (int)min(carry + incl - need, (long long)c.n_pages);
        carry += total;
    }
    if (threadIdx.x == 0) w.first[n] = (int)min(carry, (long long)c.n_pages);
    __syncthreads();
    bool ok = !s_bad;
    int got = 0;  // free pages below the part of the pool that was scanned
    if (ok) {
        for (int64_t base = 0; base < c.n_pages && got < carry; base += 32 * kPlanThreads) {
            const int64_t at = base + 32 * threadIdx.x;
            uint32_t m = at < c.n_pages ? free_mask(c, at) : 0u;
            int total;
            int rank = got + block_scan(__popc(m), s_warp, total) - __popc(m);
            for (; m && rank < carry; m &= m - 1) w.pages[rank++] = (int)at + __ffs(m) - 1;
            got += total;
        }
    }
    if (threadIdx.x == 0) {
        const bool room = got >= carry;
        w.hdr[0] = ok && room;
        if (!ok) report_status(c.status, ATTN_EINVAL);
        else if (!room) report_status(c.status, ATTN_ENOPAGES);
    }
}

// Copies rows [0, rows) of a page to another, one layer of k or v; 16 bytes a
// thread and pass.
__device__ __forceinline__ void copy_rows(const CacheParams &c, char *pool, int layer, int from, int to, int rows) {
    const int per_row = c.row_bytes >> 4, per_tok = c.H * per_row;
    const char *src = pool + layer * c.b_layer + from * c.b_page;
    char *dst = pool + layer * c.b_layer + to * c.b_page;
    const int total = rows * per_tok;
    for (int x = threadIdx.x; x < total; x += kCopyThreads) {
        const int t = x / per_tok, r = x - t * per_tok, h = r / per_row, ch = r - h * per_row;
        const int64_t off = t * c.b_tok + h * c.b_head + 16 * ch;
        *reinterpret_cast<uint4 *>(dst + off) = *reinterpret_cast<const uint4 *>(src + off);
    }
}

// Block (i, y): entry i; y walks the layers of k and v; y = 0 also does the
// entry's tables, counts and length.  Source pages come from the plan, because
// the tables change here.
template <bool kFork>
__global__ void __launch_bounds__(kCopyThreads) alloc_apply_kernel(const CacheParams c, const CachePlan w,
                                                                   const int *a,
                                                                   const int *b) {
    pdl_trigger();
    pdl_wait();
    if (!w.hdr[0]) return;
    const int i = blockIdx.x;
    const int s = a[i], other = b[i], len = w.len[i], src = w.src[i], first = w.first[i], need = w.first[i + 1] - first;
    const int tail = len & ((1 << c.page_shift) - 1);
    if (blockIdx.y == 0) {
        if (kFork) {
            int *row = c.table + (int64_t)other * c.table_stride;
            const int full = len >> c.page_shift;
            for (int k = threadIdx.x; k < full; k += kCopyThreads) {
                const int p = table_at(c, s, k);
                row[k] = p;
                if (in_range(p, c.n_pages)) atomicAdd(&c.refs[p], 1);
                else report_status(c.status, ATTN_EINVAL);
            }
            if (threadIdx.x == 0) {
                if (need) {
                    row[full] = w.pages[first];
                    c.refs[w.pages[first]] = 1;
                }
                c.lens[other] = len;
            }
        } else {
            int *row = c.table + (int64_t)s * c.table_stride + pages_of(c, len) - (src >= 0);
            for (int k = threadIdx.x; k < need; k += kCopyThreads) {
                const int p = w.pages[first + k];
                row[k] = p;
                c.refs[p] = 1;
            }
            if (threadIdx.x == 0) {
                if (src >= 0) atomicSub(&c.refs[src], 1);
                c.lens[s] = len + other;
            }
        }
    }
    if (src < 0 || need == 0) return;
    for (int y = blockIdx.y; y < 2 * c.n_layers; y += gridDim.y)
        copy_rows(c, y & 1 ? c.v : c.k, y >> 1, src, w.pages[first], tail);
}

template <bool kFork>
cudaError_t launch_alloc(const CacheParams &c, const CachePlan &w, const int *a, const int *b, int n, cudaStream_t s) {
    cudaError_t e = launch_pdl(alloc_plan_kernel<kFork>, dim3(1), dim3(kPlanThreads), 0, s, c, w, a, b, n);
    count_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(alloc_apply_kernel<kFork>, dim3(n, 2 * c.n_layers), dim3(kCopyThreads), 0, s, c, w, a, b);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ---- keep ------------------------------------------------------------------------------

// Plan: validates (one warp per entry) and, if every entry passes, cuts the
// lengths and releases the pages behind the new ends; len[i] = the length
// before the drafts.
__global__ void __launch_bounds__(kPlanThreads) keep_plan_kernel(const CacheParams c, const CachePlan w,
                                                                 const int *seqs,
                                                                 const int *n_draft,
                                                                 const int *keep, int64_t keep_stride,
                                                                 const int *n_keep, int n) {
    __shared__ uint32_t seen[kSeenWords];
    __shared__ int s_bad;
    pdl_trigger();
    pdl_wait();
    clear_seen(c, seen);
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kPlanThreads / 32;
    for (int i = warp; i < n; i += warps) {
        const int s = seqs[i], d = n_draft[i], k = n_keep[i];
        bool bad = !in_range(s, c.max_seqs);
        const int len = bad ? 0 : c.lens[s];
        bad = bad || !length_fits(c, len) || d < 0 || d > len || k < 0 || k > d || k > keep_stride;
        if (lane == 0 && !bad) bad = !list_once(seen, s);
        if (!__any_sync(0xffffffffu, bad)) {
            const int base = len - d;
            for (int j = lane; j < k; j += 32) {
                const int at = keep[i * keep_stride + j];
                if (!in_range(at, d) || (j > 0 && keep[i * keep_stride + j - 1] >= at)) {
                    bad = true;
                } else if (at != j) {  // the row moves: both pages have to exist, and the one it enters be its own
                    const int to = table_at(c, s, (base + j) >> c.page_shift);
                    const int from = table_at(c, s, (base + at) >> c.page_shift);
                    if (!in_range(to, c.n_pages) || !in_range(from, c.n_pages) || c.refs[to] > 1) bad = true;
                }
            }
            if (lane == 0) w.len[i] = base;
        }
        if (bad) s_bad = 1;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        w.hdr[0] = !s_bad;
        if (s_bad) report_status(c.status, ATTN_EINVAL);
    }
    if (s_bad) return;
    for (int i = warp; i < n; i += warps) {
        const int s = seqs[i], len = w.len[i] + n_keep[i], old = w.len[i] + n_draft[i];
        for (int k = pages_of(c, len) + lane; k < pages_of(c, old); k += 32) {
            const int p = table_at(c, s, k);
            if (in_range(p, c.n_pages) && atomicSub(&c.refs[p], 1) > 0) continue;
            report_status(c.status, ATTN_EINVAL);
            if (in_range(p, c.n_pages)) atomicAdd(&c.refs[p], 1);
        }
        if (lane == 0) c.lens[s] = len;
    }
}

// Block (i, y): entry i, layers of k / v.  Each thread owns 16-byte columns of
// the rows and moves them in ascending order, kBatch loads ahead of the stores.
// That is safe in place: offsets ascend, so offset j goes from keep[j] >= j to
// j, and a store to j can only meet the source of an earlier (already loaded) row.
__global__ void __launch_bounds__(kCopyThreads) keep_move_kernel(const CacheParams c, const CachePlan w,
                                                                 const int *seqs,
                                                                 const int *keep, int64_t keep_stride,
                                                                 const int *n_keep) {
    constexpr int kBatch = 4;
    pdl_trigger();
    pdl_wait();
    if (!w.hdr[0]) return;
    const int i = blockIdx.x, s = seqs[i], k = n_keep[i], base = w.len[i];
    const int *kp = keep + i * keep_stride;
    int j0 = 0;  // rows that stay where they are
    while (j0 < k && kp[j0] == j0) ++j0;
    if (j0 == k) return;
    const int per_row = c.row_bytes >> 4, per_tok = c.H * per_row, mask = (1 << c.page_shift) - 1;
    for (int y = blockIdx.y; y < 2 * c.n_layers; y += gridDim.y) {
        char *pool = (y & 1 ? c.v : c.k) + (y >> 1) * c.b_layer;
        for (int x = threadIdx.x; x < per_tok; x += kCopyThreads) {
            const int h = x / per_row;
            char *col = pool + h * c.b_head + 16 * (x - h * per_row);
            auto row = [&](int t) {
                return reinterpret_cast<uint4 *>(col + table_at(c, s, t >> c.page_shift) * c.b_page + (t & mask) * c.b_tok);
            };
            for (int j = j0; j < k; j += kBatch) {
                uint4 r[kBatch];
#pragma unroll
                for (int q = 0; q < kBatch; ++q)
                    if (j + q < k) r[q] = *row(base + kp[j + q]);
#pragma unroll
                for (int q = 0; q < kBatch; ++q)
                    if (j + q < k) *row(base + j + q) = r[q];
            }
        }
    }
}

// ---- free ------------------------------------------------------------------------------

// One block per entry.  The block that exchanges the length for 0 releases the pages, so
// that a sequence listed twice is released once.
__global__ void __launch_bounds__(kCopyThreads) free_kernel(const CacheParams c, const int *seqs) {
    __shared__ int s_len;
    pdl_trigger();
    pdl_wait();
    const int s = seqs[blockIdx.x];
    if (!in_range(s, c.max_seqs)) {
        if (threadIdx.x == 0) report_status(c.status, ATTN_EINVAL);
        return;
    }
    if (threadIdx.x == 0) {
        const int len = *const_cast<volatile int *>(&c.lens[s]);
        s_len = 0;
        if (!length_fits(c, len)) report_status(c.status, ATTN_EINVAL);
        else if (atomicCAS(&c.lens[s], len, 0) == len) s_len = len;
    }
    __syncthreads();
    const int held = pages_of(c, s_len);
    for (int k = threadIdx.x; k < held; k += kCopyThreads) {
        const int p = table_at(c, s, k);
        if (in_range(p, c.n_pages) && atomicSub(&c.refs[p], 1) > 0) continue;
        report_status(c.status, ATTN_EINVAL);
        if (in_range(p, c.n_pages)) atomicAdd(&c.refs[p], 1);
    }
}

// ---- compact -----------------------------------------------------------------------------

// Plan: L = live pages (hdr[1]); the j-th live page at or above L (from[j])
// moves to the j-th free page below L (pages[j]); as many of one as of the
// other (hdr[2]).  remap: every page's new index.  With a length among lens that does
// not fit, whose table cannot follow, L is the whole pool and nothing moves.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CacheParams c, const CachePlan w) {
    __shared__ int s_warp[32];
    pdl_trigger();
    pdl_wait();
    int live = 0;
    for (int64_t base = 0; base < c.n_pages; base += 32 * kPlanThreads) {
        const int64_t at = base + 32 * threadIdx.x;
        const int exist = (int)max((int64_t)0, min((int64_t)32, c.n_pages - at));
        live += exist - (exist ? __popc(free_mask(c, at)) : 0);
    }
    int front;
    block_scan(live, s_warp, front);
    bool bad = false;
    for (int s = threadIdx.x; s < c.max_seqs; s += kPlanThreads) bad = bad || !length_fits(c, c.lens[s]);
    if (__syncthreads_or(bad)) {
        front = c.n_pages;
        if (threadIdx.x == 0) report_status(c.status, ATTN_EINVAL);
    }
    int holes = 0, movers = 0;
    for (int64_t base = 0; base < c.n_pages; base += 32 * kPlanThreads) {
        const int64_t at = base + 32 * threadIdx.x;
        const int exist = (int)max((int64_t)0, min((int64_t)32, c.n_pages - at));
        const uint32_t all = exist == 32 ? 0xffffffffu : (1u << exist) - 1;
        const uint32_t m = exist ? free_mask(c, at) : 0u;
        const int below = (int)max((int64_t)0, min((int64_t)32, front - at));
        const uint32_t low = below == 32 ? 0xffffffffu : (1u << below) - 1;
        uint32_t hole = m & low, mover = ~m & all & ~low;
        int th, tm;
        int rh = holes + block_scan(__popc(hole), s_warp, th) - __popc(hole);
        int rm = movers + block_scan(__popc(mover), s_warp, tm) - __popc(mover);
        for (; hole; hole &= hole - 1) w.pages[rh++] = (int)at + __ffs(hole) - 1;
        for (; mover; mover &= mover - 1) w.from[rm++] = (int)at + __ffs(mover) - 1;
        holes += th;
        movers += tm;
        for (int k = 0; k < exist; ++k) w.remap[at + k] = (int)at + k;
    }
    __syncthreads();  // the lists and the identity are written
    for (int j = threadIdx.x; j < movers; j += kPlanThreads) w.remap[w.from[j]] = w.pages[j];
    if (threadIdx.x == 0) {
        w.hdr[1] = front;
        w.hdr[2] = movers;
    }
}

// Every block takes (move, layer, k / v) units in turn and a share of the
// tables' rows.  Moved and filled pages are disjoint, so the order is free.
__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const CacheParams c, const CachePlan w) {
    pdl_trigger();
    pdl_wait();
    const int moves = w.hdr[2], per = 2 * c.n_layers;
    if (moves == 0) return;
    for (int64_t u = blockIdx.x; u < (int64_t)moves * per; u += gridDim.x) {
        const int j = (int)(u / per), y = (int)(u - (int64_t)j * per);
        const int from = w.from[j], to = w.pages[j];
        copy_rows(c, y & 1 ? c.v : c.k, y >> 1, from, to, 1 << c.page_shift);
        if (y == 0 && threadIdx.x == 0) {
            c.refs[to] = c.refs[from];
            c.refs[from] = 0;
        }
    }
    const int front = w.hdr[1];
    for (int s = blockIdx.x; s < c.max_seqs; s += gridDim.x) {
        const int held = pages_of(c, c.lens[s]);
        int *row = c.table + (int64_t)s * c.table_stride;
        for (int k = threadIdx.x; k < held; k += kCopyThreads) {
            const int p = row[k];
            if (!in_range(p, c.n_pages)) report_status(c.status, ATTN_EINVAL);
            else if (p >= front) row[k] = w.remap[p];
        }
    }
}

// ---- write -----------------------------------------------------------------------------

// One warp per new row.  Its data (the first kAhead 16-byte chunks a lane of k and of
// v) is loaded first, and lands while the warp looks its place up: a chain of five
// dependent loads (offsets, sequence, length, page, count), which is what bounds
// the small calls that decoding and drafting make.  The entry is the last one whose
// offset is at most the row: counted by the lanes together for short lists, by
// binary search for long ones.
constexpr int kAhead = 4;

__global__ void __launch_bounds__(kCopyThreads)
    write_kernel(const CacheParams c, int layer, const int *seqs, const int *cu, int n,
                 const char *kb, const char *vb, int64_t ks_tok, int64_t ks_head,
                 int64_t vs_tok, int64_t vs_head, int n_rows) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kCopyThreads / 32);
    const int per_row = c.row_bytes >> 4, per_tok = c.H * per_row;
    for (int64_t r = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); r < n_rows; r += warps) {
        uint4 kr[kAhead], vr[kAhead];
        auto load = [&](int x0) {
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int x = x0 + 32 * q + lane, h = x / per_row, ch = 16 * (x - h * per_row);
                if (x < per_tok) {
                    kr[q] = *reinterpret_cast<const uint4 *>(kb + r * ks_tok + h * ks_head + ch);
                    vr[q] = *reinterpret_cast<const uint4 *>(vb + r * vs_tok + h * vs_head + ch);
                }
            }
        };
        load(0);
        int lo = 0;
        if (n <= 256) {
            int below = 0;
            for (int j = lane; j < n; j += 32) below += cu[j] <= r;
            lo = max(0, __reduce_add_sync(0xffffffffu, below) - 1);
        } else {
            int hi = n - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= r) lo = mid;
                else hi = mid - 1;
            }
        }
        const int s = seqs[lo], begin = cu[lo], end = cu[lo + 1];
        // rows behind the last entry (a last offset below the one before it is reported instead)
        if (lo == n - 1 && 0 <= begin && begin <= end && end <= r) break;
        bool bad = !in_range(s, c.max_seqs) || begin < 0 || r < begin || r >= end || end > n_rows;
        for (int j = lane; j < lo; j += 32) bad = bad || seqs[j] == s;  // an earlier entry has the sequence
        int64_t off = 0;
        if (!__any_sync(0xffffffffu, bad)) {
            const int len = c.lens[s], t = (int)(len - end + r);
            bad = len < end - begin || !length_fits(c, len);
            if (!bad) {
                const int p = table_at(c, s, t >> c.page_shift);
                bad = !in_range(p, c.n_pages) || c.refs[p] > 1;
                off = layer * c.b_layer + p * c.b_page + (t & ((1 << c.page_shift) - 1)) * c.b_tok;
            }
        }
        if (__any_sync(0xffffffffu, bad)) {
            if (lane == 0) report_status(c.status, ATTN_EINVAL);
            continue;
        }
        for (int x0 = 0; x0 < per_tok; x0 += 32 * kAhead) {
            if (x0) load(x0);
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int x = x0 + 32 * q + lane, h = x / per_row, ch = 16 * (x - h * per_row);
                if (x < per_tok) {
                    *reinterpret_cast<uint4 *>(c.k + off + h * c.b_head + ch) = kr[q];
                    *reinterpret_cast<uint4 *>(c.v + off + h * c.b_head + ch) = vr[q];
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_cache_extend(const CacheParams &c, const CachePlan &w, const int *seqs, const int *counts, int n,
                                cudaStream_t s) {
    return launch_alloc<false>(c, w, seqs, counts, n, s);
}

cudaError_t launch_cache_fork(const CacheParams &c, const CachePlan &w, const int *parents, const int *children, int n,
                              cudaStream_t s) {
    return launch_alloc<true>(c, w, parents, children, n, s);
}

cudaError_t launch_cache_keep(const CacheParams &c, const CachePlan &w, const int *seqs, const int *n_draft,
                              const int *keep, int64_t keep_stride, const int *n_keep, int n, cudaStream_t s) {
    cudaError_t e = launch_pdl(keep_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, c, w, seqs, n_draft, keep,
                               keep_stride, n_keep, n);
    count_launch();
    if (e != cudaSuccess || keep_stride == 0) return e != cudaSuccess ? e : cudaGetLastError();
    e = launch_pdl(keep_move_kernel, dim3(n, 2 * c.n_layers), dim3(kCopyThreads), 0, s, c, w, seqs, keep, keep_stride,
                   n_keep);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_free(const CacheParams &c, const int *seqs, int n, cudaStream_t s) {
    const cudaError_t e = launch_pdl(free_kernel, dim3(n), dim3(kCopyThreads), 0, s, c, seqs);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheParams &c, const CachePlan &w, cudaStream_t s) {
    cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, c, w);
    count_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(compact_apply_kernel, dim3(sm_count() * 8), dim3(kCopyThreads), 0, s, c, w);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_write(const CacheParams &c, int layer, const int *seqs, const int *cu, int n, const char *kb,
                               const char *vb, int64_t ks_tok, int64_t ks_head, int64_t vs_tok, int64_t vs_head,
                               int n_rows, cudaStream_t s) {
    const int per = kCopyThreads / 32;
    const int64_t want = ((int64_t)n_rows + per - 1) / per, cap = (int64_t)sm_count() * 8;
    const cudaError_t e = launch_pdl(write_kernel, dim3((int)(want < cap ? want : cap)), dim3(kCopyThreads), 0, s, c,
                                     layer, seqs, cu, n, kb, vb, ks_tok, ks_head, vs_tok, vs_head, n_rows);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace attn
