// Equal shares of work whose sizes only the device knows.
//
// Work units (the query rows of one entry and key head, and the key tiles they
// scan) stand in one line, tile after tile.  Block b of a grid of B takes the
// b-th of B equal stretches, so blocks finish together whatever the lengths are.
// Every block finds its stretch from the lengths alone: no schedule is prepared,
// nothing is counted with atomics, and the same lengths give the same cuts, so
// results do not depend on timing.
//
// A stretch holds whole units, whose results the block writes out itself, and at
// most two cut ones: a unit's later part first, another one's first part last.
// Their partial sums go to the block's two workspace slots (0: the unit begins in
// an earlier block, 1: it begins here), and the block whose stretch a unit begins
// in leaves a note (CutUnit) for the merge kernel, which joins the unit's parts in
// block order.
#pragma once

#include "common.cuh"

namespace attn {

// Sum of `x` over the threads before this one, and over the whole block
// (kWarps warps; every thread calls it).
template <int kWarps>
__device__ __forceinline__ long long block_prefix(long long x, long long &total) {
    __shared__ long long s_sum[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = y;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    return before + y - x;
}

struct Stretch {
    long long at, end;   // the block's tiles of the line
    long long share;     // tiles of a block (the last ones may have fewer)
    long long before;    // tiles of the entries before the first one
    int entry;           // entry that tile `at` lies in
};

// The block's stretch; tiles(i, report): key tiles of entry i's units.  The
// share is a multiple of `turn` where it is longer than that.  False: no work.
template <int kWarps, typename F>
__device__ __forceinline__ bool find_stretch(int n, int turn, F tiles, Stretch &s) {
    __shared__ int s_entry;
    __shared__ long long s_before;
    long long total = 0, mine = 0, count = 0;
    for (int base = 0; base < n; base += 32 * kWarps) {
        const int i = base + threadIdx.x;
        count = i < n ? tiles(i, blockIdx.x == 0) : 0;
        long long sum;
        mine = total + block_prefix<kWarps>(count, sum);
        total += sum;
    }
    s.share = (total + gridDim.x - 1) / gridDim.x;
    if (s.share > turn) s.share = (s.share + turn - 1) / turn * turn;
    s.at = blockIdx.x * s.share;
    s.end = min(s.at + s.share, total);
    if (s.at >= s.end) return false;
    // the entry: in hand if one pass covered them all
    long long carry = 0;
    for (int base = 0; base < n; base += 32 * kWarps) {
        const int i = base + threadIdx.x;
        if (n > 32 * kWarps) {
            count = i < n ? tiles(i, false) : 0;
            long long sum;
            mine = carry + block_prefix<kWarps>(count, sum);
            carry += sum;
        }
        if (s.at >= mine && s.at < mine + count) {
            s_entry = i;
            s_before = mine;
        }
        if (n > 32 * kWarps && s.at < carry) break;  // the same for every thread
    }
    __syncthreads();
    s.entry = s_entry;
    s.before = s_before;
    return true;
}

}  // namespace attn
