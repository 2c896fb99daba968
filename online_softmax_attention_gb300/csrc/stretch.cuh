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

// Work of an entry: its units and the key tiles they scan, in one word, so that
// one prefix sum adds up both: fewer than 2^27 units (rows are fewer than 2^31, and a
// unit has more than 16 on average, or there are 2048 entries of 2^14 key heads at the
// most) and fewer than 2^36 tiles (at 16 KiB of keys and values and more each, 1 PB).
constexpr int kTileBits = 36;
__device__ __forceinline__ long long work_of(long long units, long long tiles) { return units << kTileBits | tiles; }
__device__ __forceinline__ long long work_units(long long w) { return w >> kTileBits; }
__device__ __forceinline__ long long work_tiles(long long w) { return w & ((1ll << kTileBits) - 1); }

struct Stretch {
    long long at, end;   // the block's part of the line
    long long share;     // length of a block's part (the last ones may be shorter)
    long long before;    // length of the line before entry `entry`
    long long work;      // work_of the entry
    int entry;           // entry that position `at` lies in
    int lead, snap;      // of a unit of n tiles: see tile()

    // A unit takes lead + n positions: `lead` stands for what a unit costs besides its
    // tiles (loading queries, masks, writing out).  Tile at which position x cuts the
    // unit that begins at u0; a cut that would part fewer than `snap` tiles moves to
    // the unit's edge.
    __device__ __forceinline__ int tile(long long x, long long u0, int n) const {
        const long long o = x - u0 - lead;
        return o >= n ? n : o <= 0 || o < snap ? 0 : o > n - snap ? n : (int)o;
    }
    __device__ __forceinline__ long long length(long long w) const { return work_tiles(w) + lead * work_units(w); }
};

// The block's stretch; work(i, report): work_of entry i.  A unit counts `lead` more
// positions than tiles where blocks have `kLeadShare` tiles and more; the share is a
// multiple of `turn` where it is longer than that.  False: no work.
constexpr int kLeadShare = 12;
template <int kWarps, typename F>
__device__ __forceinline__ bool find_stretch(int n, int turn, int lead, F work, Stretch &s) {
    __shared__ int s_entry;
    __shared__ long long s_before, s_work;
    long long total = 0, mine = 0, count = 0;
    // pass 0 adds all entries up; pass 1 looks for the block's first one (its threads
    // have their entry in hand already where one step covers them all)
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        long long carry = 0;
#pragma unroll 1
        for (int base = 0; base < n; base += 32 * kWarps) {
            const int i = base + threadIdx.x;
            if (pass == 0 || n > 32 * kWarps) {
                count = i < n ? work(i, pass == 0 && blockIdx.x == 0) : 0;
                long long sum;
                mine = carry + block_prefix<kWarps>(count, sum);
                carry += sum;
            }
            if (pass == 0) continue;
            if (s.at >= s.length(mine) && s.at < s.length(mine + count)) {
                s_entry = i;
                s_before = s.length(mine);
                s_work = count;
            }
            if (n > 32 * kWarps && s.at < s.length(carry)) break;  // the same for every thread
        }
        if (pass == 1) break;
        total = carry;
        const bool long_enough = work_tiles(total) >= (long long)kLeadShare * gridDim.x;
        s.lead = long_enough ? lead : 0;
        s.snap = long_enough && lead ? 2 : 0;
        const long long all = s.length(total);
        s.share = all < 0x7fffffff - gridDim.x ? (long long)(((uint32_t)all + gridDim.x - 1) / gridDim.x)
                                               : (all + gridDim.x - 1) / gridDim.x;
        if (s.share > turn) s.share = (s.share + turn - 1) / turn * turn;
        s.at = blockIdx.x * s.share;
        s.end = min(s.at + s.share, all);
        if (s.at >= s.end) return false;
    }
    __syncthreads();
    s.entry = s_entry;
    s.before = s_before;
    s.work = s_work;
    return true;
}

}  // namespace attn
