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
#include "line.h"

namespace attn {

// Sum of `x` over the threads before this one, and over the whole block
// (kWarps warps; every thread calls it).  Without kUnits, of the tiles only.
template <int kWarps, bool kUnits>
__device__ __forceinline__ Work block_prefix(Work x, Work &total) {
    __shared__ Work s_sum[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Work y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        Work z = {0, __shfl_up_sync(0xffffffffu, y.tiles, o)};
        if (kUnits) z.units = __shfl_up_sync(0xffffffffu, y.units, o);
        if (lane >= o) y = y + z;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = y;
    __syncthreads();
    Work before = {0, 0};
    total = {0, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before = before + s_sum[w];
        total = total + s_sum[w];
    }
    return before + y - x;
}

// The block's stretch; work(i, report): the Work of entry i.  A unit counts kLead more
// positions than tiles where blocks have `kLeadShare` tiles and more (units are counted
// only then: kLead = 0 leaves them out); the share is a multiple of `turn` where it is
// longer than that.  False: no work.
constexpr int kLeadShare = 12;
template <int kWarps, int kLead, typename F>
__device__ __forceinline__ bool find_stretch(int n, int turn, F work, Stretch &s) {
    __shared__ int s_entry;
    __shared__ long long s_before;
    __shared__ Work s_work;
    Work mine = {0, 0}, count = {0, 0};
    // pass 0 adds all entries up; pass 1 looks for the block's first one (its threads
    // have their entry in hand already where one step covers them all)
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        Work carry = {0, 0};
#pragma unroll 1
        for (int base = 0; base < n; base += 32 * kWarps) {
            const int i = base + threadIdx.x;
            if (pass == 0 || n > 32 * kWarps) {
                count = i < n ? work(i, pass == 0 && blockIdx.x == 0) : Work{0, 0};
                Work sum;
                mine = carry + block_prefix<kWarps, kLead != 0>(count, sum);
                carry = carry + sum;
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
        if (!s.take(carry, gridDim.x, blockIdx.x, turn, kLead, kLeadShare)) return false;
    }
    __syncthreads();
    s.entry = s_entry;
    s.before = s_before;
    s.work = s_work;
    return true;
}

}  // namespace attn
