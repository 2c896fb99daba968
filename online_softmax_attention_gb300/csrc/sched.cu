// Schedule preparation for the persistent attention kernels.
//
// One block validates the cu_seqlens offsets on the device (no host copy of
// them is needed) and writes, for tiles of `block` rows (each counted `splits`
// times under split-K), the prefix of work items per sequence into the workspace; it also resets the dynamic work
// counter.  Inconsistent offsets make the schedule empty and set the device
// status word to ATTN_EINVAL, so the attention kernel that follows does no
// work and reads nothing out of bounds.
#include "../../include/attn.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kPrepThreads = 1024;

// Block b prepares schedule b (the backward's two in one launch).  kOrdered: some of them
// take the sequences longest-first.  (Without it, a kernel of its own, and the jobs are read
// where they are passed: one kernel with a copy of them cost a forward 1 us.)
template <bool kOrdered>
__global__ void __launch_bounds__(kPrepThreads)
prep_kernel(const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int n_seq,
            int n_q, int n_k, int causal, const __grid_constant__ PrepJobs jobs, int *status) {
    const PrepJob &job = jobs.job[blockIdx.x];
    const int H = job.H, block = job.block, rows_are_keys = job.rows_are_keys, splits = job.splits;
    int *hdr = job.sched.hdr, *prefix = const_cast<int *>(job.sched.prefix), *order = kOrdered ? job.sched.order : nullptr;
    __shared__ int s_len[kOrdered ? kSortedSeqs : 1], s_order[kOrdered ? kSortedSeqs : 1];
    __shared__ int s_bad;
    __shared__ int s_warp[kPrepThreads / 32];
    __shared__ long long s_carry;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();  // the previous kernel on the stream may still read this schedule block
    if (tid == 0) {
        s_bad = 0;
        s_carry = 0;
    }
    __syncthreads();

    int bad = 0;
    for (int b = tid; b < n_seq; b += kPrepThreads) {
        const int q0 = cu_q ? cu_q[b] : 0, q1 = cu_q ? cu_q[b + 1] : n_q;
        const int k0 = cu_k ? cu_k[b] : 0, k1 = cu_k ? cu_k[b + 1] : n_k;
        if (b == 0 && (q0 != 0 || k0 != 0)) bad = 1;
        if (q1 < q0 || k1 < k0 || q1 > n_q || k1 > n_k) bad = 1;
        if (causal && (q1 - q0) != (k1 - k0)) bad = 1;
    }
    if (bad) atomicOr(&s_bad, 1);
    __syncthreads();
    bad = s_bad;

    auto length = [&](int b) {
        return rows_are_keys ? ((cu_k ? cu_k[b + 1] - cu_k[b] : n_k)) : ((cu_q ? cu_q[b + 1] - cu_q[b] : n_q));
    };
    // longest sequences first, equal ones as they are: a sequence's place is the number
    // that go before it (n_seq <= kSortedSeqs = the block's threads)
    if (order) {
        if (tid < n_seq) s_len[tid] = length(tid);
        __syncthreads();
        if (tid < n_seq) {
            const int mine = s_len[tid];
            int place = 0;
            for (int j = 0; j < n_seq; ++j) place += s_len[j] > mine || (s_len[j] == mine && j < tid);
            s_order[place] = tid;
            order[place] = tid;
        }
        __syncthreads();
    }

    for (int base = 0; base < n_seq; base += kPrepThreads) {
        const int b = base + tid;
        int cnt = 0;
        if (b < n_seq && !bad) {
            const int len = order ? s_len[s_order[b]] : length(b);
            cnt = (len + block - 1) / block * H * splits;
        }
        // inclusive scan across the block
        int x = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int w = s_warp[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += y;
            }
            s_warp[lane] = w;
        }
        __syncthreads();
        const int incl = x + (warp > 0 ? s_warp[warp - 1] : 0);
        const long long carry = s_carry;
        if (b < n_seq) prefix[b] = (int)(carry + incl - cnt);
        __syncthreads();
        if (tid == kPrepThreads - 1) s_carry = carry + incl;
        __syncthreads();
    }
    if (tid == 0) {
        prefix[n_seq] = (int)s_carry;
        hdr[0] = 0;
        hdr[1] = (int)s_carry;
        if (bad) report_status(status, ATTN_EINVAL);
    }
}

}  // namespace

cudaError_t launch_prep(const int32_t *cu_q, const int32_t *cu_k, int n_seq, int n_q, int n_k, int causal,
                        const PrepJobs &jobs, int n_jobs, int *status, cudaStream_t s) {
    bool ordered = false;
    for (int i = 0; i < n_jobs; ++i) ordered = ordered || jobs.job[i].sched.order;
    cudaError_t e = launch_pdl(ordered ? prep_kernel<true> : prep_kernel<false>, dim3(n_jobs), dim3(kPrepThreads), 0, s,
                               cu_q, cu_k, n_seq, n_q, n_k, causal, jobs, status);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace attn
