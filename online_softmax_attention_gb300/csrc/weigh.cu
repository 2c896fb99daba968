// The attention that cached tokens get from new ones (attn_weigh_args): for every token j of
// an entry, w_j += sum over its query rows (new token t, query head h) of
// exp(scale <q_th, k_j> - lse_th), where t sees j.  The rows' lse is known, so there is no
// running maximum, values are not read, and nothing is joined between blocks.
//
// Decomposition.  A unit is a run of keys of one entry with all its heads and rows, so that
// one block has a token's whole sum: no atomics, a fixed order.  Its warps share the
// (32 keys, key head) pairs; a warp holds its 32 K rows in registers, as the A operand of
// mma.sync m16n8k16 (rows = keys), while the group's query rows pass as the B operand, eight
// at a time.  The order of the contraction over D is free, so both operands are loaded
// straight from memory, 16 bytes a lane: the quarter-warp's lanes c hold elements
// [32 i + 8 c, + 8) of a row as the operands' columns (2 c, 2 c + 1, 2 c + 8, 2 c + 9) of
// two steps.  Nothing is staged in shared memory.  Every lane sums exponentials of four
// keys over its columns; lanes and warps are joined once a unit.  Blocks take equal
// stretches of all units (stretch.cuh).  f32 caches use FFMA, a key a lane.
//
// Bound: HBM, the K rows read once, for few rows; the mma.sync rate for many.
#include "../../include/attn.h"
#include "mma.cuh"
#include "stretch.cuh"
#include "window.h"

namespace attn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 32;   // of a warp
constexpr int kRows = 8;    // query rows at a time

struct Entry {
    int s, L, T, q0, fresh;
    int units;  // runs of `keys` tokens
};

// Bitmaps of the sequences that are listed, and that are listed more than once.
struct Listed {
    uint32_t *once, *twice;
};

__device__ __forceinline__ Entry entry_at(const WeighParams &p, const Listed &listed, int i, int keys, bool report) {
    Entry e;
    e.q0 = p.cu[i];
    e.T = p.cu[i + 1] - e.q0;
    e.s = p.seqs[i];
    bool ok = (unsigned)e.s < (unsigned)p.c.max_seqs && e.q0 >= 0 && e.q0 <= p.cu[i + 1] && p.cu[i + 1] <= p.n_q;
    ok = ok && !((listed.twice[e.s >> 5] >> (e.s & 31)) & 1);
    e.L = ok ? p.c.lens[e.s] : 0;
    e.fresh = p.fresh ? p.fresh[i] : e.T;
    ok = ok && e.L >= e.T && e.L <= p.cols && (long long)e.L <= (long long)p.c.max_pages << p.c.page_shift &&
         e.fresh >= 0 && e.fresh <= e.L;
    if (!ok) {
        if (report) report_status(p.c.status, ATTN_EINVAL);
        e.L = 0;
    }
    e.units = e.T > 0 || e.fresh > 0 ? (e.L + keys - 1) / keys : 0;
    return e;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) weigh_kernel(const WeighParams p) {
    constexpr bool kMma = sizeof(T) == 2;
    constexpr int kSteps = D / 32;  // 16-byte chunks of a row a lane
    extern __shared__ uint32_t s_listed[];
    __shared__ float s_sum[kWarps][kKeys];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    pdl_trigger();
    pdl_wait();

    const int words = (p.c.max_seqs + 31) / 32;
    const Listed listed{s_listed, s_listed + words};
    for (int x = tid; x < 2 * words; x += kThreads) s_listed[x] = 0;
    __syncthreads();
    for (int i = tid; i < p.n; i += kThreads) {
        const int s = p.seqs[i];
        if ((unsigned)s >= (unsigned)p.c.max_seqs) continue;
        const uint32_t bit = 1u << (s & 31);
        if (atomicOr(&listed.once[s >> 5], bit) & bit) atomicOr(&listed.twice[s >> 5], bit);
    }
    __syncthreads();

    // few key heads: several runs of 32 keys a unit, so that every warp has a pair
    const int subs = p.c.H >= kWarps ? 1 : kWarps / p.c.H, at_once = kWarps / subs;
    const int sub = warp % subs, first_head = warp / subs, unit_keys = kKeys * subs;
    Stretch st;
    const bool any = find_stretch<kWarps, 0>(
        p.n, 1, [&](int i, bool report) { return Work{0, entry_at(p, listed, i, unit_keys, report).units}; }, st);
    if (!any) return;
    long long before = st.before;
    int ei = st.entry;
    Entry e = entry_at(p, listed, ei, unit_keys, false);

    for (long long at = st.at; at < st.end; ++at) {
        while (at >= before + e.units) {
            before += e.units;
            e = entry_at(p, listed, ++ei, unit_keys, false);
        }
        const int unit0 = (int)(at - before) * unit_keys, key0 = unit0 + kKeys * sub;
        const int ctx = e.L - e.T, rows = e.T * p.group;
        // a run that every new token sees whole, or that none sees
        const bool hidden = p.window && key0 + kKeys <= ctx + 1 - p.window && key0 >= p.sinks;
        const bool whole = key0 + kKeys <= ctx + 1 && (!p.window || key0 >= ctx + e.T - p.window || key0 + kKeys <= p.sinks);
        auto sees = [&](int t, int key) {
            return key <= ctx + t && (!p.window || key > ctx + t - p.window || key < p.sinks);
        };
        long long off = 0;  // of this lane's key's row
        bool live = false;
        if (key0 + lane < e.L && !hidden) {
            const int key = key0 + lane, page = p.c.table[(int64_t)e.s * p.c.table_stride + (key >> p.c.page_shift)];
            live = (unsigned)page < (unsigned)p.c.n_pages;
            if (!live) report_status(p.c.status, ATTN_EINVAL);
            off = live ? page * p.c.b_page + (key & ((1 << p.c.page_shift) - 1)) * p.c.b_tok : 0;
        }
        const bool skip = !__any_sync(0xffffffffu, live);

        float acc[kMma ? 4 : 1];  // keys g + 8 i; FFMA: the lane's
#pragma unroll
        for (int i = 0; i < (kMma ? 4 : 1); ++i) acc[i] = 0.f;
        for (int hk = first_head; hk < p.c.H && !skip && first_head < at_once; hk += at_once) {
            const char *kh = p.c.k + hk * p.c.b_head;
            const T *qh = static_cast<const T *>(p.q) + (int64_t)e.q0 * p.q_st + (int64_t)hk * p.group * p.q_sh;
            const float *lh = p.lse + (int64_t)hk * p.group * p.n_q + e.q0;
            // row r of the head: its token and head of the group
            auto token_of = [&](int r) { return key_head(r, p.group_inv); };
            // minus its lse in log2 units; a row that does not exist, or saw nothing, adds 2^-inf
            auto lse_of = [&](int r) -> float {
                if (r >= rows) return -INFINITY;
                const int t = token_of(r);
                const float x = __ldg(lh + (int64_t)(r - t * p.group) * p.n_q + t);
                return x == -INFINITY ? -INFINITY : -x * kLog2e;
            };
            if constexpr (kMma) {
                uint4 k[4][kSteps];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long o = __shfl_sync(0xffffffffu, off, g + 8 * i);
                    const bool there = __shfl_sync(0xffffffffu, (int)live, g + 8 * i);
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
                        k[i][s] = there ? __ldg(reinterpret_cast<const uint4 *>(kh + o + 64 * s + 16 * c)) : make_uint4(0, 0, 0, 0);
                }
                for (int r0 = 0; r0 < rows; r0 += kRows) {
                    uint4 q[kSteps];
                    const int r = r0 + g, t = token_of(r);
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
                        q[s] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(qh + (int64_t)t * p.q_st + (r - t * p.group) * p.q_sh + 32 * s + 8 * c))
                                        : make_uint4(0, 0, 0, 0);
                    const float l0 = lse_of(r0 + 2 * c), l1 = lse_of(r0 + 2 * c + 1);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {  // 16 keys
                        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int s = 0; s < kSteps; ++s) {
                            const uint4 &lo = k[2 * m][s], &hi = k[2 * m + 1][s];
                            const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
                            mma16816<T>(x, a0, q[s].x, q[s].y);
                            mma16816<T>(x, a1, q[s].z, q[s].w);
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            float pv = exp2_approx(fmaf(x[y], p.scale_log2, y & 1 ? l1 : l0));
                            if (!whole && !sees(token_of(r0 + 2 * c + (y & 1)), key0 + 16 * m + g + (y & 2 ? 8 : 0))) pv = 0.f;
                            acc[2 * m + (y >> 1)] += pv;
                        }
                    }
                }
            } else {
                const float4 *kr = reinterpret_cast<const float4 *>(kh + off);
                for (int r0 = 0; r0 < rows; r0 += kRows) {
                    float x[kRows];
                    const float *qr[kRows];
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const int row = min(r0 + r, rows - 1), t = token_of(row);
                        qr[r] = reinterpret_cast<const float *>(qh) + (int64_t)t * p.q_st + (row - t * p.group) * p.q_sh;
                        x[r] = 0.f;
                    }
#pragma unroll 4
                    for (int d = 0; d < D / 4; ++d) {
                        const float4 kv = live ? __ldg(kr + d) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int r = 0; r < kRows; ++r) {
                            const float4 qv = __ldg(reinterpret_cast<const float4 *>(qr[r]) + d);
                            x[r] = fmaf(qv.x, kv.x, x[r]);
                            x[r] = fmaf(qv.y, kv.y, x[r]);
                            x[r] = fmaf(qv.z, kv.z, x[r]);
                            x[r] = fmaf(qv.w, kv.w, x[r]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const float pv = exp2_approx(fmaf(x[r], p.scale_log2, lse_of(r0 + r)));
                        if (whole || sees(token_of(r0 + r), key0 + lane)) acc[0] += pv;
                    }
                }
            }
        }
        if constexpr (kMma) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 1);
                acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 2);
                if (c == 0) s_sum[warp][g + 8 * i] = acc[i];
            }
        } else {
            s_sum[warp][lane] = acc[0];
        }
        __syncthreads();
        const int key = unit0 + tid;
        if (tid < unit_keys && key < e.L) {
            float *w = p.weights + (int64_t)e.s * p.weights_stride + key;
            float sum = key < e.L - e.fresh ? *w : 0.f;
            float got = 0.f;
            for (int h = 0; h < at_once; ++h) got += s_sum[h * subs + tid / kKeys][tid % kKeys];
            *w = sum + got;
        }
        __syncthreads();
    }
}

template <typename T, int D>
cudaError_t launch_typed(const WeighParams &p, cudaStream_t s) {
    auto kern = weigh_kernel<T, D>;
    const size_t smem = 2 * sizeof(uint32_t) * (size_t)((p.c.max_seqs + 31) / 32);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(2 * sm_count()), dim3(kThreads), smem, s, p);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const WeighParams &p, cudaStream_t s) {
    return p.D == 64 ? launch_typed<T, 64>(p, s) : launch_typed<T, 128>(p, s);
}

}  // namespace

cudaError_t launch_cache_weigh(const WeighParams &p, cudaStream_t s) {
    switch (p.dtype) {
    case ATTN_F16: return launch_d<__half>(p, s);
    case ATTN_BF16: return launch_d<__nv_bfloat16>(p, s);
    default: return launch_d<float>(p, s);
    }
}

}  // namespace attn
