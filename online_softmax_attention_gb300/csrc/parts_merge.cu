// Merge of the partial results of units that were cut between blocks
// (stretch.cuh): with part c's row max m_c (log2 units), sum l_c and numerator
// U_c, m = max m_c, l = sum 2^(m_c - m) l_c and O = sum 2^(m_c - m) U_c / l, the
// (m, l, U) combination of the online-softmax recurrence, in block order.
//
// Block (b, y) merges rows y, y + gridDim.y, ... (times the warps) of the unit
// that block b of the attention kernel noted as begun and cut, if it did.
// Latency-bound: a note, the parts' (m, l), then the parts, a few of them at a
// time in flight.  (A fixed grid that first lists the noted units, so that no
// block finds none, was slower: the list's latency is longer than what the empty
// blocks take.)
#include "../../include/attn.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;

// A part's sums as they count: none where it admits no key, and they may not have been written (a query
// of NaN has the same max, but a sum of NaN, which has to reach the output).
__device__ __forceinline__ bool admits_none(float2 ml) { return ml.x == -INFINITY && ml.y == 0.f; }

// Load where they stand: the compiler would put loads of sums that may not count behind their conditions.
__device__ __forceinline__ float4 load_now(const float4 *p) {
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float2 load_now(const float2 *p) {
    float2 v;
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}

template <typename Tout>
__device__ __forceinline__ void store_lse(const PartsMergeParams &p, int64_t head, int64_t token, float mx, float sum) {
    if (p.lse) p.lse[head * p.n_q + token] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * kLn2;
}

// Units of 16 rows at most (over the cache): a warp a row, D / 32 columns a lane.  One sequence's key head is
// cut over up to 19 blocks: kBatch parts at a time, all loaded before any is added, those that are left out
// as zeros.  (33 parts of 8 units 6.3 us; 8.4 with a loop that the compiler unrolled by four.)
template <typename Tout, int D>
__global__ void __launch_bounds__(32 * kWarps) row_merge_kernel(const PartsMergeParams p) {
    constexpr int kCols = D / 32, kBatch = 4;
    pdl_trigger();
    pdl_wait();
    const CutUnit u = p.parts.cut[blockIdx.x];
    const int first = blockIdx.x;
    if (u.last <= first) return;
    const int lane = threadIdx.x & 31, d = lane * kCols, r = blockIdx.y * kWarps + (threadIdx.x >> 5), row = u.base + r;
    if (r >= p.rows || row >= u.rows) return;
    auto slot = [&](int b) { return (int64_t)(b == first ? 2 * b + 1 : 2 * b) * p.rows + r; };
    float mx = -INFINITY, sum = 0.f, acc[kCols];
    for (int b = first + lane; b <= u.last; b += 32) mx = fmaxf(mx, p.parts.ml[slot(b)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
    for (int j = 0; j < kCols; ++j) acc[j] = 0.f;
    for (int b0 = first; b0 <= u.last; b0 += kBatch) {
        float2 ml[kBatch];
        float v[kBatch][kCols];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t at = slot(min(b0 + k, u.last));
            ml[k] = load_now(p.parts.ml + at);
            const float *part = p.parts.o + at * D + d;
            if constexpr (kCols == 4) *reinterpret_cast<float4 *>(v[k]) = load_now(reinterpret_cast<const float4 *>(part));
            else *reinterpret_cast<float2 *>(v[k]) = load_now(reinterpret_cast<const float2 *>(part));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool none = b0 + k > u.last || admits_none(ml[k]);
            const float f = none ? 0.f : exp2_approx(ml[k].x - mx);
            sum = fmaf(f, none ? 0.f : ml[k].y, sum);
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = fmaf(f, none ? 0.f : v[k][j], acc[j]);
        }
    }
    const int t = row / p.group;
    const int64_t token = u.q0 + t, head = u.hk * p.group + row - t * p.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    Tout *orow = static_cast<Tout *>(p.o) + token * p.o_st + head * p.o_sh + d;
    if constexpr (kCols == 4) {
        store4(orow, make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv));
    } else {
        orow[0] = from_f32<Tout>(acc[0] * inv);
        orow[1] = from_f32<Tout>(acc[1] * inv);
    }
    if (lane == 0) store_lse<Tout>(p, head, token, mx, sum);
}

// Units of query tiles (group_tc.cuh), in two or three parts mostly: a warp takes 64 columns of 8 rows, of which
// a lane has 4 columns of every 16, and two parts at a time.  The parts lie with four columns of 32 rows after the
// other, so that 8 rows' are a line.  (Trees of 63 drafts, 64 units cut in two or three: 8.8 us; 10.7 with a
// warp a row and parts that lie row after row.)
template <typename Tout, int D>
__global__ void __launch_bounds__(32 * kWarps) tile_merge_kernel(const PartsMergeParams p) {
    constexpr int kRows = 8, kCols = 4, kHalves = D / 64, kBatch = 2;
    pdl_trigger();
    pdl_wait();
    const CutUnit u = p.parts.cut[blockIdx.x];
    const int first = blockIdx.x;
    if (u.last <= first) return;
    const int lane = threadIdx.x & 31, task = blockIdx.y * kWarps + (threadIdx.x >> 5);
    const int d4 = 16 * (task % kHalves) + lane / kRows;  // four columns: the first ones of the lane
    const int r = kRows * (task / kHalves) + lane % kRows, tile = r / p.tile_rows, in = r - tile * p.tile_rows;
    const int row = u.base + tile * p.tile_live + in;  // of the entry
    const bool live = in < p.tile_live && row < u.rows;
    if (r >= p.rows || !__any_sync(0xffffffffu, live)) return;  // (p.rows is a multiple of 8)
    auto slot = [&](int b) { return (int64_t)(b == first ? 2 * b + 1 : 2 * b) * p.rows; };
    float mx = -INFINITY, sum = 0.f;
    float4 acc[kCols];
#pragma unroll 4
    for (int b = first; b <= u.last; ++b) mx = fmaxf(mx, p.parts.ml[slot(b) + r].x);
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b0 = first; b0 <= u.last; b0 += kBatch) {
        float2 ml[kBatch];
        float4 v[kBatch][kCols];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t at = slot(min(b0 + k, u.last));
            ml[k] = load_now(p.parts.ml + at + r);
            const float4 *part = reinterpret_cast<const float4 *>(p.parts.o + (at + (r & ~31)) * D) + (r & 31);
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[k][i] = load_now(part + 32 * (4 * i + d4));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const bool none = b0 + k > u.last || admits_none(ml[k]);
            const float f = none ? 0.f : exp2_approx(ml[k].x - mx);
            sum = fmaf(f, none ? 0.f : ml[k].y, sum);
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
                acc[i].x = fmaf(f, none ? 0.f : v[k][i].x, acc[i].x);
                acc[i].y = fmaf(f, none ? 0.f : v[k][i].y, acc[i].y);
                acc[i].z = fmaf(f, none ? 0.f : v[k][i].z, acc[i].z);
                acc[i].w = fmaf(f, none ? 0.f : v[k][i].w, acc[i].w);
            }
        }
    }
    if (!live) return;
    const int t = row / p.group;
    const int64_t token = u.q0 + t, head = u.hk * p.group + row - t * p.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    Tout *orow = static_cast<Tout *>(p.o) + token * p.o_st + head * p.o_sh + 4 * d4;
#pragma unroll
    for (int i = 0; i < kCols; ++i)
        store4(orow + 16 * i, make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
    if (d4 == 0) store_lse<Tout>(p, head, token, mx, sum);
}

template <typename Tout, int D>
cudaError_t launch_d(const PartsMergeParams &p, cudaStream_t s) {
    if (p.rows <= 16)
        return launch_pdl(row_merge_kernel<Tout, D>, dim3(p.blocks, (p.rows + kWarps - 1) / kWarps), dim3(32 * kWarps), 0, s, p);
    return launch_pdl(tile_merge_kernel<Tout, D>, dim3(p.blocks, (p.rows / 8 * (D / 64) + kWarps - 1) / kWarps), dim3(32 * kWarps), 0, s, p);
}

template <typename Tout>
cudaError_t launch_typed(const PartsMergeParams &p, cudaStream_t s) {
    return p.D == 64 ? launch_d<Tout, 64>(p, s) : launch_d<Tout, 128>(p, s);
}

}  // namespace

cudaError_t launch_parts_merge(const PartsMergeParams &p, cudaStream_t s) {
    cudaError_t e;
    switch (p.o_dtype) {
    case ATTN_F16: e = launch_typed<__half>(p, s); break;
    case ATTN_BF16: e = launch_typed<__nv_bfloat16>(p, s); break;
    default: e = launch_typed<float>(p, s); break;
    }
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace attn
