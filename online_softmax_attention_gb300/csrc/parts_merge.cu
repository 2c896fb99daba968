// Merge of the partial results of units that were cut between blocks
// (stretch.cuh): with part c's row max m_c (log2 units), sum l_c and numerator
// U_c, m = max m_c, l = sum 2^(m_c - m) l_c and O = sum 2^(m_c - m) U_c / l, the
// (m, l, U) combination of the online-softmax recurrence, in block order.
//
// Block (b, y) merges rows y, y + gridDim.y, ... (times the warps) of the unit
// that block b of the attention kernel noted as begun and cut, if it did; one
// warp per row, D / 32 columns a lane.  Latency-bound: a note, the parts' (m, l),
// then the parts, a few of them at a time in flight.  (A fixed grid that first
// lists the noted units, so that no block finds none, was slower: the list's
// latency is longer than what the empty blocks take.)
#include "../../include/attn.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;

template <typename Tout, int D>
__global__ void __launch_bounds__(32 * kWarps) parts_merge_kernel(const PartsMergeParams p) {
    constexpr int kCols = D / 32;
    pdl_trigger();
    pdl_wait();
    const CutUnit u = p.parts.cut[blockIdx.x];
    const int first = blockIdx.x;
    if (u.last <= first) return;
    const int lane = threadIdx.x & 31, d = lane * kCols;
    for (int r = blockIdx.y * kWarps + (threadIdx.x >> 5); r < p.rows; r += gridDim.y * kWarps) {
        const int tile = r / p.tile_rows, in = r - tile * p.tile_rows, row = u.base + tile * p.tile_live + in;
        if (in >= p.tile_live || row >= u.rows) continue;
        auto slot = [&](int b) { return (int64_t)(b == first ? 2 * b + 1 : 2 * b) * p.rows + r; };
        float mx = -INFINITY;
        for (int b = first + lane; b <= u.last; b += 32) mx = fmaxf(mx, p.parts.ml[slot(b)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float sum = 0.f, acc[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) acc[j] = 0.f;
#pragma unroll 4
        for (int b = first; b <= u.last; ++b) {
            const float2 ml = p.parts.ml[slot(b)];
            const float *part = p.parts.o + slot(b) * D + d;
            float v[kCols];
            if constexpr (kCols == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(part);
            else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(part);
            // a part that admits no key: its sums may not have been written (a query of NaN has the
            // same max, but a sum of NaN, which has to reach the output)
            if (ml.x == -INFINITY && ml.y == 0.f) continue;
            const float f = exp2_approx(ml.x - mx);
            sum = fmaf(f, ml.y, sum);
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = fmaf(f, v[j], acc[j]);
        }
        const int t = row / p.group;
        const int64_t token = u.q0 + t, head = u.hk * p.group + row - t * p.group;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        Tout *orow = static_cast<Tout *>(p.o) + token * p.o_st + head * p.o_sh + d;
        if constexpr (kCols == 4) store4(orow, make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv));
        else {
            orow[0] = from_f32<Tout>(acc[0] * inv);
            orow[1] = from_f32<Tout>(acc[1] * inv);
        }
        if (lane == 0 && p.lse) p.lse[head * p.n_q + token] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * kLn2;
    }
}

template <typename Tout>
cudaError_t launch_typed(const PartsMergeParams &p, cudaStream_t s) {
    const int y = (p.rows + kWarps - 1) / kWarps;
    const dim3 grid(p.blocks, y < 16 ? y : 16);
    if (p.D == 64) return launch_pdl(parts_merge_kernel<Tout, 64>, grid, dim3(32 * kWarps), 0, s, p);
    return launch_pdl(parts_merge_kernel<Tout, 128>, grid, dim3(32 * kWarps), 0, s, p);
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
