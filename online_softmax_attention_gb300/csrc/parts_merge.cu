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

// A warp takes kRows rows at once, and of each kBatch parts, all loaded before any is added: units of 16
// rows over the cache have many parts (one sequence's key head is cut over up to 19 blocks), units of 256
// rows two or three but many rows.  Parts that are left out count as zeros.
//   kRows, kBatch = 1, 4: 33 parts of 8 units 6.3 us; 8.4 with a loop that the compiler unrolled by four
//   kRows, kBatch = 2, 2: 64 units of 256 rows in two or three parts 7.7 us; 8.2 with one row at a time
template <typename Tout, int D, int kRows, int kBatch>
__global__ void __launch_bounds__(32 * kWarps) parts_merge_kernel(const PartsMergeParams p) {
    constexpr int kCols = D / 32;
    pdl_trigger();
    pdl_wait();
    const CutUnit u = p.parts.cut[blockIdx.x];
    const int first = blockIdx.x;
    if (u.last <= first) return;
    const int lane = threadIdx.x & 31, d = lane * kCols, step = gridDim.y * kWarps;
    for (int r0 = blockIdx.y * kWarps + (threadIdx.x >> 5); r0 < p.rows; r0 += kRows * step) {
        int row[kRows];  // of the entry; -1: none
        int64_t at0[kRows];
        float mx[kRows], sum[kRows], acc[kRows][kCols];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * step, tile = r / p.tile_rows, in = r - tile * p.tile_rows;
            row[i] = u.base + tile * p.tile_live + in;
            if (r >= p.rows || in >= p.tile_live || row[i] >= u.rows) row[i] = -1;
            at0[i] = row[i] < 0 ? r0 : r;
            mx[i] = -INFINITY;
            sum[i] = 0.f;
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[i][j] = 0.f;
        }
        auto slot = [&](int b, int i) { return (int64_t)(b == first ? 2 * b + 1 : 2 * b) * p.rows + at0[i]; };
        for (int b = first + lane; b <= u.last; b += 32)
#pragma unroll
            for (int i = 0; i < kRows; ++i) mx[i] = fmaxf(mx[i], p.parts.ml[slot(b, i)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < kRows; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
        for (int b0 = first; b0 <= u.last; b0 += kBatch) {
            float2 ml[kBatch][kRows];
            float v[kBatch][kRows][kCols];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int64_t at = slot(min(b0 + k, u.last), i);
                    ml[k][i] = p.parts.ml[at];
                    const float *part = p.parts.o + at * D + d;
                    if constexpr (kCols == 4) *reinterpret_cast<float4 *>(v[k][i]) = *reinterpret_cast<const float4 *>(part);
                    else *reinterpret_cast<float2 *>(v[k][i]) = *reinterpret_cast<const float2 *>(part);
                }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    // a part that admits no key: its sums may not have been written (a query of NaN has the
                    // same max, but a sum of NaN, which has to reach the output)
                    const bool none = b0 + k > u.last || (ml[k][i].x == -INFINITY && ml[k][i].y == 0.f);
                    const float f = none ? 0.f : exp2_approx(ml[k][i].x - mx[i]);
                    sum[i] = fmaf(f, none ? 0.f : ml[k][i].y, sum[i]);
#pragma unroll
                    for (int j = 0; j < kCols; ++j) acc[i][j] = fmaf(f, none ? 0.f : v[k][i][j], acc[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (row[i] < 0) continue;
            const int t = row[i] / p.group;
            const int64_t token = u.q0 + t, head = u.hk * p.group + row[i] - t * p.group;
            const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];
            Tout *orow = static_cast<Tout *>(p.o) + token * p.o_st + head * p.o_sh + d;
            if constexpr (kCols == 4) {
                store4(orow, make_float4(acc[i][0] * inv, acc[i][1] * inv, acc[i][2] * inv, acc[i][3] * inv));
            } else {
                orow[0] = from_f32<Tout>(acc[i][0] * inv);
                orow[1] = from_f32<Tout>(acc[i][1] * inv);
            }
            if (lane == 0 && p.lse) p.lse[head * p.n_q + token] = sum[i] == 0.f ? -INFINITY : (mx[i] + __log2f(sum[i])) * kLn2;
        }
    }
}

template <typename Tout, int D>
cudaError_t launch_d(const PartsMergeParams &p, cudaStream_t s) {
    if (p.rows <= 16) {
        const dim3 grid(p.blocks, (p.rows + kWarps - 1) / kWarps);
        return launch_pdl(parts_merge_kernel<Tout, D, 1, 4>, grid, dim3(32 * kWarps), 0, s, p);
    }
    const int y = (p.rows + kWarps - 1) / kWarps;
    const dim3 grid(p.blocks, y < 16 ? y : 16);
    return launch_pdl(parts_merge_kernel<Tout, D, 2, 2>, grid, dim3(32 * kWarps), 0, s, p);
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
