// The windowed backward's key blocks with a sink, whose query blocks are cut into several items
// (window.h): dK and dV are the sums of the items' partial ones, in the items' order.
//
// Block (head, key block and sequences, rows): a thread has four columns of one row of dV or dK.
// Bound: the partial sums read once (2 rows of 8192 tokens, 8 key heads of D = 128: 29 MB, 11 us).
#include "../../include/attn.h"
#include "common.cuh"
#include "window.h"

namespace attn {

namespace {

constexpr int kLanes = 32;  // sequences at a time
constexpr int rows_of(int D) { return 128 / (D / 4); }

template <typename Tg, int D, int B>
__global__ void __launch_bounds__(256) sink_sum_kernel(const BwdParams p) {
    pdl_trigger();
    pdl_wait();
    if (p.sched_kv.hdr[1] == 0) return;  // offsets that do not fit
    const int h = blockIdx.x, which = threadIdx.x >> 7, x = threadIdx.x & 127;
    const int r = blockIdx.z * rows_of(D) + x / (D / 4), d = x % (D / 4) * 4;
    for (int b = blockIdx.y % kLanes; b < p.n_seq; b += kLanes) {
        int start, len;
        seq_bounds(p.cu_q, p.n_q, b, start, len);
        const int blocks = (len + B - 1) / B;
        const SinkItems sink = sink_items(blocks, p.sink_tiles, p.sink_chunk);
        if (sink.chunks == 1) continue;
        for (int t = blockIdx.y / kLanes; t < sink.tiles; t += gridDim.y / kLanes) {
            const int used = (blocks - t + p.sink_chunk - 1) / p.sink_chunk;  // chunks that hold a query block
            const int key = t * B + r;
            if (key >= len) continue;
            const long long slot = h * sink_slot(p.n_q, B, p.sink_tiles, p.sink_chunk) +
                                   sink_slot(start, B, p.sink_tiles, p.sink_chunk) + t * sink.chunks;
            const float *at = p.sink_parts + (slot * 2 + which) * (B * D) + r * D + d;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int c = 0; c < used; ++c) {
                const float4 v = *reinterpret_cast<const float4 *>(at + (int64_t)c * 2 * B * D);
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            const float mul = which ? p.scale : 1.f;
            store4(static_cast<Tg *>(which ? p.dk : p.dv) + (int64_t)(start + key) * (which ? p.dk_st : p.dv_st) +
                       (int64_t)h * (which ? p.dk_sh : p.dv_sh) + d,
                   make_float4(sum.x * mul, sum.y * mul, sum.z * mul, sum.w * mul));
        }
    }
}

template <typename Tg, int D>
cudaError_t launch_block(const BwdParams &p, int block, cudaStream_t s) {
    const dim3 grid(p.Hkv, kLanes * (p.sink_tiles < 64 ? p.sink_tiles : 64), block / rows_of(D));
    if (block == kSimtBlock) return launch_pdl(sink_sum_kernel<Tg, D, kSimtBlock>, grid, dim3(256), 0, s, p);
    return launch_pdl(sink_sum_kernel<Tg, D, 128>, grid, dim3(256), 0, s, p);
}

template <typename Tg>
cudaError_t launch_d(const BwdParams &p, int block, cudaStream_t s) {
    return p.D == 64 ? launch_block<Tg, 64>(p, block, s) : launch_block<Tg, 128>(p, block, s);
}

}  // namespace

cudaError_t launch_sink_sum(const BwdParams &p, int block, cudaStream_t s) {
    cudaError_t e;
    switch (p.grad_dtype) {
    case ATTN_F16: e = launch_d<__half>(p, block, s); break;
    case ATTN_BF16: e = launch_d<__nv_bfloat16>(p, block, s); break;
    default: e = launch_d<float>(p, block, s); break;
    }
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace attn
