// The attention that cached tokens get from new ones (attn_weigh_args): for every token j of
// an entry, w_j += sum over its query rows (new token t, query head h) of
// exp(scale <q_th, k_j> - lse_th), where t sees j.  The rows' lse is known, so there is no
// running maximum, values are not read, and nothing is joined between blocks.
//
// Decomposition.  A unit is 32 keys of one entry with all its heads and rows, and one warp (of f32: a
// block, mostly) has all of it, so that a token's sum is in one place: no atomics, a fixed order.
// Blocks take equal stretches of all units (stretch.cuh), their warps a unit each in turn.
//
// 16-bit caches.  A warp's K rows, a key head at a time, come through a ring of cp.async stages
// of its own.  They are the A operand of mma.sync m16n8k16 (rows = keys), held in registers while
// the group's query rows pass as the B operand, eight at a time.  The order of the
// contraction over D is free, so both operands are read 16 bytes a lane: the quarter-warp's
// lanes c hold elements [32 i + 8 c, + 8) of a row as the operands' columns (2 c, 2 c + 1,
// 2 c + 8, 2 c + 9) of two steps; queries come straight from the L1.  Every lane sums
// exponentials of four keys over its columns, and lanes are joined once a unit.  f32 caches use
// FFMA, a key a lane.
//
// Bound: HBM, the K rows read once.  (More than eight rows a key head run weigh_tc.cu, but for f32, pages below
// 8 rows and groups of more than 128.)  With a window K rows that it hides from every new token are not read, but
// their units are counted and their weights pass through, so that the time goes with the sequence's length.
#include "../../include/attn.h"
#include "mma.cuh"
#include "stretch.cuh"
#include "window.h"

namespace attn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 32;  // of a unit
constexpr int kRows = 8;   // query rows at a time

template <typename T, int D>
struct Cfg {
    static constexpr bool kMma = sizeof(T) == 2;
    static constexpr int kRowBytes = D * (int)sizeof(T);
    static constexpr int kTileBytes = kKeys * kRowBytes;
    // stages of a warp's ring: 24 KiB a warp keeps 128 KiB of loads in flight per SM
    static constexpr int kStages = kMma ? 24 * 1024 / kTileBytes : 0;
    static constexpr int kRingBytes = kWarps * kStages * kTileBytes;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

struct Entry {
    int s, L, T, q0, fresh;
    int units;  // runs of kKeys tokens
};

__device__ __forceinline__ Entry entry_at(const WeighParams &p, int i, bool report) {
    Entry e;
    e.q0 = p.cu[i];
    e.T = p.cu[i + 1] - e.q0;
    e.s = p.seqs[i];
    bool ok = (unsigned)e.s < (unsigned)p.c.max_seqs && e.q0 >= 0 && e.q0 <= p.cu[i + 1] && p.cu[i + 1] <= p.n_q;
    e.L = ok ? p.c.lens[e.s] : 0;
    e.fresh = p.fresh ? p.fresh[i] : e.T;
    ok = ok && e.L >= e.T && e.L <= p.cols && (long long)e.L <= (long long)p.c.max_pages << p.c.page_shift &&
         e.fresh >= 0 && e.fresh <= e.L;
    if (!ok) {
        if (report) report_status(p.c.status, ATTN_EINVAL);
        e.L = 0;
    }
    e.units = e.T > 0 || e.fresh > 0 ? (e.L + kKeys - 1) / kKeys : 0;
    return e;
}

// Where a warp is among the stretch's units.
struct Cursor {
    long long at, before;  // unit; units before the entry's
    int ei;
    Entry e;
};

// kWide (f32): a block's warps share a unit, its rows eight at a time, and add their sums up in order.
template <typename T, int D, bool kWide>
__global__ void __launch_bounds__(kThreads, Cfg<T, D>::kMma ? 1 : 2) weigh_kernel(const WeighParams p) {
    using C = Cfg<T, D>;
    constexpr bool kMma = C::kMma;
    constexpr int kSteps = D / 32;  // 16-byte chunks of a row a lane
    constexpr int kTurn = kWide ? 1 : kWarps;  // units at a time
    static_assert(!kMma || !kWide);
    __shared__ float s_sum[kWide ? kWarps : 1][kKeys];
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    pdl_trigger();
    pdl_wait();

    // a list that has a sequence twice is refused: two warps would add to the same weights.  (The
    // sequences' bits stand where the rings will.)
    if (p.n > 1) {
        uint32_t *seen = reinterpret_cast<uint32_t *>(smem);
        for (int x = tid; x < (p.c.max_seqs + 31) / 32; x += kThreads) seen[x] = 0;
        __syncthreads();
        bool twice = false;
        for (int i = tid; i < p.n; i += kThreads) {
            const int s = p.seqs[i];
            const uint32_t bit = 1u << (s & 31);
            if ((unsigned)s < (unsigned)p.c.max_seqs) twice = twice || (atomicOr(&seen[s >> 5], bit) & bit);
        }
        if (__syncthreads_or(twice)) {
            if (blockIdx.x == 0 && tid == 0) report_status(p.c.status, ATTN_EINVAL);
            return;
        }
    }
    Stretch st;
    const bool any = find_stretch<kWarps, 0>(
        p.n, kTurn, [&](int i, bool report) { return Work{0, entry_at(p, i, report).units}; }, st);
    if (!any) return;
    Cursor now{st.at + (kWide ? 0 : warp), st.before, st.entry, entry_at(p, st.entry, false)};
    // to the entry of unit cur.at, which is one of the stretch's
    auto seek = [&](Cursor &cur) {
        while (cur.at >= cur.before + cur.e.units) {
            cur.before += cur.e.units;
            cur.e = entry_at(p, ++cur.ei, false);
        }
    };
    if (now.at >= st.end) return;
    // a run that no new token sees
    auto hidden = [&](const Entry &e, int key0) {
        return p.window && key0 + kKeys <= e.L - e.T + 1 - p.window && key0 >= p.sinks;
    };
    // offset of this lane's key's row; -1: no such key, or none that is seen
    auto row_of = [&](const Entry &e, int key0) -> long long {
        const int key = key0 + lane;
        if (key >= e.L || e.T == 0 || (p.window && key >= p.sinks && key < e.L - e.T + 1 - p.window)) return -1;
        const int page = p.c.table[(int64_t)e.s * p.c.table_stride + (key >> p.c.page_shift)];
        if ((unsigned)page < (unsigned)p.c.n_pages)
            return page * p.c.b_page + (key & ((1 << p.c.page_shift) - 1)) * p.c.b_tok;
        report_status(p.c.status, ATTN_EINVAL);
        return -1;
    };

    // the ring's next tile: key head `hk` of unit `load.at`
    Cursor load = now;
    int load_hk = 0;
    long long load_off = 0;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * C::kStages * C::kTileBytes;
    auto load_next = [&](int stage) {
        if constexpr (kMma) {
            if (load.at < st.end) {
                if (load_hk == 0) {
                    seek(load);
                    load_off = row_of(load.e, (int)(load.at - load.before) * kKeys);
                }
                constexpr int kChunks = C::kRowBytes / 16, kPer = 32 / kChunks;  // of a row; rows an instruction
                const char *kh = p.c.k + load_hk * p.c.b_head;
#pragma unroll
                for (int i = 0; i < kKeys / kPer; ++i) {
                    const int r = i * kPer + lane / kChunks, ch = lane % kChunks;
                    const long long o = __shfl_sync(0xffffffffu, load_off, r);
                    // (two rows' halves trade places, so that the reads below meet every bank once)
                    cp_async16(ring + stage * C::kTileBytes + r * C::kRowBytes + 16 * (ch ^ (4 * (r & 1))),
                               kh + (o < 0 ? 0 : o + 16 * ch), o >= 0);
                }
                if (++load_hk == p.c.H) {
                    load_hk = 0;
                    load.at += kWarps;
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) load_next(s);

    int stage = 0;
    for (; now.at < st.end; now.at += kTurn) {
        seek(now);
        const Entry &e = now.e;
        const int key0 = (int)(now.at - now.before) * kKeys, ctx = e.L - e.T, rows = e.T * p.group;
        // a run that every new token sees whole
        const bool whole = key0 + kKeys <= ctx + 1 && (!p.window || key0 >= ctx + e.T - p.window || key0 + kKeys <= p.sinks);
        auto sees = [&](int t, int key) {
            return key <= ctx + t && (!p.window || key > ctx + t - p.window || key < p.sinks);
        };
        auto token_of = [&](int r) { return key_head(r, p.group_inv); };  // of row r of a head
        // the lse of row r of the head whose rows begin at lh
        auto lse_of = [&](const float *lh, int r) -> float {
            if (r >= rows) return -INFINITY;
            const int t = token_of(r);
            return __ldg(lh + (int64_t)(r - t * p.group) * p.n_q + t);
        };
        // minus that in log2 units; a row that does not exist, or saw nothing, adds 2^-inf
        auto added = [](float x) -> float { return x == -INFINITY ? -INFINITY : -x * kLog2e; };
        // the key that this lane writes, and its weight so far
        const int mine = key0 + (kMma ? g + 8 * c : lane);
        float *const w = p.weights + (int64_t)e.s * p.weights_stride + mine;
        const float old = mine < e.L - e.fresh ? *w : 0.f;
        float sum = 0.f;
        if constexpr (kMma) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};  // keys g + 8 i
            const bool none = e.T == 0 || hidden(e, key0);
            uint4 q[kSteps];
            float l0 = 0.f, l1 = 0.f;
            // rows r0 .. of head hk: the operand's column g, and the lse of the columns 2 c, 2 c + 1
            auto queries = [&](int hk, int r0) {
                const T *qh = static_cast<const T *>(p.q) + (int64_t)e.q0 * p.q_st + (int64_t)hk * p.group * p.q_sh;
                const float *lh = p.lse + (int64_t)hk * p.group * p.n_q + e.q0;
                const int r = r0 + g, t = token_of(r);
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    q[s] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(qh + (int64_t)t * p.q_st + (r - t * p.group) * p.q_sh + 32 * s + 8 * c))
                                    : make_uint4(0, 0, 0, 0);
                l0 = lse_of(lh, r0 + 2 * c);
                l1 = lse_of(lh, r0 + 2 * c + 1);
            };
            if (!none) queries(0, 0);
            for (int hk = 0; hk < p.c.H; ++hk) {
                asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages > 1 ? C::kStages - 2 : 0) : "memory");
                __syncwarp();  // every lane's part has landed, and the stage before it has been read
                load_next(stage == 0 ? C::kStages - 1 : stage - 1);
                uint4 k[4][kSteps];
                const uint8_t *tile = smem + (warp * C::kStages + stage) * C::kTileBytes;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
                        k[i][s] = *reinterpret_cast<const uint4 *>(tile + (g + 8 * i) * C::kRowBytes + 16 * ((4 * s + c) ^ (4 * (g & 1))));
                stage = stage + 1 == C::kStages ? 0 : stage + 1;
                if (none) continue;
                for (int r0 = 0; r0 < rows; r0 += kRows) {
                    float x[2][4];
                    const float n0 = added(l0), n1 = added(l1);  // (here, where the loads have landed)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int y = 0; y < 4; ++y) x[m][y] = 0.f;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {  // 16 keys
                            const uint4 &lo = k[2 * m][s], &hi = k[2 * m + 1][s];
                            const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
                            mma16816<T>(x[m], a0, q[s].x, q[s].y);
                            mma16816<T>(x[m], a1, q[s].z, q[s].w);
                        }
                    // the next rows' loads are in flight during the exponentials
                    if (r0 + kRows < rows) queries(hk, r0 + kRows);
                    else if (hk + 1 < p.c.H) queries(hk + 1, 0);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            float pv = exp2_approx(fmaf(x[m][y], p.scale_log2, y & 1 ? n1 : n0));
                            if (!whole && !sees(token_of(r0 + 2 * c + (y & 1)), key0 + 16 * m + g + (y & 2 ? 8 : 0))) pv = 0.f;
                            acc[2 * m + (y >> 1)] += pv;
                        }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 1);
                acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 2);
            }
            sum = c == 0 ? acc[0] : c == 1 ? acc[1] : c == 2 ? acc[2] : acc[3];
        } else {
            const long long off = row_of(e, key0);
            const int runs = (rows + kRows - 1) / kRows;  // of a head's rows
            int hk = 0, run = kWide ? warp : 0;
            for (; __any_sync(0xffffffffu, off >= 0); run += kWide ? kWarps : 1) {
                while (run >= runs && hk < p.c.H) {
                    run -= runs;
                    ++hk;
                }
                if (hk == p.c.H) break;
                const int r0 = run * kRows;
                const float4 *kr = reinterpret_cast<const float4 *>(p.c.k + hk * p.c.b_head + (off < 0 ? 0 : off));
                const T *qh = static_cast<const T *>(p.q) + (int64_t)e.q0 * p.q_st + (int64_t)hk * p.group * p.q_sh;
                const float *lh = p.lse + (int64_t)hk * p.group * p.n_q + e.q0;
                float x[kRows];
                const float4 *qr[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int row = min(r0 + r, rows - 1), t = token_of(row);
                    qr[r] = reinterpret_cast<const float4 *>(qh + (int64_t)t * p.q_st + (row - t * p.group) * p.q_sh);
                    x[r] = 0.f;
                }
#pragma unroll 4
                for (int d = 0; d < D / 4; ++d) {
                    const float4 kv = off >= 0 ? __ldg(kr + d) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const float4 qv = __ldg(qr[r] + d);
                        x[r] = fmaf(qv.x, kv.x, x[r]);
                        x[r] = fmaf(qv.y, kv.y, x[r]);
                        x[r] = fmaf(qv.z, kv.z, x[r]);
                        x[r] = fmaf(qv.w, kv.w, x[r]);
                    }
                }
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float pv = exp2_approx(fmaf(x[r], p.scale_log2, added(lse_of(lh, r0 + r))));
                    if (whole || sees(token_of(r0 + r), mine)) sum += pv;
                }
            }
            if constexpr (kWide) {
                s_sum[warp][lane] = sum;
                __syncthreads();
                sum = 0.f;
                for (int x = 0; x < kWarps; ++x) sum += s_sum[x][lane];
                __syncthreads();  // (before the next unit's)
            }
        }
        if (mine < e.L && (!kWide || warp == 0)) *w = old + sum;
    }
}

template <typename T, int D, bool kWide>
cudaError_t launch_kernel(const WeighParams &p, cudaStream_t s) {
    auto kern = weigh_kernel<T, D, kWide>;
    using C = Cfg<T, D>;
    const size_t bits = p.n > 1 ? sizeof(uint32_t) * (size_t)((p.c.max_seqs + 31) / 32) : 0;
    const size_t smem = C::kRingBytes > bits ? C::kRingBytes : bits;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((C::kMma ? 1 : 2) * sm_count()), dim3(kThreads), smem, s, p);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

// f32: a block a unit where that gives all its warps rows, eight of a key head's to each.  (A chunk of 128 of
// 5000 tokens, window 1000, 32 / 8 heads: 3907 us with a warp a unit, 665 so; 64 sequences of 3000, a new
// token each: 439 and 397.)
template <typename T, int D>
cudaError_t launch_typed(const WeighParams &p, cudaStream_t s) {
    if constexpr (!Cfg<T, D>::kMma)
        if (p.c.H * ((int64_t)p.n_q * p.group / p.n / kRows + 1) >= kWarps) return launch_kernel<T, D, true>(p, s);
    return launch_kernel<T, D, false>(p, s);
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
