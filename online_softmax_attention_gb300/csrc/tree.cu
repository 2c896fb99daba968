// Attention of new tokens (one, a chunk, a tree of drafts) over the paged cache.
//
// Per entry (sequence of L cached tokens, T of them new), key head and query
// row (new token, head of the group): the online-softmax recurrence over the L
// keys, a key before the new tokens always visible, a new one by the mask.
//
// Decomposition.  A unit is (entry, key head, tile of kRows query rows); its
// keys are cut in tiles of 32 (16 for rows over 256 bytes), and every block (one
// per SM) takes an equal stretch of all units' tiles (stretch.cuh).
//
// Inside a block the four warps take the stretch's tiles in turn, each with a
// ring of cp.async stages of its own (no block-wide barrier in the loop), and
// combine their (m, l, U) through shared memory at the unit's end.  16-bit
// types use mma.sync m16n8k16: with 16 query rows the contraction does 16
// operations per cached byte, far below what even that path sustains beside the
// HBM rate, and its row granularity fits a group's few rows, where tcgen05 tiles
// would be 128 rows high (entries of more rows go to group_tc.cu).  f32 caches use
// FFMA, one key per lane.
//
// Bound: HBM, the cache rows of every sequence read once.  Rows past L are
// zero-filled by cp.async and never read from memory, so stale slots (NaN
// included) do not matter.
#include "../../include/attn.h"
#include <type_traits>

#include "stretch.cuh"

namespace attn {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

template <typename T, int D>
struct Cfg {
    static constexpr int kRows = 16;
    static constexpr int kRowBytes = D * (int)sizeof(T);
    static constexpr int kKeys = kRowBytes > 256 ? 16 : 32;  // keys of a tile
    static constexpr int kChunks = kRowBytes / 16;          // 16-byte chunks of a row
    static constexpr int kTileBytes = kKeys * kRowBytes;    // K or V of a tile
    // stages of a warp's ring: 48 KiB a warp keeps about 128 KiB of loads in
    // flight per SM (the HBM rate times its latency needs about 50)
    static constexpr int kStages = 48 * 1024 / (2 * kTileBytes) >= 6 ? 6 : 48 * 1024 / (2 * kTileBytes) >= 3 ? 3 : 2;
    static constexpr int kRingBytes = kWarps * kStages * 2 * kTileBytes;
    static constexpr int kMergeBytes = kWarps * kRows * D * 4;  // the warps' U, over the rings
    static_assert(kMergeBytes <= kRingBytes, "the rings hold the warps' sums at a unit's end");
    static constexpr int kQBytes = kRows * kRowBytes;
    static constexpr int kSmem = kRingBytes + kQBytes + kWarps * kRows * 8;
    static_assert(kSmem + 1024 <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (sizeof(T) == 2) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    } else {
        __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    }
}

// ---- the entries ----------------------------------------------------------------

struct Entry {
    int s, L, T, q0;   // sequence, cached tokens, new tokens, first query row
    int row_tiles, key_tiles;
    long long tiles;   // of all its units
};

__device__ __forceinline__ Entry entry_at(const TreeParams &p, int i, int rows, int keys, bool report) {
    Entry e;
    e.q0 = p.cu[i];
    e.T = p.cu[i + 1] - e.q0;
    e.s = p.seqs[i];
    bool ok = (unsigned)e.s < (unsigned)p.c.max_seqs && e.q0 >= 0 && e.q0 <= p.cu[i + 1] && p.cu[i + 1] <= p.n_q;
    e.L = ok ? p.c.lens[e.s] : 0;
    ok = ok && e.L >= e.T && (long long)e.L <= (long long)p.c.max_pages << p.c.page_shift &&
         (!p.mask || e.T <= 64 * p.mask_words);
    if (!ok) {
        if (report) report_status(p.c.status, ATTN_EINVAL);
        e.T = 0;
    }
    e.row_tiles = (e.T * p.group + rows - 1) / rows;
    e.key_tiles = (e.L + keys - 1) / keys;
    e.tiles = (long long)p.c.H * e.row_tiles * e.key_tiles;
    return e;
}

// ---- attention kernel -------------------------------------------------------------

// Whether new token u is visible to the entry's new token t.
__device__ __forceinline__ bool sees(const TreeParams &p, const Entry &e, int t, int u) {
    if (u < 0) return true;
    if (!p.mask) return u <= t;
    return (p.mask[(int64_t)(e.q0 + t) * p.mask_words + (u >> 6)] >> (u & 63)) & 1;
}

// Writes one row's four columns: the output row, or the block's partial slot.
template <typename Tout>
__device__ __forceinline__ void store_out(const TreeParams &p, int token, int head, int d, float4 v) {
    store4(static_cast<Tout *>(p.o) + token * p.o_st + head * p.o_sh + d, v);
}

template <typename T, typename Tout, int D>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const TreeParams p) {
    using C = Cfg<T, D>;
    constexpr int kRows = C::kRows, kKeys = C::kKeys;
    constexpr bool kMma = sizeof(T) == 2;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *sQ = smem + C::kRingBytes;
    float2 *s_ml = reinterpret_cast<float2 *>(sQ + C::kQBytes);  // (warps, rows): m, l
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t *ring = smem + warp * C::kStages * 2 * C::kTileBytes;
    const uint32_t ring_a = smem_addr(ring);
    pdl_trigger();
    pdl_wait();

    Stretch st;
    const bool any = find_stretch<kWarps, 0>(
        p.n, kWarps, [&](int i, bool report) { return Work{0, entry_at(p, i, kRows, kKeys, report).tiles}; }, st);
    if (!any) {
        if (tid == 0) p.parts.cut[blockIdx.x].last = -1;
        return;
    }
    long long at = st.at, before = st.before;
    const long long end = st.end;
    int ei = st.entry;
    Entry e = entry_at(p, ei, kRows, kKeys, false);

    while (at < end) {
        while (at >= before + e.tiles) {  // past this entry's units (empty entries too)
            before += e.tiles;
            e = entry_at(p, ++ei, kRows, kKeys, false);
        }
        // the unit that tile `at` lies in, and the stretch's part [t0, t1) of its key tiles
        const int unit = (int)((at - before) / e.key_tiles);
        const int t0 = (int)(at - before - (long long)unit * e.key_tiles);
        const int t1 = (int)min((long long)e.key_tiles, t0 + end - at);
        const int hk = unit / e.row_tiles, row0 = (unit - hk * e.row_tiles) * kRows;
        const int live_rows = min(kRows, e.T * p.group - row0);
        const int ctx = e.L - e.T;  // tokens before the new ones
        at += t1 - t0;
        if (at == end && tid == 0) {  // a unit that begins here and goes on behind the stretch: noted for the merge
            const long long last = (before + (long long)(unit + 1) * e.key_tiles - 1) / st.share;
            p.parts.cut[blockIdx.x] = CutUnit{t0 == 0 ? (int)last : -1, e.q0, hk, row0, e.T * p.group, {0, 0, 0}};
        }

        // query rows: (token, head of the group), row-major; 16-byte chunks swizzled
        // by the row's low bits so that ldmatrix reads are conflict-free
        for (int x = tid; x < kRows * C::kChunks; x += kThreads) {
            const int r = x / C::kChunks, ch = x - r * C::kChunks;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < live_rows) {
                const int t = (row0 + r) / p.group, g = (row0 + r) - t * p.group;
                v = *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(
                        static_cast<const T *>(p.q) + (e.q0 + t) * p.q_st + (hk * p.group + g) * p.q_sh) + 16 * ch);
            }
            *reinterpret_cast<uint4 *>(sQ + r * C::kRowBytes + 16 * (ch ^ (r & 7))) = v;
        }

        // this warp's tiles: t0 + warp, t0 + warp + kWarps, ...
        const int *table = p.c.table + (int64_t)e.s * p.c.table_stride;
        const int page_mask = (1 << p.c.page_shift) - 1;
        const char *kh = p.c.k + hk * p.c.b_head, *vh = p.c.v + hk * p.c.b_head;
        auto page_at = [&](int tile) -> int {  // the page of this lane's key of the tile
            const int key = tile * kKeys + lane;
            return lane < kKeys && tile < t1 && key < e.L ? table[key >> p.c.page_shift] : -1;
        };
        auto load = [&](int tile, int page, int stage) {
            const int key = tile * kKeys + lane;
            const bool live = (unsigned)page < (unsigned)p.c.n_pages;
            if (!live && lane < kKeys && tile < t1 && key < e.L) report_status(p.c.status, ATTN_EINVAL);
            const long long off = live ? page * p.c.b_page + (key & page_mask) * p.c.b_tok : -1;
            const uint32_t dst = ring_a + stage * 2 * C::kTileBytes;
            constexpr int kPer = 32 / C::kChunks > 0 ? 32 / C::kChunks : 1;  // rows per instruction
#pragma unroll
            for (int i = 0; i < kKeys / kPer; ++i) {
                const int r = i * kPer + lane / C::kChunks, ch = lane % C::kChunks;
                const long long o = __shfl_sync(0xffffffffu, off, r);
                const uint32_t to = dst + r * C::kRowBytes + 16 * (ch ^ (r & 7));
                const long long src = o < 0 ? 0 : o + 16 * ch;
                cp_async16(to, kh + src, o >= 0);
                cp_async16(to + C::kTileBytes, vh + src, o >= 0);
            }
        };
        int next = t0 + warp;  // the next tile to load
        int page = page_at(next);
#pragma unroll
        for (int s = 0; s < C::kStages - 1; ++s) {
            if (next < t1) load(next, page, s);
            cp_async_commit();
            next += kWarps;
            page = page_at(next);
        }
        __syncthreads();  // the query rows are in shared memory

        float m[2], l[2], u[kMma ? D / 8 : 1][4];                                        // mma: rows lane / 4 and + 8
        float sm[kMma ? 1 : kRows], sl[kMma ? 1 : kRows], su[kMma ? 1 : kRows][D / 32];  // FFMA: every row
        uint32_t qf[kMma ? D / 16 : 1][4];
        const uint32_t q_a = smem_addr(sQ);
        if constexpr (kMma) {
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) u[j][k] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {  // the 16 x 16 block of columns 16 kk ..
                const int r = lane & 15, ch = 2 * kk + (lane >> 4);
                ldsm4(q_a + r * C::kRowBytes + 16 * (ch ^ (r & 7)), qf[kk]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                sm[r] = -INFINITY;
                sl[r] = 0.f;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) su[r][j] = 0.f;
            }
        }

        int stage = 0;
        for (int tile = t0 + warp; tile < t1; tile += kWarps) {
            cp_async_wait<C::kStages - 2>();
            __syncwarp();  // every lane's part of the tile has landed, and the stage before it has been read
            {
                const int free_stage = stage == 0 ? C::kStages - 1 : stage - 1;
                if (next < t1) load(next, page, free_stage);
                cp_async_commit();
                next += kWarps;
                page = page_at(next);
            }
            const uint32_t k_a = ring_a + stage * 2 * C::kTileBytes, v_a = k_a + C::kTileBytes;
            const int key0 = tile * kKeys;
            const bool masked = key0 + kKeys > ctx;  // the tile reaches the new tokens or the end
            if constexpr (kMma) {
                float sc[kKeys / 8][4];
#pragma unroll
                for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[j][k] = 0.f;
                // S = Q K^T: one ldmatrix gives the B operands of 16 keys x 16 columns
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int j = 0; j < kKeys / 16; ++j) {
                        const int r = 16 * j + (lane & 7) + ((lane >> 4) << 3), ch = 2 * kk + ((lane >> 3) & 1);
                        uint32_t b[4];
                        ldsm4(k_a + r * C::kRowBytes + 16 * (ch ^ (r & 7)), b);
                        mma16816<T>(sc[2 * j], qf[kk], b[0], b[1]);
                        mma16816<T>(sc[2 * j + 1], qf[kk], b[2], b[3]);
                    }
                // into log2 units, then the mask: lane holds rows lane / 4 (+ 8), columns 2 (lane % 4) (+ 1) of each 8
#pragma unroll
                for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[j][k] *= p.scale_log2;
                if (masked) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int t = min((row0 + 8 * hf + (lane >> 2)) / p.group, e.T - 1);
#pragma unroll
                        for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int key = key0 + 8 * j + 2 * (lane & 3) + k;
                                if (key >= e.L || !sees(p, e, t, key - ctx)) sc[j][2 * hf + k] = -INFINITY;
                            }
                    }
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int j = 0; j < kKeys / 8; ++j) mx = fmaxf(mx, fmaxf(sc[j][2 * hf], sc[j][2 * hf + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float m_new = fmaxf(m[hf], mx);
                    const float m_use = m_new == -INFINITY ? 0.f : m_new;
                    const float alpha = exp2_approx(m[hf] - m_use);
                    m[hf] = m_new;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float x = exp2_approx(sc[j][2 * hf + k] - m_use);
                            sc[j][2 * hf + k] = x;
                            sum += x;
                        }
                    l[hf] = l[hf] * alpha + sum;  // this lane's columns; joined at the unit's end
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        u[j][2 * hf] *= alpha;
                        u[j][2 * hf + 1] *= alpha;
                    }
                }
                // U += P V, P in the value type (the MMA's operand; rounded to nearest, as in the
                // other kernels): transposed ldmatrix gives the B operands of 16 keys x 16 columns
#pragma unroll
                for (int j = 0; j < kKeys / 16; ++j) {
                    const uint32_t pf[4] = {pack_pair<T>(sc[2 * j][0], sc[2 * j][1]), pack_pair<T>(sc[2 * j][2], sc[2 * j][3]),
                                            pack_pair<T>(sc[2 * j + 1][0], sc[2 * j + 1][1]),
                                            pack_pair<T>(sc[2 * j + 1][2], sc[2 * j + 1][3])};
#pragma unroll
                    for (int dd = 0; dd < D / 16; ++dd) {
                        const int r = 16 * j + (lane & 15), ch = 2 * dd + (lane >> 4);
                        uint32_t b[4];
                        ldsm4_t(v_a + r * C::kRowBytes + 16 * (ch ^ (r & 7)), b);
                        mma16816<T>(u[2 * dd], pf, b[0], b[1]);
                        mma16816<T>(u[2 * dd + 1], pf, b[2], b[3]);
                    }
                }
            } else {
                // FFMA: lane = key; the row's products with every query row
                float sc[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r) sc[r] = 0.f;
                const uint8_t *kp = ring + stage * 2 * C::kTileBytes, *vp = kp + C::kTileBytes;
#pragma unroll 4
                for (int ch = 0; ch < C::kChunks; ++ch) {
                    const float4 kv = *reinterpret_cast<const float4 *>(kp + (lane % kKeys) * C::kRowBytes + 16 * (ch ^ (lane & 7)));
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const float4 qv = *reinterpret_cast<const float4 *>(sQ + r * C::kRowBytes + 16 * (ch ^ (r & 7)));
                        sc[r] = fmaf(qv.x, kv.x, sc[r]);
                        sc[r] = fmaf(qv.y, kv.y, sc[r]);
                        sc[r] = fmaf(qv.z, kv.z, sc[r]);
                        sc[r] = fmaf(qv.w, kv.w, sc[r]);
                    }
                }
                const int key = key0 + lane;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int t = min((row0 + r) / p.group, e.T - 1);
                    float x = sc[r] * p.scale_log2;
                    if (lane >= kKeys) x = -INFINITY;  // (lanes without a key)
                    if (masked && lane < kKeys && (key >= e.L || !sees(p, e, t, key - ctx))) x = -INFINITY;
                    float mx = x;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float m_new = fmaxf(sm[r], mx);
                    const float m_use = m_new == -INFINITY ? 0.f : m_new;
                    const float alpha = exp2_approx(sm[r] - m_use);
                    sm[r] = m_new;
                    sc[r] = exp2_approx(x - m_use);
                    sl[r] = sl[r] * alpha + sc[r];  // this lane's keys
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) su[r][j] *= alpha;
                }
                // lane = columns D / 32 * lane ..
                for (int k = 0; k < kKeys; ++k) {
                    float vv[D / 32];
                    const int byte = lane * (D / 8), ch = byte >> 4;
                    const uint8_t *at_v = vp + k * C::kRowBytes + 16 * (ch ^ (k & 7)) + (byte & 15);
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) vv[j] = reinterpret_cast<const float *>(at_v)[j];
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const float pv = __shfl_sync(0xffffffffu, sc[r], k);
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) su[r][j] = fmaf(pv, vv[j], su[r][j]);
                    }
                }
            }
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
        }
        cp_async_wait<0>();
        __syncthreads();  // every warp has read its last tile: the rings take the sums

        float *s_u = reinterpret_cast<float *>(smem) + warp * kRows * D;
        if constexpr (kMma) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float sum = l[hf];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int r = 8 * hf + (lane >> 2);
                if ((lane & 3) == 0) s_ml[warp * kRows + r] = make_float2(m[hf], sum);
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<float2 *>(s_u + r * D + 8 * j + 2 * (lane & 3)) =
                        make_float2(u[j][2 * hf], u[j][2 * hf + 1]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float sum = sl[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) s_ml[warp * kRows + r] = make_float2(sm[r], sum);
#pragma unroll
                for (int j = 0; j < D / 32; ++j) s_u[r * D + lane * (D / 32) + j] = su[r][j];
            }
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == e.key_tiles;
        const int slot = 2 * blockIdx.x + (t0 == 0);  // a cut unit: its later part first in the stretch, its first part last
        for (int x = tid; x < live_rows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), d = 4 * (x - r * (D / 4));
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_ml[w * kRows + r].x);
            const float m_use = mx == -INFINITY ? 0.f : mx;
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = s_ml[w * kRows + r];
                const float f = exp2_approx(ml.x - m_use);
                const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(smem) + (w * kRows + r) * D + d);
                sum = fmaf(f, ml.y, sum);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            if (whole) {
                const int t = (row0 + r) / p.group, head = hk * p.group + (row0 + r) - t * p.group;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                store_out<Tout>(p, e.q0 + t, head, d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
                if (d == 0 && p.lse)
                    p.lse[(int64_t)head * p.n_q + e.q0 + t] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * kLn2;
            } else {
                store4(p.parts.o + ((int64_t)slot * kRows + r) * D + d, acc);
                if (d == 0) p.parts.ml[(int64_t)slot * kRows + r] = make_float2(mx, sum);
            }
        }
        __syncthreads();  // the rings and the query rows may be overwritten
    }
}

template <typename T, typename Tout, int D>
cudaError_t launch_typed(const TreeParams &p, cudaStream_t s) {
    using C = Cfg<T, D>;
    auto kern = tree_kernel<T, Tout, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int blocks = tree_blocks();
    e = launch_pdl(kern, dim3(blocks), dim3(kThreads), C::kSmem, s, p);
    count_launch();
    if (e != cudaSuccess) return e;
    PartsMergeParams m;
    m.parts = p.parts;
    m.o = p.o;
    m.lse = p.lse;
    m.o_st = p.o_st;
    m.o_sh = p.o_sh;
    m.n_q = p.n_q;
    m.group = p.group;
    m.D = p.D;
    m.o_dtype = p.o_dtype;
    m.rows = m.tile_rows = m.tile_live = C::kRows;
    m.blocks = blocks;
    return launch_parts_merge(m, s);
}

template <typename T, typename Tout>
cudaError_t launch_d(const TreeParams &p, cudaStream_t s) {
    return p.D == 64 ? launch_typed<T, Tout, 64>(p, s) : launch_typed<T, Tout, 128>(p, s);
}

template <typename T>
cudaError_t launch_out(const TreeParams &p, cudaStream_t s) {
    if (p.o_dtype == ATTN_F32) return launch_d<T, float>(p, s);
    return launch_d<T, T>(p, s);
}

}  // namespace

int tree_blocks() { return sm_count(); }

// Entries of more than 16 rows on average take the tensor-core kernel's units: the
// keys are read once for up to 256 rows (32 sequences of 2000-4000 tokens, 32 key heads'
// rows each, D = 128: 84 us; two 16-row units here: 102).  With 16 rows it is this
// kernel that is faster (75 against 84 us; 4 rows: 71 against 82), without a 128-row
// tile's latency per key tile.  Pages of fewer than 8 rows have no TMA box.
int tree_rows(const TreeParams &p) {
    const bool many = (int64_t)p.n_q * p.group > (int64_t)16 * p.n;
    return many && p.c.page_shift >= 3 && group_supported(p.dtype, p.D, p.group) ? kGroupRows : 16;
}

cudaError_t launch_tree_fwd(const TreeParams &p, cudaStream_t s) {
    if (tree_rows(p) == kGroupRows) {
        GroupParams g = {};
        g.q = p.q; g.o = p.o; g.lse = p.lse;
        g.q_st = p.q_st; g.q_sh = p.q_sh; g.o_st = p.o_st; g.o_sh = p.o_sh;
        g.n = p.n; g.n_q = p.n_q; g.H = p.H; g.Hkv = p.c.H; g.group = p.group; g.D = p.D;
        g.cu_q = p.cu;
        g.paged = 1;
        g.c = p.c;
        g.seqs = p.seqs;
        g.mask = p.mask;
        g.mask_words = p.mask_words;
        g.scale_log2 = p.scale_log2;
        g.dtype = p.dtype; g.o_dtype = p.o_dtype;
        g.parts = p.parts;
        g.status = p.c.status;
        g.watchdog_cycles = p.watchdog_cycles;
        return launch_group(g, s);
    }
    switch (p.dtype) {
    case ATTN_F16: return launch_out<__half>(p, s);
    case ATTN_BF16: return launch_out<__nv_bfloat16>(p, s);
    default: return launch_d<float, float>(p, s);
    }
}

}  // namespace attn
