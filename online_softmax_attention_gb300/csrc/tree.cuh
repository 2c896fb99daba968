// Attention of new tokens (one, a chunk, a tree of drafts) over the paged cache.
//
// Per entry (sequence of L cached tokens, T of them new), key head and query
// row (new token, head of the group): the online-softmax recurrence over the L
// keys, a key before the new tokens always visible, a new one by the mask.
//
// Decomposition.  A unit is (entry, key head, tile of kRows query rows); its
// keys are cut in tiles of 32 (16 for rows over 256 bytes), and every block (one
// per SM; two of half the warps with a window) takes an equal stretch of all
// units' tiles (stretch.cuh).
//
// Inside a block the four warps take the stretch's tiles in turn, each with a
// ring of cp.async stages of its own (no block-wide barrier in the loop), and
// combine their (m, l, U) through shared memory at the unit's end.  16-bit
// types use mma.sync m16n8k16: with 16 query rows the contraction does 16
// operations per cached byte, far below what even that path sustains beside the
// HBM rate, and its row granularity fits a group's few rows, where tcgen05 tiles
// would be 128 rows high (entries of more rows go to group_tc.cuh).  f32 caches use
// FFMA, one key per lane.
//
// Bound: HBM, the cache rows of every sequence read once.  Rows past L are
// zero-filled by cp.async and never read from memory, so stale slots (NaN
// included) do not matter.
//
// kWindow: a sliding window with sinks (window.h).  An entry's keys are a list, the sinks and those from
// the first new token's window on, and its tiles count the list's places; the list is the same for
// all its units (its new tokens are few here; a chunk of T reads T keys more than its last row
// needs).  Mostly clusters of blocks take the units (cluster_of), which leaves no merge.  kMask: with a mask too
// (tree_masks.cu, so that the others keep their code): keys that none of a unit's rows sees are not loaded.
#pragma once

#include "../../include/attn.h"
#include <algorithm>
#include <climits>
#include <type_traits>

#include "mma.cuh"
#include "stretch.cuh"
#include "window.h"

namespace attn {

namespace {

// Warps of a block; with as many warps an SM, blocks of an SM.
constexpr int warps_of(bool window, bool f32) { return window && !f32 ? 2 : 4; }
constexpr int per_sm(bool window, bool f32) { return 4 / warps_of(window, f32); }

template <typename T, int D, bool kWindow>
struct Cfg {
    static constexpr int kWarps = warps_of(kWindow, sizeof(T) == 4), kThreads = 32 * kWarps;
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
    static_assert((kSmem + 1024 + 256) * per_sm(kWindow, sizeof(T) == 4) <= 233472, "shared memory budget");
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
    KeyList list;      // the keys
    long long tiles;   // of all its units
};

// Entry of rows [from, to), sequence s of `len` tokens (0 where there is no such sequence).
template <bool kWindow>
__device__ __forceinline__ Entry entry_of(const TreeParams &p, int from, int to, int s, int len, int rows, int keys, int turn,
                                          bool report) {
    Entry e;
    e.q0 = from;
    e.T = to - from;
    e.s = s;
    bool ok = (unsigned)e.s < (unsigned)p.c.max_seqs && e.q0 >= 0 && e.q0 <= to && to <= p.n_q;
    e.L = ok ? len : 0;
    ok = ok && e.L >= e.T && (long long)e.L <= (long long)p.c.max_pages << p.c.page_shift &&
         (!p.mask || e.T <= 64 * p.mask_words);
    if (!ok) {
        if (report) report_status(p.c.status, ATTN_EINVAL);
        e.T = 0;
    }
    e.row_tiles = (e.T * p.group + rows - 1) / rows;
    e.key_tiles = (e.L + keys - 1) / keys;
    e.list = {0, 0};
    if (kWindow && e.T > 0) {
        // (a row of a tree may see none of the new tokens)
        e.list = key_list(p.window, p.sinks, e.L - e.T + (p.mask ? 0 : 1), 1, 1);
        e.key_tiles = (e.L - e.list.shift + keys - 1) / keys;
        // whole turns of a block's warps, so that short stretches (of one turn) do not meet two units, one after
        // the other (one sequence of window 1024 in stretches: 16.5 -> 14.3 us); the tiles behind the list's end load nothing
        if (turn > 1) e.key_tiles = (e.key_tiles + turn - 1) & ~(turn - 1);
    }
    e.tiles = (long long)p.c.H * e.row_tiles * e.key_tiles;
    return e;
}

template <bool kWindow>
__device__ __forceinline__ Entry entry_at(const TreeParams &p, int i, int rows, int keys, int turn, bool report) {
    const int s = p.seqs[i], from = p.cu[i], to = p.cu[i + 1];
    return entry_of<kWindow>(p, from, to, s, (unsigned)s < (unsigned)p.c.max_seqs ? p.c.lens[s] : 0, rows, keys, turn, report);
}

// ---- attention kernel -------------------------------------------------------------

// The bits of a word that are below the nth.
__device__ __forceinline__ unsigned long long bits_below64(int n) { return n >= 64 ? ~0ull : n > 0 ? (1ull << n) - 1 : 0ull; }

// Whether new token u is visible to the entry's new token t.
__device__ __forceinline__ bool sees(const TreeParams &p, const Entry &e, int t, int u) {
    if (u < 0) return true;
    if (!p.mask) return u <= t;
    return (p.mask[(int64_t)(e.q0 + t) * p.mask_words + (u >> 6)] >> (u & 63)) & 1;
}

// Whether new token u (`key` of the entry) is visible to one of a unit's rows; `row`: the first row of the token whose mask is
// given (below 0 where the unit begins behind it).
__device__ __forceinline__ bool seen_draft(const unsigned long long *mask, int words, const RowWindow *window, int row, int rows,
                                        int group, int u, int key) {
    for (; row < rows; row += group, mask += words) {
        const RowWindow w = window[max(row, 0)];
        if (((mask[u >> 6] >> (u & 63)) & 1) && (key < w.hi || key >= w.lo)) return true;
    }
    return false;
}

// Writes one row's four columns: the output row, or the block's partial slot.
template <typename Tout>
__device__ __forceinline__ void store_out(const TreeParams &p, int token, int head, int d, float4 v) {
    store4(static_cast<Tout *>(p.o) + token * p.o_st + head * p.o_sh + d, v);
}

// A cluster's barrier, and another block's shared memory.
template <int kBlocks>
__device__ __forceinline__ void cluster_barrier() {
    if constexpr (kBlocks == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_block(uint32_t addr, int rank) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(addr), "r"(rank));
    return to;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Key tiles [t0, t1) of a unit: query rows row0 .. of key head hk.  `whole`: they, with kBlocks - 1 other
// blocks' of the cluster, are all of them, and the output's rows are written; else slot `slot`'s.
template <typename T, typename Tout, int D, bool kWindow, bool kMask, int kBlocks>
__device__ __forceinline__ void take_unit(const TreeParams &p, const Entry &e, int hk, int row0, int t0, int t1, int rank, bool whole,
                                          int slot, uint8_t *smem, RowWindow *s_window) {
    using C = Cfg<T, D, kWindow>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    constexpr int kRows = C::kRows, kKeys = C::kKeys;
    constexpr bool kMma = sizeof(T) == 2;
    uint8_t *sQ = smem + C::kRingBytes;
    float2 *s_ml = reinterpret_cast<float2 *>(sQ + C::kQBytes);  // (warps, rows): m, l
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t *ring = smem + warp * C::kStages * 2 * C::kTileBytes;
    const uint32_t ring_a = smem_addr(ring);
    const int live_rows = min(kRows, e.T * p.group - row0);
    const int ctx = e.L - e.T;  // tokens before the new ones
    // kMask: the list can hold keys that none of the rows sees (it begins as for a row that sees no draft, and a draft may be
    // in no row's window).  They may hold anything, and so are not loaded: p = 0 times a NaN of V would be NaN.  What the
    // rows see together: keys before the new tokens below `unit.hi` or from `unit.lo` on, and the bits of the first 64 new
    // ones.  Every warp has a row a lane, twice.  (Clearing them in shared memory instead took the loop over tiles 3 % in
    // 16-bit types and 2 to 8 % in f32, this 1 and 2; 64 sequences' trees of 4.)
    [[maybe_unused]] RowWindow unit = {0, 0};
    [[maybe_unused]] unsigned long long unit_drafts = 0;
    if constexpr (kMask) {
        const int t = min((row0 + lane % kRows) / p.group, e.T - 1);
        const unsigned long long *mask = p.mask + (int64_t)(e.q0 + t) * p.mask_words;
        const RowWindow w = tree_window(mask, e.T, ctx, p.window, p.sinks);
        const unsigned long long drafts = mask[0] & (~bits_below64(w.lo - ctx) | bits_below64(w.hi - ctx));
        unit = {__reduce_min_sync(0xffffffffu, w.lo), __reduce_max_sync(0xffffffffu, w.hi)};
        unit_drafts = (unsigned long long)__reduce_or_sync(0xffffffffu, (uint32_t)(drafts >> 32)) << 32 |
                      __reduce_or_sync(0xffffffffu, (uint32_t)drafts);
        if (tid < kRows) s_window[tid] = w;
        if (e.T > 64) __syncthreads();  // more new tokens: seen_draft reads the rows' windows
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

    if (kWindow && !kMask && tid < kRows) {
        const int t = min((row0 + tid) / p.group, e.T - 1);
        s_window[tid] = RowWindow{ctx + t + 1 - p.window, p.sinks};
    }
    // places [hidden0, hidden1) of the list are hidden from some row of the entry
    const int hidden0 = e.list.shift ? e.list.held : p.sinks, hidden1 = ctx + e.T - p.window - e.list.shift;
    auto hidden = [&](int row, int key) { return key < s_window[row].lo && key >= s_window[row].hi; };
    auto key_of = [&](int place) { return kWindow ? e.list.at(place) : place; };
    auto unit_sees = [&](int key) -> bool {
        if constexpr (kMask) {
            const int u = key - ctx, t = row0 / p.group;
            if (u < 0) return key < unit.hi || key >= unit.lo;
            if (u < 64) return (unit_drafts >> u) & 1;
            return seen_draft(p.mask + (int64_t)(e.q0 + t) * p.mask_words, p.mask_words, s_window, t * p.group - row0, live_rows,
                              p.group, u, key);
        }
        return true;
    };

    // this warp's tiles: t0 + warp, t0 + warp + kWarps, ...
    const int *table = p.c.table + (int64_t)e.s * p.c.table_stride;
    const int page_mask = (1 << p.c.page_shift) - 1;
    const char *kh = p.c.k + hk * p.c.b_head, *vh = p.c.v + hk * p.c.b_head;
    constexpr int kNone = -2;  // no such key, or none that is seen
    auto page_at = [&](int tile) -> int {  // the page of this lane's key of the tile
        const int key = key_of(tile * kKeys + lane);
        if constexpr (kMask) return lane < kKeys && tile < t1 && key < e.L && unit_sees(key) ? max(table[key >> p.c.page_shift], -1) : kNone;
        return lane < kKeys && tile < t1 && key < e.L ? table[key >> p.c.page_shift] : -1;
    };
    auto load = [&](int tile, int page, int stage) {
        const int key = key_of(tile * kKeys + lane);
        const bool live = (unsigned)page < (unsigned)p.c.n_pages;
        if (!live && (kMask ? page != kNone : lane < kKeys && tile < t1 && key < e.L)) report_status(p.c.status, ATTN_EINVAL);
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
        const int key0 = tile * kKeys;  // with a window, the list's place
        // the tile reaches the new tokens or the end
        const bool masked = key0 + kKeys > (kWindow ? ctx - e.list.shift : ctx) ||
                            (kWindow && hidden0 < hidden1 && key0 < hidden1 && key0 + kKeys > hidden0);
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
                            const int key = key_of(key0 + 8 * j + 2 * (lane & 3) + k);
                            if (key >= e.L || !sees(p, e, t, key - ctx) || (kWindow && hidden(8 * hf + (lane >> 2), key)))
                                sc[j][2 * hf + k] = -INFINITY;
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
            const int key = key_of(key0 + lane);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int t = min((row0 + r) / p.group, e.T - 1);
                float x = sc[r] * p.scale_log2;
                if (lane >= kKeys) x = -INFINITY;  // (lanes without a key)
                if (masked && lane < kKeys && (key >= e.L || !sees(p, e, t, key - ctx) || (kWindow && hidden(r, key))))
                    x = -INFINITY;
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
    cluster_barrier<kBlocks>();
    const uint32_t ml_a = smem_addr(s_ml), u_a = smem_addr(smem);
    for (int x = rank * kThreads + tid; x < live_rows * (D / 4); x += kBlocks * kThreads) {
        const int r = x / (D / 4), d = 4 * (x - r * (D / 4));
        // sums of the block's warps, or of the cluster's, block after block
        auto part_ml = [&](int w) -> float2 {
            if constexpr (kBlocks == 1) return s_ml[w * kRows + r];
            else return ld_cluster2(in_block(ml_a + ((w % kWarps) * kRows + r) * 8, w / kWarps));
        };
        auto part_u = [&](int w) -> float4 {
            if constexpr (kBlocks == 1)
                return *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(smem) + (w * kRows + r) * D + d);
            else return ld_cluster4(in_block(u_a + (((w % kWarps) * kRows + r) * D + d) * 4, w / kWarps));
        };
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kBlocks * kWarps; ++w) mx = fmaxf(mx, part_ml(w).x);
        const float m_use = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll(kBlocks == 1 ? kWarps : 8)
        for (int w = 0; w < kBlocks * kWarps; ++w) {
            const float2 ml = part_ml(w);
            const float f = exp2_approx(ml.x - m_use);
            const float4 v = part_u(w);
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
    cluster_barrier<kBlocks>();  // the rings and the query rows may be overwritten
}

template <typename T, typename Tout, int D, bool kWindow, bool kMask>
__global__ void __launch_bounds__(32 * warps_of(kWindow, sizeof(T) == 4), per_sm(kWindow, sizeof(T) == 4)) tree_kernel(const TreeParams p) {
    using C = Cfg<T, D, kWindow>;
    constexpr int kWarps = C::kWarps;
    constexpr int kRows = C::kRows, kKeys = C::kKeys;
    constexpr int kTurn = sizeof(T) == 2 ? kWarps : 1;  // (with a window; f32 tiles cost too much to have empty ones)
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x;
    __shared__ RowWindow s_window[kWindow ? kRows : 1];  // of the unit's rows
    pdl_trigger();
    pdl_wait();

    Stretch st;
    const bool any = find_stretch<kWarps, 0>(
        p.n, kWarps, [&](int i, bool report) { return Work{0, entry_at<kWindow>(p, i, kRows, kKeys, kTurn, report).tiles}; }, st,
        kWindow ? kWarps : 1);  // (a tile a warp at least: the same sequence 14.5 us, 20.5 with a tile a block)
    if (!any) {
        if (tid == 0) p.parts.cut[blockIdx.x].last = -1;
        return;
    }
    long long at = st.at, before = st.before;
    const long long end = st.end;
    int ei = st.entry;
    Entry e = entry_at<kWindow>(p, ei, kRows, kKeys, kTurn, false);

    while (at < end) {
        while (at >= before + e.tiles) {  // past this entry's units (empty entries too)
            before += e.tiles;
            e = entry_at<kWindow>(p, ++ei, kRows, kKeys, kTurn, false);
        }
        // the unit that tile `at` lies in, and the stretch's part [t0, t1) of its key tiles
        const int unit = (int)((at - before) / e.key_tiles);
        const int t0 = (int)(at - before - (long long)unit * e.key_tiles);
        const int t1 = (int)min((long long)e.key_tiles, t0 + end - at);
        const int hk = unit / e.row_tiles, row0 = (unit - hk * e.row_tiles) * kRows;
        at += t1 - t0;
        if (at == end && tid == 0) {  // a unit that begins here and goes on behind the stretch: noted for the merge
            const long long last = (before + (long long)(unit + 1) * e.key_tiles - 1) / st.share;
            p.parts.cut[blockIdx.x] = CutUnit{t0 == 0 ? (int)last : -1, e.q0, hk, row0, e.T * p.group, {0, 0, 0}};
        }

        // (a cut unit's slot: its later part first in the stretch, its first part last)
        take_unit<T, Tout, D, kWindow, kMask, 1>(p, e, hk, row0, t0, t1, 0, t0 == 0 && t1 == e.key_tiles, 2 * blockIdx.x + (t0 == 0), smem,
                                          s_window);
    }
}

// Over a window: a cluster takes a unit, whose tiles its blocks share and whose sums they join through their
// shared memory.  No second kernel follows.
template <typename T, typename Tout, int D, bool kMask, int kCluster>
__global__ void __cluster_dims__(kCluster, 1, 1)
    __launch_bounds__(32 * warps_of(true, sizeof(T) == 4), per_sm(true, sizeof(T) == 4)) tree_cluster_kernel(const TreeParams p) {
    using C = Cfg<T, D, true>;
    constexpr int kRows = C::kRows, kWarps = C::kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RowWindow s_window[kRows];  // of the unit's rows
    const int lane = threadIdx.x & 31, rank = blockIdx.x % kCluster, last = gridDim.x / kCluster - 1;
    pdl_trigger();
    pdl_wait();
    // Unit c: head c mod H of row tile c / H of the entries' ones, which every warp counts, by the offsets alone.
    auto take = [&](int c) -> bool {
        const int mine = c / p.c.H;
        int ei = -1, row_tile = 0, before = 0, s = 0, len = 0;
        constexpr int kAhead = 4;
        for (int i0 = 0; i0 < p.n && ei < 0; i0 += 32 * kAhead) {
            int from[kAhead], to[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + 32 * k + lane;
                from[k] = i < p.n ? p.cu[i] : 0;
                to[k] = i < p.n ? p.cu[i + 1] : 0;
            }
            if (i0 == 0) {  // (the lengths' loads go ahead of the count)
                s = lane < p.n ? p.seqs[lane] : -1;
                len = (unsigned)s < (unsigned)p.c.max_seqs ? p.c.lens[s] : 0;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int there = p.n - (i0 + 32 * k);
                if (there <= 0 || ei >= 0) break;
                const int n = from[k] >= 0 && from[k] <= to[k] && to[k] <= p.n_q ? ((to[k] - from[k]) * p.group + kRows - 1) / kRows : 0;
                int upto = min(lane + 1, there);
                if (!__all_sync(0xffffffffu, n == 1 || lane >= there)) {
                    upto = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int x = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += x;
                    }
                }
                const unsigned here = __ballot_sync(0xffffffffu, mine < before + upto);
                if (here) {
                    const int at = __ffs(here) - 1;
                    ei = i0 + 32 * k + at;
                    row_tile = mine - before - __shfl_sync(0xffffffffu, upto - n, at);
                }
                before += __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        if (ei < 0) return false;
        if (ei < 32) {
            s = __shfl_sync(0xffffffffu, s, ei);
            len = __shfl_sync(0xffffffffu, len, ei);
        } else {
            s = p.seqs[ei];
            len = (unsigned)s < (unsigned)p.c.max_seqs ? p.c.lens[s] : 0;
        }
        const Entry e = entry_of<true>(p, p.cu[ei], p.cu[ei + 1], s, len, kRows, C::kKeys, 1, false);
        if (row_tile >= e.row_tiles) return true;  // (the whole cluster: the entry does not fit)
        const int each = (e.key_tiles + kCluster * kWarps - 1) / (kCluster * kWarps) * kWarps;  // whole turns of the warps
        const int t0 = min(e.key_tiles, rank * each), t1 = min(e.key_tiles, t0 + each);
        take_unit<T, Tout, D, true, kMask, kCluster>(p, e, c - mine * p.c.H, row_tile * kRows, t0, t1, rank, true, 0, smem, s_window);
        return true;
    };
    int c = blockIdx.x / kCluster, end = c + 1;
    if (c == last) {
        // one more than units that offsets in order can have: reports entries that do not fit, and takes the units
        // that are more (of offsets that go back, entries that do fit are carried out)
        bool back = false;
        for (int i = threadIdx.x; i < p.n; i += C::kThreads) {
            entry_at<true>(p, i, kRows, C::kKeys, 1, rank == 0);
            back = back || p.cu[i + 1] < p.cu[i];
        }
        if (__syncthreads_or(back)) end = INT_MAX;
        else return;
    }
    for (; c < end; ++c)
        if (!take(c)) return;
}

// Units of all entries, at most.
int64_t most_units(const TreeParams &p) {
    const int64_t more = (int64_t)p.n_q * p.group / 16 + p.n, whole = (int64_t)p.n_q * ((p.group + 15) / 16);
    return p.c.H * std::min(more, whole);
}

// Blocks of a cluster over a window; 0: stretches and a merge.  As many as are resident at once (two
// blocks an SM), two at least for units of many keys; stretches where clusters would leave half of the
// blocks' places empty and their warps have 16 tiles and more.  (32 / 8 heads, D = 128, us with stretches and
// with clusters.  One sequence, windows of 64, 1024, 4096 and 8192 keys: 8.1 and 6.4, 11.7 and 7.4, 17.2 and
// 12.3, 18.9 and 18.9.  16 sequences: 9.1 and 6.4, 17.7 and 12.9, 49.4 and 44.0, 86.6 and 79.1 in clusters of
// two; 96 of one length, a block a unit: 19.7 and 17.1, 73.5 and 72.4; of 64 to 10000 tokens, window 1024: 81
// and 55, 4096: 146 and 135, 120 in clusters of two.)  f32, whose blocks fill an SM and whose
// tiles take long: clusters of few tiles a warp.  (One sequence, D = 64: 22.8 and 13.2, 23.0 and 17.9,
// window 2048: 24.4 and 24.0; two sequences, clusters of 8: 23.0 and 25.2.)
template <typename C>
int cluster_of(const TreeParams &p, bool f32) {
    constexpr int kMost = 8;
    if (p.n > 512 || most_units(p) >= 1 << 27) return 0;  // (every cluster counts the entries: 300 of them cost 3 us)
    const int64_t keys = std::min<int64_t>((int64_t)p.window + p.sinks, (int64_t)p.c.max_pages << p.c.page_shift);
    const int64_t units = most_units(p), places = f32 ? sm_count() / 2 : 2 * sm_count(), each = C::kWarps * C::kKeys;
    int size = kMost;
    while (size > 1 && units * size > places) size /= 2;
    if (f32) return keys <= 2 * size * each ? size : 0;
    if (size == 1 && keys > 34 * each) size = 2;
    return keys <= 16 * size * each || 2 * units * size > places ? size : 0;
}

// A cluster a unit.
template <typename T, typename Tout, int D, bool kMask, int kCluster>
cudaError_t launch_cluster(const TreeParams &p, cudaStream_t s) {
    using C = Cfg<T, D, true>;
    auto kern = tree_cluster_kernel<T, Tout, D, kMask, kCluster>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)(kCluster * (most_units(p) + 1))), dim3(C::kThreads), C::kSmem, s, p);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, typename Tout, int D, bool kWindow, bool kMask>
cudaError_t launch_typed(const TreeParams &p, cudaStream_t s) {
    using C = Cfg<T, D, kWindow>;
    if constexpr (kWindow) {
        switch (cluster_of<C>(p, sizeof(T) == 4)) {
        case 8: return launch_cluster<T, Tout, D, kMask, 8>(p, s);
        case 4: return launch_cluster<T, Tout, D, kMask, 4>(p, s);
        case 2: return launch_cluster<T, Tout, D, kMask, 2>(p, s);
        case 1: return launch_cluster<T, Tout, D, kMask, 1>(p, s);
        }
    }
    auto kern = tree_kernel<T, Tout, D, kWindow, kMask>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int blocks = tree_blocks(p);
    e = launch_pdl(kern, dim3(blocks), dim3(C::kThreads), C::kSmem, s, p);
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

template <typename T, typename Tout, bool kWindow, bool kMask>
cudaError_t launch_d(const TreeParams &p, cudaStream_t s) {
    return p.D == 64 ? launch_typed<T, Tout, 64, kWindow, kMask>(p, s) : launch_typed<T, Tout, 128, kWindow, kMask>(p, s);
}

template <typename T, bool kWindow, bool kMask>
cudaError_t launch_out(const TreeParams &p, cudaStream_t s) {
    if (p.o_dtype == ATTN_F32) return launch_d<T, float, kWindow, kMask>(p, s);
    return launch_d<T, T, kWindow, kMask>(p, s);
}

template <bool kWindow, bool kMask>
cudaError_t launch_tree(const TreeParams &p, cudaStream_t s) {
    switch (p.dtype) {
    case ATTN_F16: return launch_out<__half, kWindow, kMask>(p, s);
    case ATTN_BF16: return launch_out<__nv_bfloat16, kWindow, kMask>(p, s);
    default: return launch_d<float, float, kWindow, kMask>(p, s);
    }
}

}  // namespace

}  // namespace attn
