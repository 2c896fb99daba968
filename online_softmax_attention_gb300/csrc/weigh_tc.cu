// The attention that cached tokens get from many new ones (attn_weigh_args, weigh.cu), on the
// sm_103a tensor cores.
//
// With the key tile as the MMA's M dimension, S^T = K Q^T has a key a TMEM lane and a query
// row a column: a thread sums exp(scale s - lse) over its columns, and nothing is exchanged.
// Query rows are (token, head of the group) pairs, 128 / G tokens a tile as in group_tc.cuh.
//
// Schedule.  A unit is two 128-key tiles of an entry, which share every query tile that is loaded;
// its steps are its (key head, tile of query rows) pairs that have a row which sees one of its
// keys.  Every block takes an equal stretch of all units' steps (stretch.cuh).  A unit that is cut
// leaves its parts' 256 sums in two slots a block, and a small kernel adds them up in block order.  With a
// window, units that it hides from every new token are left out, and a unit's steps end with the last token
// that sees one of its keys.
//
// Warp roles: 0 walks the stretch and loads key tiles (TMA; pages as in group_tc.cuh), several heads
// ahead, since they come from HBM; 2 loads the query tiles, which the L2 holds; 1 issues tcgen05
// MMAs into two TMEM buffers a key tile, 4-7 and 8-11 take the exponentials of a key tile each.
// Every wait is bounded, as in fwd_tc.cu.
//
// Bound: the L2's reads.  A step takes 32 KiB of queries and, where a head has two tiles of them, 32 KiB of
// keys (D = 128) into every SM: about 0.95 us a step at the 10 TB/s that all SMs draw so, of which the
// exponentials and sums of a key tile take 0.55.  A third stage of queries does not fit the shared memory.
#include "sm100.cuh"
#include "stretch.cuh"
#include "tc.h"

namespace attn {

namespace {

using namespace sm100;

constexpr int BM = 128, BN = 128;  // keys; query rows
constexpr int kThreads = 384;
constexpr int kSegs = 4;
constexpr int kSumWarps = 8;
constexpr int kSegConsumers = 2 + kSumWarps;
constexpr int NKT = 2, kUnit = NKT * BM;  // key tiles of a unit; keys
constexpr int kBuffers = 2;  // TMEM, of a key tile

template <int D>
struct Cfg {
    static constexpr int kBoxBytes = 128 * 128;  // 128 rows x 64 columns
    static constexpr int kBoxes = D / 64;
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kKStages = D == 128 ? 4 : 8, kQStages = D == 128 ? 2 : 4;
    static constexpr int kSmemBytes = (kKStages + kQStages) * kTileBytes + 1024;
    static_assert(kSmemBytes + 4 * kSumWarps * 2 * BN + 6144 <= 232448, "shared memory budget (dynamic + static)");
    static constexpr int kRegsProducer = 88, kRegsSum = 208;
    static_assert(128 * kRegsProducer + 256 * kRegsSum <= kThreads * 168, "register split");
};

struct WeighArgs {
    CUtensorMap tq, tk;
    WeighParams p;
};

struct Entry {
    int s, L, T, q0, fresh;
    int units;       // runs of kUnit keys, without those that a window hides from every new token:
    int held, gap;   // the first `held` runs, and those behind the next `gap`
    int tiles;       // of query rows
    __device__ int unit(int i) const { return i < held ? i : i + gap; }
};

// A part of a unit: steps [j0, j0 + n), of `tiles` tiles of query rows a key head, from tile `tile0` on.
struct Seg {
    int key0, L, T, q0, s, fresh;
    int j0, n;    // n = -1: the stretch is done
    int tile0, tiles;
    int slot;     // workspace slot of a cut unit; -1: the whole unit
};

struct __align__(8) Bars {
    uint64_t q_full[4], q_empty[4], k_full[8], k_empty[8];
    uint64_t s_full[NKT][kBuffers], s_empty[NKT][kBuffers];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t mma_drain;
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ Entry entry_at(const WeighParams &p, int i, int tok, bool report) {
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
        e.L = e.T = e.fresh = 0;
    }
    e.units = e.T > 0 || e.fresh > 0 ? cdiv(e.L, kUnit) : 0;
    e.held = e.gap = 0;
    if (p.window) {
        // (without new tokens all are hidden)
        const int from = e.T > 0 ? max(0, e.L - e.T + 1 - p.window) / kUnit : e.units;
        e.held = min(e.units, e.T > 0 ? cdiv(p.sinks, kUnit) : 0);
        e.gap = max(0, from - e.held);
        e.units -= e.gap;
    }
    e.tiles = max(1, cdiv(e.T, tok));  // (without new tokens: a tile of no rows)
    return e;
}

// First tile of query rows that sees a key of run u: token key0 - ctx does.
__device__ __forceinline__ int first_tile(const Entry &e, int u, int tok) {
    return max(0, kUnit * u - (e.L - e.T)) / tok;
}

// Tiles of query rows that see a key of run u; its last key is the last one to leave a window.
__device__ __forceinline__ int tiles_of(const WeighParams &p, const Entry &e, int u, int tok) {
    int last = e.tiles;
    if (p.window && kUnit * u >= p.sinks) {
        const long long behind = (long long)kUnit * u + kUnit - 1 + p.window - (e.L - e.T);
        if (behind < e.T) last = cdiv((int)behind, tok);
    }
    return last - first_tile(e, u, tok);
}

// Steps of the entry's units, of one key head.
__device__ __forceinline__ long long head_steps(const WeighParams &p, const Entry &e, int tok) {
    const int full = p.window ? 0 : min(e.units, (e.L - e.T) / kUnit + 1);  // units that every tile sees a key of
    long long r = (long long)full * e.tiles;
    for (int i = full; i < e.units; ++i) r += tiles_of(p, e, e.unit(i), tok);
    return r;
}

constexpr long long kDrainCycles = 1ll << 31;  // post-abort wait for TMA loads and MMAs in flight
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, long long budget) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (clock64() - t0 > budget) return;
    }
}

// ---- warp 2: loads query tiles ----------------------------------------------------------

template <int D>
__device__ void query_producer(const WeighArgs &a, Bars &bars, const Seg *segs, uint32_t sQ, const Watchdog &wd) {
    using C = Cfg<D>;
    const WeighParams &p = a.p;
    const int tok = BN / p.group;
    const uint32_t q_bytes = tok * p.group * 128 * C::kBoxes;
    RingPos<C::kQStages> qr;
    auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_small(smem_u32(&bar), parity, wd));
    };
    bool ok = true;
    for (int i = 0; ok; ++i) {
        const int slot = i % kSegs;
        ok = wait(bars.seg_full[slot], (i / kSegs) & 1);
        if (!ok) break;
        const int n = segs[slot].n, tiles = segs[slot].tiles, j0 = segs[slot].j0, row0 = segs[slot].q0 + segs[slot].tile0 * tok;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bars.seg_empty[slot]));
        if (n < 0) break;
        int hk = j0 / tiles, tile = j0 - hk * tiles;
        for (int j = 0; j < n; ++j) {
            const uint32_t qs = qr.slot();
            ok = wait(bars.q_empty[qs], qr.phase() ^ 1);
            if (!ok) break;
            if (elect_one()) {
                const uint32_t bar = smem_u32(&bars.q_full[qs]);
                mbar_expect_tx(bar, q_bytes);
#pragma unroll
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sQ + qs * C::kTileBytes + b * C::kBoxBytes, &a.tq, 64 * b, hk * p.group, row0 + tile * tok, bar);
            }
            __syncwarp();
            ++qr.i;
            if (++tile == tiles) {
                tile = 0;
                ++hk;
            }
        }
    }
    if (aborting(wd) && (threadIdx.x & 31) == 0)  // the newest load of every slot may still be landing in shared memory
        for (uint32_t k = qr.i > (uint32_t)C::kQStages ? qr.i - C::kQStages : 0; k < qr.i; ++k)
            drain_wait(smem_u32(&bars.q_full[k % C::kQStages]), (k / C::kQStages) & 1, kDrainCycles);
}

// ---- warp 0: walks the stretch, loads key tiles ------------------------------------------

template <int D>
__device__ void producer(const WeighArgs &a, Bars &bars, Seg *segs, const Stretch &st, uint32_t sK, const Watchdog &wd) {
    using C = Cfg<D>;
    const WeighParams &p = a.p;
    const int lane = threadIdx.x & 31, tok = BN / p.group;
    const int psz = min(1 << p.c.page_shift, BM), pieces = BM / psz;  // of a key tile: 16 at most
    RingPos<C::kKStages> kr;
    auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_small(smem_u32(&bar), parity, wd));
    };
    int i = 0;
    auto publish = [&](const Seg &g) -> bool {
        const int slot = i % kSegs;
        if (!wait(bars.seg_empty[slot], ((i / kSegs) & 1) ^ 1)) return false;
        if (lane == 0) {
            segs[slot] = g;
            mbar_arrive(smem_u32(&bars.seg_full[slot]));
        }
        __syncwarp();
        ++i;
        return true;
    };
    Entry e = {};
    int ei = st.entry, unit = 0;
    long long u0 = st.at < st.end ? st.before : st.end;  // where the unit begins in the line
    bool fresh = st.at < st.end, entered = false, ok = true;
    while (u0 < st.end) {
        if (!entered) {  // entry ei or the next one with units
            for (;; ++ei) {
                e = entry_at(p, ei, tok, false);
                if (e.units > 0) break;
            }
            entered = true;
            unit = 0;
            if (fresh) {  // the unit that the stretch begins in
                fresh = false;
                const long long off = st.at - st.before;
                const int full = p.window ? 0 : min(e.units, (e.L - e.T) / kUnit + 1);
                unit = (int)min((long long)full, off / ((long long)p.c.H * e.tiles));
                u0 += (long long)unit * p.c.H * e.tiles;
                while (unit >= full && unit < e.units) {
                    const int n = p.c.H * tiles_of(p, e, e.unit(unit), tok);
                    if (u0 + n > st.at) break;
                    u0 += n;
                    ++unit;
                }
            }
        }
        Seg g;
        g.tile0 = first_tile(e, e.unit(unit), tok);
        g.tiles = tiles_of(p, e, e.unit(unit), tok);
        const int n_unit = p.c.H * g.tiles, t0 = st.tile(st.at, u0, n_unit), t1 = st.tile(st.end, u0, n_unit);
        if (t0 < t1) {
            g.key0 = kUnit * e.unit(unit);
            g.L = e.L;
            g.T = e.T;
            g.q0 = e.q0;
            g.s = e.s;
            g.fresh = e.fresh;
            g.j0 = t0;
            g.n = t1 - t0;
            g.slot = t1 - t0 == n_unit ? -1 : 2 * (int)blockIdx.x + (t0 == 0);
            if (t0 == 0 && t1 < n_unit && lane == 0)  // begins here and goes on behind the stretch: for the merge
                p.cut[blockIdx.x] = WeighCut{st.last_block(u0, n_unit), e.s, g.key0, e.L, e.fresh, 0};
            ok = publish(g);
            if (!ok) break;
            // this lane's piece of the key tiles
            const int pos = g.key0 + lane * psz, there = min(NKT * pieces, cdiv(e.L - g.key0, psz));
            const int my_tile = lane / pieces;
            int page = 0;
            if (lane < there) {
                // (a piece that a window hides from every new token may be gone)
                const bool gone = p.window && pos >= p.sinks && pos + psz <= e.L - e.T + 1 - p.window;
                if (!gone) page = p.c.table[(int64_t)e.s * p.c.table_stride + (pos >> p.c.page_shift)];
                if ((unsigned)page >= (unsigned)p.c.n_pages) {
                    report_status(p.c.status, ATTN_EINVAL);
                    page = 0;  // any page that exists: the entry's weights are reported as invalid
                }
            }
            for (int hk = t0 / g.tiles; hk <= (t1 - 1) / g.tiles; ++hk) {
                for (int t = 0; t < NKT && t * pieces < there && ok; ++t) {
                    const uint32_t ks = kr.slot();
                    ok = wait(bars.k_empty[ks], kr.phase() ^ 1);
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&bars.k_full[ks]);
                    if (lane == 0) mbar_expect_tx(bar, min(pieces, there - t * pieces) * psz * 128 * C::kBoxes);
                    __syncwarp();
                    if (lane < there && my_tile == t) {
#pragma unroll
                        for (int b = 0; b < C::kBoxes; ++b)
                            tma_load_4d(sK + ks * C::kTileBytes + b * C::kBoxBytes + (lane - t * pieces) * psz * 128, &a.tk, 64 * b,
                                        pos & ((1 << p.c.page_shift) - 1), hk, page, bar);
                    }
                    __syncwarp();
                    ++kr.i;
                }
                if (!ok) break;
            }
            if (!ok) break;
        }
        u0 += n_unit;
        if (++unit == e.units) {
            ++ei;
            entered = false;
        }
    }
    if (ok) {
        Seg g;
        g.n = -1;
        publish(g);
    }
    if (aborting(wd) && lane == 0) {
        // the newest load of every slot may still be landing in shared memory
        for (uint32_t k = kr.i > (uint32_t)C::kKStages ? kr.i - C::kKStages : 0; k < kr.i; ++k)
            drain_wait(smem_u32(&bars.k_full[k % C::kKStages]), (k / C::kKStages) & 1, kDrainCycles);
    }
}

// ---- warp 1: MMA issuer (the whole warp, one elected lane issuing) ----------------------

// Query rows of tile `tile` of the part's, from the unit's first one on.
__device__ __forceinline__ int rows_of(const Seg &g, int tile, int tok, int group) {
    return max(0, min(tok, g.T - (g.tile0 + tile) * tok)) * group;
}

template <int D, bool kBF16>
__device__ void mma_issuer(const WeighParams &p, Bars &bars, const Seg *segs, uint32_t sK, uint32_t sQ, uint32_t tmem,
                           const Watchdog &wd) {
    using C = Cfg<D>;
    const int tok = BN / p.group;
    RingPos<C::kKStages> kr;
    RingPos<C::kQStages> qr;
    RingPos<kBuffers> sr[NKT];
    const uint64_t k_desc = sdesc_sw128(sK, 16, 1024), q_desc = sdesc_sw128(sQ, 16, 1024);
    auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_small(smem_u32(&bar), parity, wd));
    };
    for (int i = 0;; ++i) {
        const int slot = i % kSegs;
        if (!wait(bars.seg_full[slot], (i / kSegs) & 1)) return;
        const Seg g = segs[slot];
        const int n = g.n;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bars.seg_empty[slot]));
        if (n < 0) return;
        const int key_tiles = min(NKT, cdiv(g.L - g.key0, BM));
        int tile = g.j0 % g.tiles;
        for (int j = 0; j < n; ++j) {
            const uint32_t qs = qr.slot();
            const bool first = j == 0 || tile == 0, last = tile + 1 == g.tiles || j + 1 == n;  // of the key tiles
            // whole MMA steps of 16 rows; a full tile's 128 columns, whatever G is: all of them are read
            const int rows = rows_of(g, tile, tok, p.group);
            const uint32_t id = idesc_f16(kBF16, BM, 0, 0) | ((uint32_t)(rows == tok * p.group ? BN / 8 : 2 * max(1, cdiv(rows, 16))) << 17);
            if (!wait(bars.q_full[qs], qr.phase())) return;
#pragma unroll
            for (int t = 0; t < NKT; ++t) {
                if (t >= key_tiles) break;
                const uint32_t ks = (kr.i + t) % C::kKStages, sb = sr[t].slot();
                if (first && !wait(bars.k_full[ks], ((kr.i + t) / C::kKStages) & 1)) return;
                if (!wait(bars.s_empty[t][sb], sr[t].phase() ^ 1)) return;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t kd = k_desc + sdesc_step(ks * C::kTileBytes), qd = q_desc + sdesc_step(qs * C::kTileBytes);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = sdesc_step((kk >> 2) * C::kBoxBytes + (kk & 3) * 32);
                        mma_ss(tmem + BN * (kBuffers * t + sb), kd + off, qd + off, id, kk > 0);
                    }
                    tc_commit(smem_u32(&bars.s_full[t][sb]));
                    if (t == key_tiles - 1) tc_commit(smem_u32(&bars.q_empty[qs]));
                    if (last) tc_commit(smem_u32(&bars.k_empty[ks]));
                }
                __syncwarp();
                ++sr[t].i;
            }
            ++qr.i;
            if (last) kr.i += key_tiles;
            if (++tile == g.tiles) tile = 0;
        }
    }
}

// ---- warps 4-11: exponentials and sums, a key tile a warpgroup ---------------------------

__device__ void sum_wg(const WeighArgs &a, Bars &bars, const Seg *segs, float *stats, uint32_t tmem, const Watchdog &wd) {
    const WeighParams &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wg = (warp - 4) >> 2, quarter = warp & 3, row = 32 * quarter + lane;  // key row
    const int tok = BN / p.group;
    // the query rows whose lse this lane puts into its warp's copy: tokens within a tile, offsets of their heads
    // (every warp has a copy, so that none waits for another)
    constexpr int kPer = BN / 32;
    int my_tok[kPer], my_head[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int r = lane + 32 * k;
        my_tok[k] = r / p.group;
        my_head[k] = r - my_tok[k] * p.group;
        if (my_tok[k] >= tok) my_tok[k] = -1;  // (G does not divide 128)
    }
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    stats += (warp - 4) * 2 * BN;
    uint32_t step = 0;  // of this warpgroup
    for (int i = 0;; ++i) {
        const int slot = i % kSegs;
        bool ok = mbar_wait_small(smem_u32(&bars.seg_full[slot]), (i / kSegs) & 1, wd);
        if (!__all_sync(0xffffffffu, ok)) return;
        const Seg g = segs[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.seg_empty[slot]));
        if (g.n < 0) return;
        const int key0 = g.key0 + BM * wg, key = key0 + row, ctx = g.L - g.T;
        if (key0 >= g.L) continue;  // (the unit has one key tile)
        // the key's weight so far
        float *const w = p.weights + (int64_t)g.s * p.weights_stride + key;
        const bool writes = g.slot < 0 && key < g.L;
        const float old = writes && key < g.L - g.fresh ? *w : 0.f;
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        int hk = g.j0 / g.tiles, tile = g.j0 - hk * g.tiles;
        // the lse of this lane's rows of a step, as it is: nothing waits for the loads before the next step
        auto fetch = [&](int hk, int tile, float (&x)[kPer]) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int t = (g.tile0 + tile) * tok + my_tok[k];
                x[k] = my_tok[k] >= 0 && t < g.T ? __ldg(p.lse + (int64_t)(hk * p.group + my_head[k]) * p.n_q + g.q0 + t) : -INFINITY;
            }
        };
        float next[kPer];
        fetch(hk, tile, next);
        for (int j = 0; j < g.n; ++j, ++step) {
            // minus the lse in log2 units; a row that does not exist, or saw nothing, adds 2^-inf
            float *sb = stats + (step & 1) * BN;
#pragma unroll
            for (int k = 0; k < kPer; ++k) sb[lane + 32 * k] = next[k] == -INFINITY ? -INFINITY : -next[k] * kLog2e;
            __syncwarp();
            const int t0 = (g.tile0 + tile) * tok, rows = rows_of(g, tile, tok, p.group);
            if (++tile == g.tiles) {
                tile = 0;
                ++hk;
            }
            if (j + 1 < g.n) fetch(hk, tile, next);  // in flight during this step
            const uint32_t buffer = step % kBuffers, at = tmem_addr(tmem, 32 * quarter, BN * (kBuffers * wg + buffer));
            ok = mbar_wait_small(smem_u32(&bars.s_full[wg][buffer]), (step / kBuffers) & 1, wd);
            if (!__all_sync(0xffffffffu, ok)) return;
            tc_fence_after();
            // a step all of whose columns see every key of the warp.  (Columns behind the tile's rows hold
            // zeros, and their lse is infinite.)
            const int first = key0 + 32 * quarter, last = first + 31;
            if (t0 + tok <= g.T && last - ctx <= t0 && (!p.window || ctx + t0 + tok - p.window <= first || last < p.sinks)) {
                uint32_t r[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_x32(at + 32 * c, r[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_wait(r[c]);
                tc_fence_before();
                mbar_arrive_warp(smem_u32(&bars.s_empty[wg][buffer]));
#pragma unroll
                for (int c = 0; c < BN / 4; ++c) {
                    const float4 l = *reinterpret_cast<const float4 *>(sb + 4 * c);
                    const uint32_t *s = &r[c >> 3][4 * (c & 7)];
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[0]), __uint_as_float(s[1])), sc2, make_float2(l.x, l.y));
                    const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[2]), __uint_as_float(s[3])), sc2, make_float2(l.z, l.w));
                    acc[(2 * c) & 3] = __fadd2_rn(acc[(2 * c) & 3], make_float2(exp2_approx(x.x), exp2_approx(x.y)));
                    acc[(2 * c + 1) & 3] = __fadd2_rn(acc[(2 * c + 1) & 3], make_float2(exp2_approx(y.x), exp2_approx(y.y)));
                }
            } else {
                // columns [lo, hi) see the key, the tile's tokens from key - ctx on, up to the last one whose window
                // it is in; 32 columns at a time
                const int lo = max(0, min(tok, key - ctx - t0)) * p.group;
                const int hi = p.window && key >= p.sinks
                                   ? min(rows, (int)max(0ll, min((long long)tok, (long long)key + p.window - ctx - t0)) * p.group)
                                   : rows;
#pragma unroll 1
                for (int c0 = 0; c0 < rows; c0 += 32) {
                    uint32_t r[32];
                    tmem_ld_x32(at + c0, r);
                    tmem_ld_wait(r);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float x = exp2_approx(fmaf(__uint_as_float(r[c]), p.scale_log2, sb[c0 + c]));
                        acc[c & 3].x += c0 + c >= lo && c0 + c < hi ? x : 0.f;
                    }
                }
                tc_fence_before();
                mbar_arrive_warp(smem_u32(&bars.s_empty[wg][buffer]));
            }
        }
        const float2 s01 = __fadd2_rn(acc[0], acc[1]), s23 = __fadd2_rn(acc[2], acc[3]), s = __fadd2_rn(s01, s23);
        const float sum = s.x + s.y;
        if (g.slot >= 0) p.slots[(int64_t)g.slot * kUnit + BM * wg + row] = sum;
        else if (writes) *w = old + sum;
    }
}

template <int D, bool kBF16>
__global__ void __launch_bounds__(kThreads, 1) weigh_tc_kernel(const __grid_constant__ WeighArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    __shared__ Seg segs[kSegs];
    __shared__ __align__(16) float stats[kSumWarps * 2 * BN];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const uint32_t raw = smem_u32(smem_raw), sK = (raw + 1023u) & ~1023u, sQ = sK + C::kKStages * C::kTileBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Watchdog wd{a.p.watchdog_cycles, &abort_flag, a.p.c.status};

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < 4; ++s) {
            mbar_init(smem_u32(&bars.q_full[s]), 1);
            mbar_init(smem_u32(&bars.q_empty[s]), 1);
        }
        for (int s = 0; s < C::kKStages; ++s) {
            mbar_init(smem_u32(&bars.k_full[s]), 1);
            mbar_init(smem_u32(&bars.k_empty[s]), 1);
        }
        for (int t = 0; t < NKT; ++t)
            for (int s = 0; s < kBuffers; ++s) {
                mbar_init(smem_u32(&bars.s_full[t][s]), 1);
                mbar_init(smem_u32(&bars.s_empty[t][s]), 4);  // the warpgroup's warps
            }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(smem_u32(&bars.seg_full[s]), 1);
            mbar_init(smem_u32(&bars.seg_empty[s]), kSegConsumers);
        }
        mbar_init(smem_u32(&bars.mma_drain), 1);
        fence_mbar_init();
        prefetch_tmap(&a.tq);
        prefetch_tmap(&a.tk);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_base), 512);
        tmem_relinquish();
    }
    // rows of the query tiles that no load fills (G does not divide 128): zeros
    const int tok = BN / a.p.group, filled = tok * a.p.group, rest = (BN - filled) * 8;
    for (int x = threadIdx.x; x < C::kQStages * C::kBoxes * rest; x += kThreads) {
        const int box = x / rest, y = x - box * rest;
        st_shared_v4(sQ + box * C::kBoxBytes + filled * 128 + 16 * y, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    // set-up above overlaps the previous kernel on the stream; inputs are read after this
    pdl_trigger();
    pdl_wait();
    // a list that has a sequence twice is refused: two blocks would add to the same weights.  (The
    // sequences' bits stand where the key tiles will; these are read by generic loads only, and the fence
    // below orders them before the first TMA write.)
    bool refused = false;
    if (a.p.n > 1) {
        uint32_t *seen = reinterpret_cast<uint32_t *>(smem_raw + (sK - raw));
        for (int x = threadIdx.x; x < (a.p.c.max_seqs + 31) / 32; x += kThreads) seen[x] = 0;
        __syncthreads();
        bool twice = false;
        for (int i = threadIdx.x; i < a.p.n; i += kThreads) {
            const int s = a.p.seqs[i];
            const uint32_t bit = 1u << (s & 31);
            if ((unsigned)s < (unsigned)a.p.c.max_seqs) twice = twice || (atomicOr(&seen[s >> 5], bit) & bit);
        }
        refused = __syncthreads_or(twice);
        if (refused && blockIdx.x == 0 && threadIdx.x == 0) report_status(a.p.c.status, ATTN_EINVAL);
        fence_proxy_async_smem();
    }
    Stretch st;
    const bool any = !refused && find_stretch<kThreads / 32, 0>(
        a.p.n, 1, [&](int i, bool report) {
            const Entry e = entry_at(a.p, i, tok, report);
            return Work{0, a.p.c.H * head_steps(a.p, e, tok)};
        }, st);
    if (!any) {
        st.at = st.end = st.before = 0;
        st.entry = 0;
    }
    if (threadIdx.x == 0) {  // (the loading warp may put a unit there)
        a.p.cut[blockIdx.x].last = -1;
        a.p.cut[blockIdx.x].refused = refused;
    }
    __syncthreads();

    if (warp < 4) {
        regs_dec<C::kRegsProducer>();
        if (warp == 0) {
            producer<D>(a, bars, segs, st, sK, wd);  // the whole warp
        } else if (warp == 2) {
            query_producer<D>(a, bars, segs, sQ, wd);
        } else if (warp == 1) {
            mma_issuer<D, kBF16>(a.p, bars, segs, sK, sQ, tmem, wd);
            if (lane == 0 && aborting(wd)) {  // let issued MMAs finish before TMEM is freed
                tc_commit(smem_u32(&bars.mma_drain));
                drain_wait(smem_u32(&bars.mma_drain), 0, kDrainCycles);
            }
        }
    } else {
        regs_inc<C::kRegsSum>();
        sum_wg(a, bars, segs, stats, tmem, wd);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds the parts of the unit that block b of the kernel above noted as begun and cut, in block order.  The
// weights that start anew of tokens in the runs that a window hides from every new token are zeroed here.
__global__ void __launch_bounds__(kUnit) weigh_merge_kernel(const WeighParams p) {
    pdl_trigger();
    pdl_wait();
    const int first = blockIdx.x;
    if (p.window && !p.cut[first].refused)
        for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
            const Entry e = entry_at(p, i, BN / p.group, false);
            const int end = min(e.L, kUnit * (e.held + e.gap));
            for (int t = max(kUnit * e.held, e.L - e.fresh) + (int)threadIdx.x; t < end; t += kUnit)
                p.weights[(int64_t)e.s * p.weights_stride + t] = 0.f;
        }
    const WeighCut u = p.cut[first];
    if (u.last <= first) return;
    const int key = u.key0 + threadIdx.x;
    if (key >= u.L) return;
    float *w = p.weights + (int64_t)u.s * p.weights_stride + key;
    const float old = key < u.L - u.fresh ? *w : 0.f;
    float sum = p.slots[(2ll * first + 1) * kUnit + threadIdx.x];
#pragma unroll 4
    for (int b = first + 1; b <= u.last; ++b) sum += p.slots[2ll * b * kUnit + threadIdx.x];
    *w = old + sum;
}

template <int D, bool kBF16>
cudaError_t launch_typed(const WeighArgs &a, cudaStream_t s) {
    auto kern = weigh_tc_kernel<D, kBF16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(sm_count()), dim3(kThreads), Cfg<D>::kSmemBytes, s, a);
    count_launch();
    return e;
}

}  // namespace

// More than 8 query rows a key head: on the tensor cores.  (64 sequences of 3000 tokens, 32 / 8 heads,
// D = 128; weigh.cu and this kernel: 8 rows 67 us and about 70, 16 rows 80 and 70, 32 rows 141 and 70, 256
// rows 1138 and 111.)
bool weigh_on_tc(const WeighParams &p) {
    return p.dtype != ATTN_F32 && p.n_q > 0 && p.group <= BN && p.c.page_shift >= 3 &&
           (int64_t)p.n_q * p.group > (int64_t)8 * p.n && tc_device_ok();
}

size_t weigh_tc_bytes(void *workspace, WeighParams &p) {
    const size_t slots = (sizeof(float) * 2 * kUnit * (size_t)sm_count() + 255) & ~(size_t)255;
    p.slots = static_cast<float *>(workspace);
    p.cut = reinterpret_cast<WeighCut *>(static_cast<char *>(workspace) + slots);
    return slots + ((sizeof(WeighCut) * (size_t)sm_count() + 255) & ~(size_t)255);
}

cudaError_t launch_weigh_tc(const WeighParams &p, cudaStream_t s) {
    WeighArgs a;
    a.p = p;
    const uint64_t D = (uint64_t)p.D;
    const int page = 1 << p.c.page_shift;
    const uint64_t q_dims[3] = {D, (uint64_t)p.H, (uint64_t)p.n_q};
    const uint64_t q_st[2] = {(uint64_t)p.q_sh * 2, (uint64_t)p.q_st * 2};
    const uint32_t q_box[3] = {64, (uint32_t)p.group, (uint32_t)(BN / p.group)};
    const uint64_t k_dims[4] = {D, (uint64_t)page, (uint64_t)p.c.H, (uint64_t)p.c.n_pages};
    const uint64_t k_st[3] = {(uint64_t)p.c.b_tok, (uint64_t)p.c.b_head, (uint64_t)p.c.b_page};
    const uint32_t k_box[4] = {64, (uint32_t)(page < BM ? page : BM), 1, 1};
    if (!make_map(&a.tq, p.q, p.dtype, 3, q_dims, q_st, q_box) || !make_map(&a.tk, p.c.k, p.dtype, 4, k_dims, k_st, k_box))
        return cudaErrorInvalidValue;
    const bool bf16 = p.dtype == ATTN_BF16;
    cudaError_t e = p.D == 64 ? bf16 ? launch_typed<64, true>(a, s) : launch_typed<64, false>(a, s)
                              : bf16 ? launch_typed<128, true>(a, s) : launch_typed<128, false>(a, s);
    if (e != cudaSuccess) return e;
    e = launch_pdl(weigh_merge_kernel, dim3(sm_count()), dim3(kUnit), 0, s, p);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace attn
