// Grouped attention on the sm_103a tensor cores: the query rows of a key head
// are (token, head of the group) pairs, packed into 128-row tiles, so that a
// key tile is loaded once for all the heads that share it and short sequences
// fill the tiles.  Keys are contiguous (whole prompts, packed sequences) or pages
// of a cache (chunks and trees of new tokens).
//
// The recurrence and the warp roles are those of the ungrouped forward
// (fwd_tc.cu): warp 0 loads (TMA), warp 1 issues tcgen05 MMAs, warps 4-7 and 8-11
// do the softmax of the two 128-row tiles of a unit, which ping-pong.
// Differences:
//  * Rows.  A tile holds kTok = 128 / G tokens of all G heads (128 - kTok G rows stay
//    unused when G does not divide 128); one TMA box {64 columns, G heads, kTok
//    tokens} fills it in row order.
//  * Schedule.  A unit is (entry, key head, 2 kTok tokens); every block takes an
//    equal stretch of all units' key tiles (stretch.cuh), so no schedule is prepared
//    and long and short entries balance.  The loading warp walks the stretch and
//    hands every part of a unit to the other roles through a ring in shared memory,
//    so that none of them waits for the lengths' and offsets' loads.
//  * Keys from pages: a 128-key tile is 128 / page_size boxes (page sizes of 8 and
//    more: boxes of whole 8-row swizzle atoms), a lane each.
//  * The last key tile of an entry reaches into rows that are not its own (another
//    sequence, stale slots), which may hold NaN: their scores are masked, and the
//    softmax warps zero their V rows before the value contraction.
//
// Bound: the tensor pipe for prompts; for trees HBM up to about 128 rows a key
// head (4 * 128 operations per 2-byte key element pair), the tensor pipe beyond.
// Every wait is bounded, as in fwd_tc.cu.
//
// kWindow: a sliding window with sinks (window.h).  A unit's keys are then a list, the sinks and those
// from its first row's window on, and its tiles 128 places of that list each: the sinks share
// the window's first tile, which is put together from boxes of 16 rows (2 prompts of 14000 to 16384
// tokens, window 2048: 876 us with whole tiles of keys, the sinks' apart, 840 so).  Behind the
// loading warp everything counts places: a part's L, ctx and ends are given less the list's shift.
// Masked tiles stand at both ends of the window, so that a loop takes either kind; the kernels without
// a window (group_tc.cu) are apart from those with one (group_tc_window.cu) and keep their two loops.  So are those with a
// window and a mask (kMask, group_tc_masks.cu), which look for tokens that no row sees: with that code in one kernel, which
// short units fetch anew, 48 packed prompts took 76.5 us, 72.8 without.
#pragma once

#include <cfloat>
#include <climits>

#include "sm100.cuh"
#include "stretch.cuh"
#include "tc.h"
#include "window.h"

namespace attn {

namespace {

using namespace sm100;

constexpr int BM = 128, BN = 128;
constexpr int NQT = 2;
constexpr int kThreads = 384;
constexpr int kSegs = 4;                // ring of unit parts
constexpr int kSegConsumers = 1 + 8;    // MMA warp, softmax warps
constexpr float kRescaleThreshold = 8.f;  // log2 units, as fwd_tc.cu
// What a unit costs besides its key tiles, in key tiles (about 1.7 us each): the
// queries' loads, the masked tile, the epilogue.  (48 packed prompts of 9 to 420
// tokens, 24 packed training rows' step, 3 prompts of 5000 to 8192, trees of 63 drafts:
// 73.6 / 194.6 / 960 / 120.2 us with 0, 61.6 / 182.4 / 924 / 118.8 with 1,
// 63.1 / 183.1 / 940 / 119.0 with 2, 63.4 / 184.9 / 947 / 117.4 with 3.)
constexpr int kLead = 1;
// With a window, whose units are short and begin and end with masked tiles (2 prompts of 14000 to 16384
// tokens take 9 us a unit more than its window's tiles).  (Trees of 63 drafts, window 4096; 48 packed
// prompts, window 128: 65.6 / 76.6 us with 1, 62.1 / 78.1 with 3, 62.0 / 77.3 with 6.)
constexpr int kWindowLead = 6;
// Uncut units over a window, by a line of tiles and leads as the cut ones', or of units.
constexpr int kTileLine = 1, kUnitLine = 2;

template <int D>
struct Cfg {
    static constexpr int kBoxBytes = 128 * 128;  // 128 rows x 64 columns
    static constexpr int kBoxes = D / 64;
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kKStages = D == 128 ? 2 : 4, kVStages = D == 128 ? 3 : 4;
    static constexpr int kSmemBytes = (NQT + kKStages + kVStages) * kTileBytes + 1024;
    static_assert(kSmemBytes + 1024 <= 232448, "shared memory budget (dynamic + static)");
    static constexpr int kRegsProducer = D == 128 ? 88 : 72;
    static constexpr int kRegsSoftmax = D == 128 ? 208 : 216;
    static_assert(128 * kRegsProducer + 256 * kRegsSoftmax <= kThreads * 168, "register split");
    static constexpr int kRegsWindowProducer = 88, kRegsWindowSoftmax = 208;
    static_assert(128 * kRegsWindowProducer + 256 * kRegsWindowSoftmax <= kThreads * 168, "register split");
};

struct GroupArgs {
    CUtensorMap tq, tk, tv;
    GroupParams p;
};
struct WindowGroupArgs : GroupArgs {
    CUtensorMap tk16, tv16;  // contiguous keys: boxes of 16 rows
};
template <bool kWindow>
using GroupArgsOf = std::conditional_t<kWindow, WindowGroupArgs, GroupArgs>;

// A part of a unit: key tiles [j0, j0 + nkv) for its two query tiles.
struct PlainSeg {
    int q0, hk;       // first query row (token) of the entry; key head
    int tok[NQT];     // first token of each query tile, within the entry
    int live[NQT];    // (token, head) rows of each tile; 0: no such tile
    int n[NQT];       // key tiles each query tile scans, from j0 on
    int nkv;          // the larger one; -1: the stretch is done
    int j0;
    int L, ctx;       // keys; keys that every row sees
    int end[NQT];     // keys that any row of each tile may see
    int slot;         // workspace slot of a cut unit; -1: the whole unit
};
struct WindowSeg : PlainSeg {
    int T;            // tokens of the entry
    int sinks;
    int from[NQT];    // first place of the window of each tile's first row
};
template <bool kWindow>
using Seg = std::conditional_t<kWindow, WindowSeg, PlainSeg>;

// Of key tile j of the unit, the 16-key MMA steps that hold a key which query tile t may see: up to
// this one (one at least: an entry without keys) ...
__device__ __forceinline__ int key_steps(int left) { return min(BN / 16, max(1, (left + 15) >> 4)); }
__device__ __forceinline__ int steps_of(const PlainSeg &g, int t, int j) { return key_steps(g.end[t] - BN * j); }
// ... from this one on.
__device__ __forceinline__ int first_step(int from, int sinks, int j) {
    return BN * j < sinks ? 0 : max(0, min(BN / 16 - 1, (from - BN * j) >> 4));
}
__device__ __forceinline__ int first_step(const PlainSeg &, int, int) { return 0; }
__device__ __forceinline__ int first_step(const WindowSeg &g, int t, int j) { return first_step(g.from[t], g.sinks, j); }

struct __align__(8) Bars {
    uint64_t q_full[NQT], q_empty[NQT];
    uint64_t k_full[4], k_empty[4], v_empty[4];  // k_full: the K and V tiles of a key tile
    uint64_t s_full[NQT], p_full[NQT], o_done[NQT], o_free[NQT];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t mma_drain;  // abort path: completion of the MMAs already issued
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// ---- entries and their key tiles ---------------------------------------------------

struct Entry {
    int s, q0, T;    // sequence (cache), first query row, tokens
    int k0, L, ctx;  // first key row (contiguous), keys, keys every token sees
    int units;       // units of a key head
};

__device__ __forceinline__ bool is_ordered(const GroupParams &p) { return p.paged ? p.mask == nullptr : p.causal != 0; }

// key tiles that tokens [0, tok) of the entry need at most
__device__ __forceinline__ int tiles_to(const GroupParams &p, const Entry &e, int tok) {
    return attn::tiles_to(is_ordered(p), e.L, e.ctx, e.T, tok);
}

__device__ __forceinline__ WindowUnits window_units(const GroupParams &p, const Entry &e, int per) {
    return {is_ordered(p), e.L, e.ctx, e.T, e.units, per, p.window, p.sinks, p.paged ? min(1 << p.c.page_shift, BN) : 0};
}

// key tiles of the first n units of a key head
template <bool kWindow>
__device__ __forceinline__ long long unit_tiles(const GroupParams &p, const Entry &e, int per, int n) {
    if constexpr (kWindow) return window_units(p, e, per).before(n);
    else return attn::unit_tiles(is_ordered(p), e.L, e.ctx, e.T, e.units, per, n);
}

__device__ __forceinline__ Entry entry_at(const GroupParams &p, int i, int per, bool report) {
    Entry e;
    bool ok;
    if (p.cu_q) {
        e.q0 = p.cu_q[i];
        e.T = p.cu_q[i + 1] - e.q0;
        ok = e.q0 >= 0 && e.q0 <= p.cu_q[i + 1] && p.cu_q[i + 1] <= p.n_q;  // (e.T may have wrapped)
    } else {
        e.q0 = 0;
        e.T = p.n_q;
        ok = true;
    }
    e.s = e.k0 = 0;
    if (p.paged) {
        e.s = p.seqs[i];
        ok = ok && (unsigned)e.s < (unsigned)p.c.max_seqs;
        e.L = ok ? p.c.lens[e.s] : 0;
        ok = ok && e.L >= e.T && (long long)e.L <= (long long)p.c.max_pages << p.c.page_shift &&
             (!p.mask || e.T <= 64 * p.mask_words);
        e.ctx = e.L - e.T;
    } else {
        e.L = p.n_k;
        if (p.cu_k) {
            e.k0 = p.cu_k[i];
            e.L = p.cu_k[i + 1] - e.k0;
            ok = ok && e.k0 >= 0 && e.k0 <= p.cu_k[i + 1] && p.cu_k[i + 1] <= p.n_k;
        }
        ok = ok && (i > 0 || (e.q0 == 0 && e.k0 == 0)) && (!p.causal || e.T == e.L);
        e.ctx = p.causal ? 0 : e.L;
    }
    if (!ok) {
        if (report) report_status(p.status, ATTN_EINVAL);
        e.T = 0;
    }
    e.units = cdiv(e.T, per);
    return e;
}

template <bool kWindow>
__device__ __forceinline__ Work entry_work(const GroupParams &p, const Entry &e, int per) {
    if (kWindow && p.whole == kUnitLine) return Work{0, (long long)p.Hkv * e.units};
    return e.T > 0 ? Work{(long long)p.Hkv * e.units, p.Hkv * unit_tiles<kWindow>(p, e, per, e.units)} : Work{0, 0};
}

// Reports the missing pages from key lost[0] to lost[1] if one of `tokens` new tokens, row q0 on, sees a key between them.
__device__ __noinline__ void check_lost(const GroupParams &p, int q0, int tokens, int T, int ctx, int *lost) {
    const int lane = threadIdx.x & 31, from = lost[0], to = lost[1];
    bool seen = to > ctx;
    for (int x = lane; x < tokens; x += 32) {
        const RowWindow w = tree_window(p.mask + (int64_t)(q0 + x) * p.mask_words, T, ctx, p.window, p.sinks);
        seen = seen || from < w.hi || to > w.lo;
    }
    if (seen) report_status(p.status, ATTN_EINVAL);
    __syncwarp();
    if (lane == 0) {
        lost[0] = INT_MAX;
        lost[1] = 0;
    }
    __syncwarp();
}

// Bounded wait for outstanding TMA writes before the CTA exits after an abort.
constexpr long long kDrainCycles = 1ll << 31;
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, long long budget) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (clock64() - t0 > budget) return;
    }
}

// ---- warp 0: walks the stretch, loads ------------------------------------------------

template <int D, bool kWindow, bool kMask>
__device__ void producer(const GroupArgsOf<kWindow> &a, Bars &bars, Seg<kWindow> *segs, const Stretch &st, uint32_t sQ, uint32_t sK,
                         uint32_t sV, const Watchdog &wd) {
    using C = Cfg<D>;
    const GroupParams &p = a.p;
    const int lane = threadIdx.x & 31;
    const int tok_tile = BM / p.group, per = NQT * tok_tile;
    const uint32_t q_bytes = tok_tile * p.group * 128 * C::kBoxes;
    RingPos<C::kKStages> kr;
    RingPos<C::kVStages> vr;
    uint32_t q_uses[NQT] = {0, 0};
    bool q_pending[NQT] = {false, false};
    auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_small(smem_u32(&bar), parity, wd));
    };
    const bool ordered = is_ordered(p);
    const bool whole = kWindow && p.whole;  // a unit is the block's in whose stretch it begins
    // pages: this lane's piece of a key tile
    const int psz = p.paged ? min(1 << p.c.page_shift, BN) : BN, pieces = BN / psz;
    Entry e = {};
    KeyList list = {0, 0};  // with a window, of the unit
    // kMask: from the first to the last key of the unit's missing pages.  (Its list begins as for a row that sees no draft; a
    // page that none of its rows sees may be gone.)
    __shared__ int lost[2];
    if constexpr (kMask) {
        if (lane == 0) {
            lost[0] = INT_MAX;
            lost[1] = 0;
        }
        __syncwarp();
    }
    auto key_at = [&](int place) { return kWindow ? list.at(place) : place; };
    auto page_at = [&](int j) -> int {
        const int pos = key_at(BN * j + lane * psz);
        if (!p.paged || lane >= pieces || pos >= e.L) return 0;
        const int id = p.c.table[(int64_t)e.s * p.c.table_stride + (pos >> p.c.page_shift)];
        if ((unsigned)id < (unsigned)p.c.n_pages) return id;
        if constexpr (kMask) {  // (looked at behind the unit)
            atomicMin(&lost[0], pos);
            atomicMax(&lost[1], pos + psz);
            return 0;
        }
        report_status(p.status, ATTN_EINVAL);
        return 0;  // any page that exists: the entry's result is reported as invalid
    };

    long long u0 = st.end;  // where the unit begins in the line
    int ei = st.entry, hk = 0, unit = 0;
    bool fresh = st.at < st.end;  // the first entry, in whose middle the stretch may begin
    auto enter = [&]() {          // entry ei or the next one with work
        for (;; ++ei) {
            e = entry_at(p, ei, per, false);
            if (e.T > 0) break;
        }
        if (!fresh) return;
        fresh = false;
        if (kWindow && p.whole == kUnitLine) {
            unit = (int)(st.at - st.before);
            hk = unit / e.units;
            unit -= hk * e.units;
            u0 = st.at;
            return;
        }
        const long long per_head = st.length(st.work) / p.Hkv;
        long long off = st.at - st.before;
        hk = (int)(off / per_head);
        off -= hk * per_head;
        // the last unit that begins at or before `off`
        int lo = 0, hi = e.units;
        long long begin = 0;
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const long long len = unit_tiles<kWindow>(p, e, per, mid) + (long long)st.lead * mid;
            if (len <= off) {
                lo = mid;
                begin = len;
            } else {
                hi = mid;
            }
        }
        unit = lo;
        u0 = st.before + hk * per_head + begin;
    };
    if (fresh) u0 = st.before;
    bool ok = true;
    int i = 0;
    auto publish = [&](const Seg<kWindow> &g) -> bool {
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
    // the next unit of the line
    bool entered = false;
    auto next_unit = [&](int n_unit) {
        u0 += kWindow && p.whole == kUnitLine ? 1 : st.lead + n_unit;
        if (++unit < e.units) return;
        unit = 0;
        if (++hk < p.Hkv) return;
        hk = 0;
        ++ei;
        entered = false;
    };
#pragma unroll 1
    while (u0 < st.end) {
        if (!entered) enter();
        entered = true;
        auto tiles_of = [&](int tok) {  // key tiles that tokens [0, tok) of the entry need of the unit's
            if constexpr (kWindow) return window_units(p, e, per).tiles_to(list, tok);
            else return tiles_to(p, e, tok);
        };
        if constexpr (kWindow) list = window_units(p, e, per).list(unit);
        const int n_unit = tiles_of((unit + 1) * per);
        const int t0 = whole ? (u0 < st.at ? n_unit : 0) : st.tile(st.at, u0, n_unit);
        const int t1 = whole ? n_unit : st.tile(st.end, u0, n_unit);
        if (t0 >= t1) {
            next_unit(n_unit);
            continue;
        }
        Seg<kWindow> g;
        if constexpr (kWindow) {
            g.T = e.T;
            g.sinks = p.sinks;
#pragma unroll
            for (int t = 0; t < NQT; ++t)
                g.from[t] = e.ctx + (ordered ? unit * per + t * tok_tile + 1 : 0) - p.window - list.shift;
        }
        g.q0 = e.q0;
        g.hk = hk;
        g.L = e.L - list.shift;
        g.ctx = e.ctx - list.shift;
        g.j0 = t0;
        g.nkv = t1 - t0;
#pragma unroll
        for (int t = 0; t < NQT; ++t) {
            g.tok[t] = unit * per + t * tok_tile;
            g.live[t] = max(0, min(tok_tile, e.T - g.tok[t])) * p.group;
            g.n[t] = g.live[t] > 0 ? max(0, min(tiles_of(g.tok[t] + tok_tile), t1) - t0) : 0;
            g.end[t] = ordered ? min(g.L, g.ctx + min(g.tok[t] + tok_tile, e.T)) : g.L;
        }
        g.slot = t1 - t0 == n_unit ? -1 : 2 * (int)blockIdx.x + (t0 == 0);
        if (t0 == 0 && t1 < n_unit && lane == 0) {  // begins here and goes on behind the stretch: for the merge
            p.parts.cut[blockIdx.x] = CutUnit{st.last_block(u0, n_unit), e.q0, hk, unit * per * p.group, e.T * p.group, {0, 0, 0}};
        }
        ok = publish(g);
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < NQT; ++t) {
            if (!ok || g.n[t] == 0) continue;
            ok = wait(bars.q_empty[t], (q_uses[t] & 1) ^ 1);
            if (!ok) continue;
            if (elect_one()) {
                const uint32_t bar = smem_u32(&bars.q_full[t]);
                mbar_expect_tx(bar, q_bytes);
#pragma unroll
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sQ + t * C::kTileBytes + b * C::kBoxBytes, &a.tq, 64 * b, hk * p.group,
                                g.q0 + g.tok[t], bar);
            }
            __syncwarp();
            ++q_uses[t];
            q_pending[t] = true;
        }
        int page = page_at(t0);
        for (int j = t0; j < t1 && ok; ++j) {
            const uint32_t ks = kr.slot(), vs = vr.slot();
            ok = wait(bars.k_empty[ks], kr.phase() ^ 1) && wait(bars.v_empty[vs], vr.phase() ^ 1);
            if (!ok) break;
            const uint32_t bar = smem_u32(&bars.k_full[ks]);
            const int place0 = BN * j;
            bool mixed = false;  // contiguous keys: sinks and keys of the window
            if constexpr (kWindow) mixed = !p.paged && place0 < list.held && place0 + BN > list.held;
            if (mixed) {
                if constexpr (kWindow) {
                    if (lane == 0) mbar_expect_tx(bar, 2 * C::kTileBytes);
                    __syncwarp();
                    if (lane < BN / 16) {
                        const int row = e.k0 + list.at(place0 + 16 * lane);
                        const uint32_t off = lane * 16 * 128;
#pragma unroll
                        for (int b = 0; b < C::kBoxes; ++b) {
                            tma_load_3d(sK + ks * C::kTileBytes + b * C::kBoxBytes + off, &a.tk16, 64 * b, row, hk, bar);
                            tma_load_3d(sV + vs * C::kTileBytes + b * C::kBoxBytes + off, &a.tv16, 64 * b, row, hk, bar);
                        }
                    }
                }
            } else if (!p.paged) {
                const int key0 = key_at(place0);
                if (elect_one()) {
                    mbar_expect_tx(bar, 2 * C::kTileBytes);
#pragma unroll
                    for (int b = 0; b < C::kBoxes; ++b) {
                        tma_load_3d(sK + ks * C::kTileBytes + b * C::kBoxBytes, &a.tk, 64 * b, e.k0 + key0, hk, bar);
                        tma_load_3d(sV + vs * C::kTileBytes + b * C::kBoxBytes, &a.tv, 64 * b, e.k0 + key0, hk, bar);
                    }
                }
            } else {
                // the pieces that hold keys, one a lane
                const int there = min(pieces, cdiv(g.L - place0, psz));
                if (lane == 0) mbar_expect_tx(bar, there * psz * 128 * C::kBoxes * 2);
                __syncwarp();
                if (lane < there) {
                    const int row = key_at(place0 + lane * psz) & ((1 << p.c.page_shift) - 1);
                    const uint32_t off = lane * psz * 128;
#pragma unroll
                    for (int b = 0; b < C::kBoxes; ++b) {
                        tma_load_4d(sK + ks * C::kTileBytes + b * C::kBoxBytes + off, &a.tk, 64 * b, row, hk, page, bar);
                        tma_load_4d(sV + vs * C::kTileBytes + b * C::kBoxBytes + off, &a.tv, 64 * b, row, hk, page, bar);
                    }
                }
            }
            __syncwarp();
            ++kr.i;
            ++vr.i;
            if (j + 1 < t1) page = page_at(j + 1);
        }
        if (!ok) break;
        if constexpr (kMask) {
            __syncwarp();
            if (lost[1] > 0) check_lost(p, e.q0 + unit * per, min(per, e.T - unit * per), e.T, e.ctx, lost);
        }
        next_unit(n_unit);
    }
    if (ok) {
        Seg<kWindow> g;
        g.nkv = -1;
        publish(g);
    }
    if (aborting(wd) && lane == 0) {
        // the newest load of every slot may still be landing in shared memory
        for (uint32_t k = kr.i > (uint32_t)C::kKStages ? kr.i - C::kKStages : 0; k < kr.i; ++k)
            drain_wait(smem_u32(&bars.k_full[k % C::kKStages]), (k / C::kKStages) & 1, kDrainCycles);
#pragma unroll
        for (int t = 0; t < NQT; ++t)
            if (q_pending[t]) drain_wait(smem_u32(&bars.q_full[t]), (q_uses[t] - 1) & 1, kDrainCycles);
    }
}

// ---- warp 1: MMA issuer (the whole warp, one elected lane issuing) ----------------------

template <int D, bool kBF16, bool kWindow>
__device__ void mma_issuer(const GroupArgs &a, Bars &bars, const Seg<kWindow> *segs, uint32_t sQ, uint32_t sK, uint32_t sV,
                           uint32_t tmem, const Watchdog &wd) {
    using C = Cfg<D>;
    const GroupParams &p = a.p;
    // a negative scale negates Q in the score MMA, so the softmax always scales by |scale|
    const uint32_t negate = p.scale_log2 < 0.f ? (1u << 13) : 0u;
    const uint32_t idS = idesc_f16(kBF16, BM, BN, 0) | negate;
    auto idS_of = [&](int steps) { return idesc_f16(kBF16, BM, 0, 0) | negate | ((uint32_t)(2 * steps) << 17); };
    constexpr uint32_t idO = idesc_f16(kBF16, BM, D, 1);
    uint32_t q_ph = 0, p_ph = 0, of_ph = 3;  // bit t: the parity that query tile t waits for next
    RingPos<C::kKStages> kr;
    RingPos<C::kVStages> vr;
    const uint64_t q_desc = sdesc_sw128(sQ, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(sK, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(sV, C::kBoxBytes, 1024);
    // S_t = Q_t K^T over keys [16 from, 16 steps)
    auto issue_s = [&](int t, uint32_t kslot, int from, int steps) {
        const uint32_t id = steps - from == BN / 16 ? idS : idS_of(steps - from);
        const uint64_t qa = q_desc + sdesc_step(t * C::kTileBytes);
        const uint64_t ka = k_desc + sdesc_step(kslot * C::kTileBytes + (kWindow ? from * 2048 : 0));
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = sdesc_step((kk >> 2) * C::kBoxBytes + (kk & 3) * 32);
                mma_ss(tmem + BN * t + (kWindow ? 16 * from : 0), qa + off, ka + off, id, kk > 0);
            }
            tc_commit(smem_u32(&bars.s_full[t]));
        }
        __syncwarp();
    };
    // U_t (+)= P_t V over keys [16 from, 16 steps)
    auto issue_pv = [&](int t, uint32_t vslot, bool acc, int from, int steps) {
        const uint64_t va = v_desc + sdesc_step(vslot * C::kTileBytes);
        if (elect_one()) {
            if (steps - (kWindow ? from : 0) == BN / 16) {
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    mma_ts(tmem + 256 + D * t, tmem + BN * t + 8 * kk, va + sdesc_step(kk * 2048), idO, acc || kk > 0);
            } else {
                for (int kk = kWindow ? from : 0; kk < steps; ++kk)
                    mma_ts(tmem + 256 + D * t, tmem + BN * t + 8 * kk, va + sdesc_step(kk * 2048), idO,
                           acc || kk > (kWindow ? from : 0));
            }
        }
        __syncwarp();
    };
    auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_small(smem_u32(&bar), parity, wd));
    };
    auto commit = [&](uint64_t &bar) {
        if (elect_one()) tc_commit(smem_u32(&bar));
        __syncwarp();
    };
    for (int i = 0;; ++i) {
        const int slot = i % kSegs;
        if (!wait(bars.seg_full[slot], (i / kSegs) & 1)) return;
        const int n0 = segs[slot].n[0], n1 = segs[slot].n[1], nkv = segs[slot].nkv;
        const int j0 = segs[slot].j0, key0 = BN * j0, left0 = segs[slot].end[0] - key0, left1 = segs[slot].end[1] - key0;
        int from0 = 0, from1 = 0, sinks = 0;
        if constexpr (kWindow) {
            from0 = segs[slot].from[0];
            from1 = segs[slot].from[1];
            sinks = segs[slot].sinks;
        }
        // the steps of query tile t and the part's j-th key tile
        auto steps_at = [&](int t, int j) { return key_steps((t ? left1 : left0) - BN * j); };
        auto first_at = [&](int t, int j) { return kWindow ? first_step(t ? from1 : from0, sinks, j0 + j) : 0; };
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bars.seg_empty[slot]));
        if (nkv < 0) return;
        const uint32_t ks = kr.slot();
#pragma unroll 1
        for (int t = 0; t < NQT; ++t) {
            const int n = t ? n1 : n0;
            if (n == 0) continue;
            if (!wait(bars.q_full[t], (q_ph >> t) & 1)) return;
            q_ph ^= 1u << t;
            if (!wait(bars.k_full[ks], kr.phase())) return;
            tc_fence_after();
            issue_s(t, ks, first_at(t, 0), steps_at(t, 0));
            if (n == 1) commit(bars.q_empty[t]);
        }
        ++kr.i;
        commit(bars.k_empty[ks]);
        for (int j = 0; j < nkv; ++j) {
            const uint32_t vs = vr.slot(), nks = kr.slot();  // V_j landed with K_j
            ++vr.i;
            bool have_next_k = false;
#pragma unroll 1
            for (int t = 0; t < NQT; ++t) {
                const int n = t ? n1 : n0;
                if (j >= n) continue;
                const int steps = steps_at(t, j), next_steps = steps_at(t, j + 1);
                if (!wait(bars.p_full[t], (p_ph >> t) & 1)) return;
                p_ph ^= 1u << t;
                if (j == 0) {
                    // the previous part's epilogue of this tile has read U_t
                    if (!wait(bars.o_free[t], (of_ph >> t) & 1)) return;
                    of_ph ^= 1u << t;
                }
                tc_fence_after();
                issue_pv(t, vs, j > 0, first_at(t, j), steps);
                if (j == n - 1) commit(bars.o_done[t]);
                if (j + 1 < n) {
                    if (!have_next_k) {
                        if (!wait(bars.k_full[nks], kr.phase())) return;
                        have_next_k = true;
                        tc_fence_after();
                    }
                    issue_s(t, nks, first_at(t, j + 1), next_steps);
                    if (j + 1 == n - 1) commit(bars.q_empty[t]);
                }
            }
            commit(bars.v_empty[vs]);
            if (have_next_k) {
                ++kr.i;
                commit(bars.k_empty[nks]);
            }
        }
    }
}

// ---- warps 4-11: softmax and epilogue ------------------------------------------------------

// The 32 new-token visibility bits of keys [u, u + 32) relative to the first new
// token (u may be negative: those keys are visible) for a mask row of `words` words.
__device__ __forceinline__ uint32_t mask_bits(const unsigned long long *row, int words, int u) {
    if (u <= -32) return 0xffffffffu;
    if (u < 0) return ((1u << -u) - 1) | (uint32_t)(row[0] << -u);
    const int w = u >> 6, sh = u & 63;
    unsigned long long x = w < words ? row[w] >> sh : 0ull;
    if (sh > 32 && w + 1 < words) x |= row[w + 1] << (64 - sh);
    return (uint32_t)x;
}

// Bits of the keys [u, u + 32) that are below `lim`.
__device__ __forceinline__ uint32_t bits_below(int lim, int u) {
    const int n = lim - u;
    return n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1 : 0u;
}

// Of the places [first, first + 32), those whose keys none of `tokens` new tokens sees, a token a lane; `ctx` places before
// the new ones'.  (Apart from the loops over tiles, whose code few calls of masks need it for.)
__device__ __noinline__ uint32_t unseen_keys(const unsigned long long *mask, int words, int tokens, int T, int ctx, int window,
                                             int sinks, int first) {
    uint32_t seen = 0;
    for (int x = threadIdx.x & 31; x < tokens; x += 32) {
        const unsigned long long *row = mask + (int64_t)x * words;
        const RowWindow w = tree_window(row, T, ctx, window, sinks);
        seen |= mask_bits(row, words, first - ctx) & (~bits_below(w.lo, first) | bits_below(w.hi, first));
    }
    return ~__reduce_or_sync(0xffffffffu, seen);
}

// As store_rows_chunk (sm100.cuh) for rows at any addresses: at[k] is the address
// of row (lane & ~3) + k of the warp's 32 (null: not written); `col` the chunk's
// first column.
template <typename T>
__device__ __forceinline__ void store_rows_at(uint32_t (&u)[32], float mul, T *const (&at)[4], int col, int lane) {
    constexpr int W = sizeof(T) == 4 ? 8 : 4;  // 32-bit words per 8 values
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    uint32_t w[4][W];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (W == 8) w[k][i] = __float_as_uint(__uint_as_float(u[8 * k + i]) * mul);
            else w[k][i] = pack2(__uint_as_float(u[8 * k + 2 * i]) * mul, __uint_as_float(u[8 * k + 2 * i + 1]) * mul, kBf16);
        }
    const int gl = lane & 3;
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
        const bool upper = (gl & d) != 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & d) continue;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint32_t send = upper ? w[k][i] : w[k | d][i];
                const uint32_t recv = __shfl_xor_sync(0xffffffffu, send, d);
                if (upper) w[k][i] = recv;
                else w[k | d][i] = recv;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!at[k]) continue;
        T *dst = at[k] + col + 8 * gl;
#pragma unroll
        for (int i = 0; i < W; i += 4)
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(dst) + i) =
                make_uint4(w[k][i], w[k][i + 1], w[k][i + 2], w[k][i + 3]);
    }
}

template <int D, bool kBF16, typename Tout, bool kWindow, bool kMask>
__device__ void softmax_wg(const GroupArgs &a, Bars &bars, const Seg<kWindow> *segs, uint32_t sV, uint32_t tmem,
                           const Watchdog &wd) {
    using C = Cfg<D>;
    const GroupParams &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = (warp - 4) >> 2;    // query tile of this warpgroup
    const int quarter = warp & 3;     // TMEM lane quarter this warp may access
    const int lrow = 32 * quarter + lane;
    const int my_tok = lrow / p.group;  // token of this row within the tile
    // tokens (low half) and heads (high half) of the rows whose pieces this lane stores
    uint32_t out_at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = 32 * quarter + (lane & ~3) + k, tk = r / p.group;
        out_at[k] = (uint32_t)tk | (uint32_t)(r - tk * p.group) << 16;
    }
    const uint32_t s_addr = tmem_addr(tmem, 32 * quarter, BN * t);
    const uint32_t o_addr = tmem_addr(tmem, 32 * quarter, 256 + D * t);
    // as in fwd_tc.cu: |scale| (the score MMA negated S), never 0 so that -inf stays -inf
    const float sl2 = fmaxf(fabsf(p.scale_log2), FLT_MIN);
    const bool ordered = is_ordered(p);
    uint32_t s_cnt = 0, o_cnt = 0, kv_base = 0;
    // U_t *= alpha; U_t is stable once S_j(t) has completed, after PV_{j-1}(t)
    auto scale_u = [&](float alpha) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t u[32];
            tmem_ld_x32(o_addr + 32 * c, u);
            tmem_ld_wait(u);
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
            tmem_st_x32(o_addr + 32 * c, u);
        }
    };

    // kMask: the place up to which no row of a part's unit sees a key behind the sinks, by the least
    // number of drafts that one of its tokens sees, a token a lane.  -1: these may not be all the keys that may hold
    // anything (a window of fewer keys than there are new tokens, sinks among these, a new token that is in no row's
    // mask), or there are more than 64 new tokens.
    [[maybe_unused]] auto unseen_until = [&](const auto &g) -> int {
        if (g.T > 64 || p.window < g.T || p.sinks > g.ctx) return -1;
        const unsigned long long exist = ~0ull >> (64 - g.T), *mask = p.mask + (int64_t)g.q0 * p.mask_words;
        unsigned long long any = 0;
        int least = 64;
#pragma unroll 2
        for (int x = lane; x < g.T; x += 32) {
            const unsigned long long drafts = mask[(int64_t)x * p.mask_words] & exist;
            if (x >= g.tok[0] && x < g.tok[0] + NQT * (BM / p.group)) least = min(least, __popcll(drafts));
            any |= drafts;
        }
        const bool all = __reduce_or_sync(0xffffffffu, (uint32_t)any) == (uint32_t)exist &&
                         __reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) == (uint32_t)(exist >> 32);
        least = __reduce_min_sync(0xffffffffu, least);
        return all ? max(0, g.ctx - p.window + least) : -1;
    };

    for (int i = 0;; ++i) {
        const int slot = i % kSegs;
        bool ok = mbar_wait_small(smem_u32(&bars.seg_full[slot]), (i / kSegs) & 1, wd);
        if (!__all_sync(0xffffffffu, ok)) return;
        // read where it is needed, so that the inner loop keeps its registers; given back at the end
        const Seg<kWindow> &sg = segs[slot];
        const int nkv = sg.nkv, n = sg.n[t];
        if (nkv < 0) return;
        const uint32_t kv0 = kv_base;  // key tiles this block took before this part
        kv_base += nkv;
        if (n == 0) {
            // rows of a cut unit that see none of this part's keys
            if (lrow < sg.live[t])
                p.parts.ml[(int64_t)sg.slot * kGroupRows + BM * t + lrow] = make_float2(-INFINITY, 0.f);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.seg_empty[slot]));
            continue;
        }
        // keys that every row of the query tile sees: [0, all_end), and with a window of those the
        // sinks and [all_from, all_end)
        const int all_end = min(sg.L, sg.ctx + (ordered ? sg.tok[t] + 1 : 0));
        // tiles of such keys
        const int plain = max(0, min(n, (all_end >> 7) - sg.j0));
        int all_from = 0;
        RowWindow mine = {0, 0};  // of this row
        // kMask: no row of the unit sees the keys [sinks, unit_from), and the first query tile, which takes every key
        // tile that the other one takes, zeroes their V; below 0: what is not seen is looked for in each masked tile.
        int unit_from = 0;
        if constexpr (kWindow) {
            if constexpr (kMask)
                if (t == 0) unit_from = unseen_until(sg);
            const int token = sg.tok[t] + my_tok;
            if (!p.mask) {
                all_from = sg.ctx + sg.tok[t] + BM / p.group - p.window;
                mine = {sg.ctx + token + 1 - p.window, p.sinks};
            } else {
                all_from = sg.ctx + sg.T - p.window;
                if (lrow < sg.live[t])
                    mine = tree_window(p.mask + (int64_t)(sg.q0 + token) * p.mask_words, sg.T, sg.ctx, p.window, p.sinks);
            }
        }

        float m = -INFINITY, l = 0.f;
        // the running max refreshed with a tile's largest score: only when it grew by more than
        // 2^8 somewhere in the warp (else the stale max is kept, which leaves O = U / l exact);
        // the factor for l and U.  Rows that are not the entry's (another sequence's queries, or
        // what shared memory held) have no say, so that they do not move its results' last bits
        const float grown = lrow < sg.live[t] ? kRescaleThreshold : INFINITY;
        auto refresh = [&](float mx, bool first, bool &rescale) -> float {
            const float m_new = fmaxf(m, mx);
            rescale = !first && __any_sync(0xffffffffu, m_new > m + grown);
            float alpha = 1.f;
            if (first) {
                m = m_new;
            } else if (rescale) {
                alpha = m == -INFINITY ? 0.f : exp2_approx(m - m_new);
                m = m_new;
            }
            return alpha;
        };
        // key tile j of the part, all of whose keys every row of the query tile sees
        auto plain_tile = [&](int j) -> bool {
            ok = mbar_wait_small(smem_u32(&bars.s_full[t]), s_cnt & 1, wd);
            ++s_cnt;
            if (!__all_sync(0xffffffffu, ok)) return false;
            tc_fence_after();
            uint32_t r[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_x32(s_addr + 32 * c, r[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_wait(r[c]);
            float s[BN];
#pragma unroll
            for (int c = 0; c < BN; ++c) s[c] = __uint_as_float(r[c >> 5][c & 31]);
            bool rescale;
            const float alpha = refresh(row_max<BN>(s) * sl2, j == 0, rescale);
            const float m_use = m == -INFINITY ? 0.f : m;
            // p = 2^(s * scale * log2e - m): packed FMA pairs, four packed partial sums
            const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-m_use, -m_use);
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 x = __ffma2_rn(make_float2(s[64 * hh + 2 * e], s[64 * hh + 2 * e + 1]), sc2, nm2);
                    const float2 pv = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                    acc[e & 3] = __fadd2_rn(acc[e & 3], pv);
                    pk[e] = pack2(pv.x, pv.y, kBF16);  // P in the value type, the MMA's operand
                }
                tmem_st_x32(s_addr + 32 * hh, pk);
            }
            const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
            const float2 a03 = __fadd2_rn(a01, a23);
            l = l * alpha + (a03.x + a03.y);
            if (rescale) scale_u(alpha);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(smem_u32(&bars.p_full[t]));
            return true;
        };
        auto masked_tile = [&](int j) -> bool {
            // masked tiles, 32 keys at a time, scores read twice (for the max, then for p).  A loop,
            // and the only masked code: unrolled over the 128 columns it is fetched anew for each
            // unit's few masked tiles, which costs more than it computes (48 packed prompts of 9 to
            // 420 tokens 63 -> 85 us, long prompts the same)
            const int key0 = BN * (sg.j0 + j), left = sg.L - key0;
            const int steps = steps_of(sg, t, sg.j0 + j);
            const int token = sg.tok[t] + my_tok;
            const int lim = min(left, ordered ? sg.ctx + token + 1 - key0 : BN);  // keys [0, lim) admitted, but for the mask
            const unsigned long long *mrow =
                p.mask && lrow < sg.live[t] ? p.mask + (int64_t)(sg.q0 + token) * p.mask_words : nullptr;
            auto visible = [&](int c) -> uint32_t {  // of the keys [32 c, 32 c + 32)
                uint32_t bits = bits_below(lim, 32 * c);
                if (p.mask) bits &= mrow ? mask_bits(mrow, p.mask_words, key0 + 32 * c - sg.ctx) : 0u;
                if (kWindow) bits &= ~bits_below(mine.lo - key0, 32 * c) | bits_below(mine.hi - key0, 32 * c);
                return bits;
            };
            uint32_t unseen = 0;
            if constexpr (kMask)
                if (unit_from < 0)
                    unseen = unseen_keys(p.mask + (int64_t)(sg.q0 + sg.tok[0]) * p.mask_words, p.mask_words,
                                         min(NQT * (BM / p.group), sg.T - sg.tok[0]), sg.T, sg.ctx, p.window, p.sinks, key0 + 32 * quarter) &
                             bits_below(left, 32 * quarter);
            ok = mbar_wait_small(smem_u32(&bars.s_full[t]), s_cnt & 1, wd);
            ++s_cnt;
            if (!__all_sync(0xffffffffu, ok)) return false;
            tc_fence_after();
            auto zero_rows = [&](int from, int to) {  // of V
                const int chunks = (to - from) * 8;   // 16-byte chunks of a box
                const uint32_t base = sV + ((kv0 + j) % C::kVStages) * C::kTileBytes + from * 128;
#pragma unroll
                for (int b = 0; b < C::kBoxes; ++b) {
                    if constexpr (kWindow) {
#pragma unroll 1
                        for (int x = lrow; x < chunks; x += BM) st_shared_v4(base + b * C::kBoxBytes + 16 * x, 0, 0, 0, 0);
                    } else {
                        if (lrow < chunks) st_shared_v4(base + b * C::kBoxBytes + 16 * lrow, 0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
            };
            // V rows of the last MMA step behind the entry's end (another sequence's, stale
            // slots; NaN times p = 0 would be NaN): zeroed, by the query tile whose value
            // contraction comes first.  (V landed with K, before the scores waited for.)
            if (left < 16 * steps && (t == 0 || j >= sg.n[0] || left >= 16 * steps_of(sg, 0, sg.j0 + j)))
                zero_rows(max(0, left), 16 * steps);
            if constexpr (kWindow) {  // so are those that no row of the unit sees, but for drafts that other units' do
                const int from = max(p.sinks - key0, 16 * first_step(sg, t, sg.j0 + j));
                const int to = min((kMask ? unit_from : sg.from[0]) - key0, 16 * steps);
                if (max(0, from) < to && (t == 0 || j >= sg.n[0])) zero_rows(max(0, from), to);
                if (kMask && unseen) {
                    const uint32_t base = sV + ((kv0 + j) % C::kVStages) * C::kTileBytes + 32 * quarter * 128;
                    for (int x = lane; x < 32 * 8; x += 32) {  // 16-byte chunks of a box
                        if (!((unseen >> (x >> 3)) & 1)) continue;
#pragma unroll
                        for (int b = 0; b < C::kBoxes; ++b) st_shared_v4(base + b * C::kBoxBytes + 16 * x, 0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
            }
            const int chunks = (steps + 1) >> 1, chunk0 = first_step(sg, t, sg.j0 + j) >> 1;
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = chunk0; c < chunks; ++c) {
                uint32_t r[32];
                tmem_ld_x32(s_addr + 32 * c, r);
                const uint32_t bits = visible(c);
                tmem_ld_wait(r);
                float x[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = (bits >> e) & 1 ? __uint_as_float(r[e]) : -INFINITY;
                mx = fmaxf(mx, row_max<32>(x));
            }
            bool rescale;
            const float alpha = refresh(mx * sl2, j == 0, rescale);
            const float m_use = m == -INFINITY ? 0.f : m;
            float sum = 0.f;
#pragma unroll 1
            for (int c = chunk0; c < chunks; ++c) {
                uint32_t r[32], pk[16];
                tmem_ld_x32(s_addr + 32 * c, r);
                const uint32_t bits = visible(c);
                tmem_ld_wait(r);
                float part_sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float x = (bits >> e) & 1 ? fmaf(__uint_as_float(r[e]), sl2, -m_use) : -INFINITY;
                    const float pv = exp2_approx(x);
                    part_sum[e & 3] += pv;
                    r[e] = __float_as_uint(pv);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    pk[e] = pack2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]), kBF16);
                sum += (part_sum[0] + part_sum[1]) + (part_sum[2] + part_sum[3]);
                // P of 32 keys takes 16 columns: those of scores read before
                tmem_st_x16(s_addr + 16 * c, pk);
            }
            l = l * alpha + sum;
            if (rescale) scale_u(alpha);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(smem_u32(&bars.p_full[t]));
            return true;
        };
        if constexpr (kWindow) {
            for (int j = 0; j < n; ++j) {
                const int key0 = BN * (sg.j0 + j);
                const bool whole = key0 + BN <= all_end && (key0 >= all_from || key0 + BN <= p.sinks);
                if (!(whole ? plain_tile(j) : masked_tile(j))) return;
            }
        } else {
            int j = 0;
            for (; j < plain; ++j)
                if (!plain_tile(j)) return;
            for (; j < n; ++j)
                if (!masked_tile(j)) return;
        }
        const int live = sg.live[t], tok = sg.tok[t], q0 = sg.q0, hk = sg.hk, part = sg.slot, token = tok + my_tok;
        const int64_t part_row = (int64_t)part * kGroupRows + BM * t;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.seg_empty[slot]));

        // epilogue: O = U / l and lse, or the part's U, m and l
        ok = mbar_wait_small(smem_u32(&bars.o_done[t]), o_cnt & 1, wd);
        ++o_cnt;
        if (!__all_sync(0xffffffffu, ok)) return;
        tc_fence_after();
        if (part < 0) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            Tout *at[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                at[k] = 32 * quarter + (lane & ~3) + k < live
                            ? static_cast<Tout *>(p.o) + (int64_t)(q0 + tok + (int)(out_at[k] & 0xffff)) * p.o_st +
                                  (int64_t)(hk * p.group + (int)(out_at[k] >> 16)) * p.o_sh
                            : nullptr;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t u[32];
                tmem_ld_x32(o_addr + 32 * c, u);
                tmem_ld_wait(u);
                store_rows_at<Tout>(u, inv, at, 32 * c, lane);
            }
            if (lrow < live && p.lse)
                p.lse[(int64_t)(hk * p.group + lrow - my_tok * p.group) * p.n_q + q0 + token] =
                    l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
        } else {
            // as parts_merge.cu reads them: four columns of a warp's 32 rows after the other, so that a store
            // writes whole lines (a row after the other: 6200 cycles for the two query tiles' 128 KiB)
            float *at = p.parts.o + (part_row + 32 * quarter) * D + 4 * lane;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t u[32];
                tmem_ld_x32(o_addr + c, u);
                tmem_ld_wait(u);
                if (lrow < live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4 *>(at + 32 * (c + e)) = make_uint4(u[e], u[e + 1], u[e + 2], u[e + 3]);
                }
            }
            if (lrow < live) p.parts.ml[part_row + lrow] = make_float2(m, l);
        }
        tc_fence_before();
        mbar_arrive_warp(smem_u32(&bars.o_free[t]));
    }
}

template <int D, bool kBF16, typename Tout, bool kWindow, bool kMask>
__global__ void __launch_bounds__(kThreads, 1) group_tc_kernel(const __grid_constant__ GroupArgsOf<kWindow> a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    __shared__ Seg<kWindow> segs[kSegs];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sQ = (raw + 1023u) & ~1023u;
    const uint32_t sK = sQ + NQT * C::kTileBytes;
    const uint32_t sV = sK + C::kKStages * C::kTileBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Watchdog wd{a.p.watchdog_cycles, &abort_flag, a.p.status};

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int t = 0; t < NQT; ++t) {
            mbar_init(smem_u32(&bars.q_full[t]), 1);
            mbar_init(smem_u32(&bars.q_empty[t]), 1);
            mbar_init(smem_u32(&bars.s_full[t]), 1);
            mbar_init(smem_u32(&bars.p_full[t]), 4);  // one arrival per softmax warp
            mbar_init(smem_u32(&bars.o_done[t]), 1);
            mbar_init(smem_u32(&bars.o_free[t]), 4);
        }
        for (int s = 0; s < C::kKStages; ++s) {
            mbar_init(smem_u32(&bars.k_full[s]), 1);
            mbar_init(smem_u32(&bars.k_empty[s]), 1);
        }
        for (int s = 0; s < C::kVStages; ++s) mbar_init(smem_u32(&bars.v_empty[s]), 1);
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(smem_u32(&bars.seg_full[s]), 1);
            mbar_init(smem_u32(&bars.seg_empty[s]), kSegConsumers);
        }
        mbar_init(smem_u32(&bars.mma_drain), 1);
        fence_mbar_init();
        prefetch_tmap(&a.tq);
        prefetch_tmap(&a.tk);
        prefetch_tmap(&a.tv);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_base), 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    // set-up above overlaps the previous kernel on the stream; inputs are read after this
    pdl_trigger();
    pdl_wait();
    const int per = NQT * (BM / a.p.group);
    Stretch st;
    const bool any = find_stretch<kThreads / 32, kWindow ? kWindowLead : kLead>(
        a.p.n, 1, [&](int i, bool report) { return entry_work<kWindow>(a.p, entry_at(a.p, i, per, report), per); }, st);
    if (!any) st.end = st.at;
    if (threadIdx.x == 0) a.p.parts.cut[blockIdx.x].last = -1;  // the loading warp may put a unit there
    __syncthreads();

    if (warp < 4) {
        regs_dec<kWindow ? C::kRegsWindowProducer : C::kRegsProducer>();
        if (warp == 0) {
            producer<D, kWindow, kMask>(a, bars, segs, st, sQ, sK, sV, wd);  // the whole warp
        } else if (warp == 1) {
            mma_issuer<D, kBF16, kWindow>(a, bars, segs, sQ, sK, sV, tmem, wd);
            if (lane == 0 && aborting(wd)) {  // let issued MMAs finish before TMEM is freed
                tc_commit(smem_u32(&bars.mma_drain));
                drain_wait(smem_u32(&bars.mma_drain), 0, kDrainCycles);
            }
        }
    } else {
        regs_inc<kWindow ? C::kRegsWindowSoftmax : C::kRegsSoftmax>();
        softmax_wg<D, kBF16, Tout, kWindow, kMask>(a, bars, segs, sV, tmem, wd);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool kBF16, typename Tout, bool kWindow, bool kMask>
cudaError_t launch_typed(const GroupArgsOf<kWindow> &args, cudaStream_t s) {
    auto kern = group_tc_kernel<D, kBF16, Tout, kWindow, kMask>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(sm_count()), dim3(kThreads), Cfg<D>::kSmemBytes, s, args);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, bool kWindow, bool kMask>
cudaError_t launch_d(const GroupArgsOf<kWindow> &a, cudaStream_t s) {
    const bool f32 = a.p.o_dtype == ATTN_F32;
    if (a.p.dtype == ATTN_BF16)
        return f32 ? launch_typed<D, true, float, kWindow, kMask>(a, s) : launch_typed<D, true, __nv_bfloat16, kWindow, kMask>(a, s);
    return f32 ? launch_typed<D, false, float, kWindow, kMask>(a, s) : launch_typed<D, false, __half, kWindow, kMask>(a, s);
}

// Units of few tiles are not cut, so that no merge follows: a block's are those that begin in its stretch, or, where
// there are no more units than blocks, the unit of its number.  (Cut and whole: one prompt of 100 tokens, 32 / 8
// heads, D = 128, 13.2 and 10.0 us; of 700, window 256, 23.2 and 15.8; 4 of 1000 tokens, window 500, 53.2 and 51.8;
// 48 of 9 to 420, window 128, 72.5 and 70.7; 2 x 8192, window 1024, of 10 tiles, the same; 64 units of 33
// tiles 59 and 75.)
int whole_units(const GroupParams &p) {
    const int64_t per = NQT * (BM / p.group), units = p.Hkv * (p.n_q / per + p.n);
    int64_t keys = (p.mask ? 64 * (int64_t)p.mask_words : per - 1) + p.window + p.sinks + (p.paged ? 2 * (BN - 1) : 15);
    const int64_t there = p.paged ? (int64_t)p.c.max_pages << p.c.page_shift : p.n_k;
    if (keys > there) keys = there;
    if (keys > 6 * BN) return 0;
    return units <= sm_count() ? kUnitLine : kTileLine;
}

// The attention kernel, and the merge of cut units.
template <bool kWindow, bool kMask>
cudaError_t launch_group_of(const GroupParams &p, cudaStream_t s) {
    GroupArgsOf<kWindow> a;
    a.p = p;
    if constexpr (kWindow) a.p.whole = whole_units(p);
    const uint64_t D = (uint64_t)p.D;
    const int tok = BM / p.group;
    bool ok;
    {
        const uint64_t dims[3] = {D, (uint64_t)p.H, (uint64_t)p.n_q};
        const uint64_t st[2] = {(uint64_t)p.q_sh * 2, (uint64_t)p.q_st * 2};
        const uint32_t box[3] = {64, (uint32_t)p.group, (uint32_t)tok};
        ok = make_map(&a.tq, p.q, p.dtype, 3, dims, st, box);
    }
    if (p.paged) {
        const int page = 1 << p.c.page_shift;
        const uint64_t dims[4] = {D, (uint64_t)page, (uint64_t)p.Hkv, (uint64_t)p.c.n_pages};
        const uint64_t st[3] = {(uint64_t)p.c.b_tok, (uint64_t)p.c.b_head, (uint64_t)p.c.b_page};
        const uint32_t box[4] = {64, (uint32_t)(page < BN ? page : BN), 1, 1};
        ok = ok && make_map(&a.tk, p.c.k, p.dtype, 4, dims, st, box) && make_map(&a.tv, p.c.v, p.dtype, 4, dims, st, box);
    } else {
        ok = ok && make_tile_map(&a.tk, p.k, p.dtype, p.D, p.n_k, p.Hkv, p.k_st, p.k_sh) &&
             make_tile_map(&a.tv, p.v, p.dtype, p.D, p.n_k, p.Hkv, p.v_st, p.v_sh);
        if constexpr (kWindow)
            ok = ok && make_tile_map(&a.tk16, p.k, p.dtype, p.D, p.n_k, p.Hkv, p.k_st, p.k_sh, 16) &&
                 make_tile_map(&a.tv16, p.v, p.dtype, p.D, p.n_k, p.Hkv, p.v_st, p.v_sh, 16);
    }
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t e = p.D == 64 ? launch_d<64, kWindow, kMask>(a, s) : launch_d<128, kWindow, kMask>(a, s);
    if (e != cudaSuccess || (kWindow && a.p.whole)) return e;
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
    m.rows = kGroupRows;
    m.tile_rows = BM;
    m.tile_live = tok * p.group;
    m.blocks = sm_count();
    return launch_parts_merge(m, s);
}

}  // namespace

}  // namespace attn
