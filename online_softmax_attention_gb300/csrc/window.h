// Sliding windows with sinks: of the keys that a query would see without a window, in
// order, it sees the first `sinks` and the last `window`.  Plain functions of their
// arguments, compiled for the host too.
//
// A run of query rows scans the key tiles that hold a sink and those from its first row's
// window on.  That list has one gap at most, so its j-th tile is j or, behind the
// gap, j + skip.
#pragma once

#include "hd.h"
#include "line.h"

namespace attn {

struct TileList {
    int sinks;  // tiles before the gap
    int skip;   // tiles that the gap leaves out
    ATTN_HD int at(int j) const { return j < sinks ? j : j + skip; }
};

// The list in tiles of `tile` keys: `seen` >= 0 is the least number of keys that one of the
// rows would see without a window, whose window begins at key seen - window.
ATTN_HD TileList tile_list(int window, int sinks, int seen, int tile) {
    const int first = seen > window ? (seen - window) / tile : 0;
    const int held = sinks / tile + (sinks % tile != 0);
    return held < first ? TileList{held, first - held} : TileList{first, 0};
}

// Key tiles of 128 that the gaps of the first n units leave out, of an entry whose tokens
// each see those up to themselves: unit i begins at token i per, before which ctx keys stand.
// sum over i < n of max(0, floor((ctx + i per + 1 - window) / 128) - tiles of the sinks)
ATTN_HD long long skipped_tiles(int window, int sinks, int ctx, int per, int n) {
    const long long held = sinks / 128 + (sinks % 128 != 0);
    const long long b = (long long)ctx + 1 - window - 128 * held;  // of unit 0; the first terms may be below 0
    if (b + (n - 1ll) * per < 0) return 0;
    const int i0 = b >= 0 ? 0 : (per - 1 - (int)b) / per;
    return floor_sum(n - i0, per, (int)(b + (long long)i0 * per));
}

// dK / dV items of a head of a sequence of `blocks` key (and query) blocks.  A block with a sink
// is seen by all queries behind it; where those are more than `chunk` blocks they are cut into
// chunks, an item each, so that no item is much longer than those of a window.
struct SinkItems {
    int tiles;   // blocks with a sink
    int chunks;  // items of each
};
ATTN_HD SinkItems sink_items(int blocks, int sink_tiles, int chunk) {
    return {sink_tiles < blocks ? sink_tiles : blocks, chunk > 0 && blocks > chunk ? (blocks - 1) / chunk + 1 : 1};
}
// Item t of a head: those of blocks with a sink come first, where they are cut.
struct SinkItem {
    int tile;         // key block
    int first, most;  // first query block; as many at most
    int part;         // its slot of partial sums, among the sequence's; -1: it has all its query blocks
};
ATTN_HD SinkItem sink_item(int t, int blocks, int sink_tiles, int chunk) {
    const SinkItems sink = sink_items(blocks, sink_tiles, chunk);
    if (sink.chunks == 1) return {t, t, blocks, -1};
    const int cut = sink.tiles * sink.chunks;
    if (t >= cut) return {t - cut + sink.tiles, t - cut + sink.tiles, blocks, -1};
    const int tile = t / sink.chunks;
    return {tile, tile + (t - tile * sink.chunks) * chunk, chunk, t};
}
// Slots of partial sums of a head before row `row` (all of them: of n_q): a sequence whose blocks of
// `block` rows are cut has more than chunk of them, so rows / (block chunk), doubled, holds its chunks.
ATTN_HD long long sink_slot(long long row, int block, int sink_tiles, int chunk) {
    return 2ll * sink_tiles * (row / ((long long)block * chunk));
}

// The same list in single keys: places [0, held) are keys 0 .. (the sinks, rounded up to whole pieces
// of a load), the places behind them the keys from the window's first on.  {0, 0}: no gap.
struct KeyList {
    int held;
    int shift;  // of the places behind
    ATTN_HD int at(int place) const { return place < held ? place : place + shift; }
};

// `seen` as in tile_list; the window begins at a multiple of `grain` keys, the sinks take a multiple of
// `held_grain` (powers of two).
ATTN_HD KeyList key_list(int window, int sinks, int seen, int grain, int held_grain) {
    const int from = seen > window ? (seen - window) & ~(grain - 1) : 0;
    const unsigned held = ((unsigned)sinks + held_grain - 1) & ~(unsigned)(held_grain - 1);
    if (held >= (unsigned)from) return {0, 0};
    return {(int)held, from - (int)held};
}

// The units of an entry over such lists, in tiles of 128 places; unit i begins at token i per.
struct WindowUnits {
    bool ordered;               // tokens see those up to themselves; else what a mask says, of all L keys
    int L, ctx, T, units, per;  // as in unit_tiles
    int window, sinks;
    int piece;                  // rows that a load of the keys takes at once (pages); 0: any

    // Of pages, many units begin at whole tiles, so that their sum has a closed form.
    ATTN_HD int grain() const { return piece == 0 ? 1 : units <= 8 || !ordered ? piece : 128; }
    ATTN_HD KeyList list(int i) const {
        return key_list(window, sinks, ordered ? ctx + i * per + 1 : ctx, grain(), piece == 0 ? 16 : grain());
    }
    // tiles of a list that hold the keys which the entry's first `tok` tokens see; one at least
    ATTN_HD int tiles_to(KeyList l, int tok) const {
        int end = L;
        if (ordered) {
            const int upto = ctx + (tok < T ? tok : T);
            end = upto < L ? upto : L;
        }
        const int n = (end - l.shift + 127) / 128;
        return n > 1 ? n : 1;
    }
    ATTN_HD int tiles(int i) const { return tiles_to(list(i), (i + 1) * per); }
    // of the first n units
    ATTN_HD long long before(int n) const {
        if (!ordered) return (long long)n * tiles(0);
        if (n <= 8) {
            long long r = 0;
            for (int i = 0; i < n; ++i) r += tiles(i);
            return r;
        }
        if (piece) return unit_tiles(true, L, ctx, T, units, per, n) - skipped_tiles(window, sinks, ctx, per, n);
        // up to the first unit with a gap as without a window; those behind it have per - 1 + window keys
        // and the sinks each, but for the entry's last one
        const long long held = (long long)(((unsigned)sinks + 15) & ~15u), x = window + held - 1 - ctx;
        if (x >= (long long)(n - 1) * per) return unit_tiles(true, L, ctx, T, units, per, n);
        const int first = x < 0 ? 0 : (int)x / per + 1, whole = n < units ? n : units - 1;
        long long r = first ? unit_tiles(true, L, ctx, T, units, per, first) : 0;
        if (whole > first) r += (whole - first) * ((per - 1 + window + held + 127) >> 7);
        return n == units ? r + tiles(units - 1) : r;
    }
};

// The keys that a row of a tree sees: below `hi`, or from `lo` on, of the ctx keys before the
// new tokens and the new tokens u < T whose bits are set in `mask`.
struct RowWindow {
    int lo, hi;
};

#if defined(__CUDA_ARCH__)
#define ATTN_POPC(x) __popcll(x)
#else
#define ATTN_POPC(x) __builtin_popcountll(x)
#endif

ATTN_HD RowWindow tree_window(const unsigned long long *mask, int T, int ctx, int window, int sinks) {
    const int words = (T + 63) / 64;
    auto word = [&](int w) -> unsigned long long {  // bits from T on do not exist
        return w == words - 1 && (T & 63) ? mask[w] & ((1ull << (T & 63)) - 1) : mask[w];
    };
    int drafts = 0;  // that the row sees
    for (int w = 0; w < words; ++w) drafts += ATTN_POPC(word(w));
    // behind the nth of the row's drafts, 0 <= n <= drafts (its first one: n = 0)
    auto behind = [&](int n) -> int {
        for (int w = 0; w < words; ++w) {
            unsigned long long x = word(w);
            const int c = ATTN_POPC(x);
            if (n <= c && n > 0) {
                for (; n > 1; --n) x &= x - 1;
                return 64 * w + ATTN_POPC((x & -x) - 1) + 1;
            }
            n -= c;
        }
        return 0;
    };
    RowWindow r;
    if (drafts >= window) r.lo = ctx + behind(drafts - window);
    else r.lo = ctx > window - drafts ? ctx - (window - drafts) : 0;
    if (sinks <= ctx) r.hi = sinks;
    else r.hi = sinks - ctx >= drafts ? ctx + T : ctx + behind(sinks - ctx);
    return r;
}

}  // namespace attn
