// Arithmetic of the line of work units that stretch.cuh cuts between blocks:
// plain functions of their arguments, compiled for the host too.
#pragma once

#include "hd.h"

namespace attn {

// Work of an entry, or of several: units, and the key tiles that they scan.  64 bits
// each: every unit counts its tiles, so the same keys count once for every 16 or 256
// query rows and every key head, and what memory holds does not bound their number
// (f32 cache, 8 key heads for 64 query heads, a chunk of 2^19 tokens: 2^36 tiles).
struct Work {
    long long units, tiles;
};
ATTN_HD Work operator+(Work a, Work b) { return {a.units + b.units, a.tiles + b.tiles}; }
ATTN_HD Work operator-(Work a, Work b) { return {a.units - b.units, a.tiles - b.tiles}; }

struct Stretch {
    long long at, end;   // the block's part of the line
    long long share;     // length of a block's part (the last ones may be shorter)
    long long before;    // length of the line before entry `entry`
    Work work;           // of the entry
    int entry;           // entry that position `at` lies in
    int lead, snap;      // of a unit of n tiles: see tile()

    // A unit takes lead + n positions: `lead` stands for what a unit costs besides its
    // tiles (loading queries, masks, writing out).  Tile at which position x cuts the
    // unit that begins at u0; a cut that would part fewer than `snap` tiles moves to
    // the unit's edge.
    ATTN_HD int tile(long long x, long long u0, int n) const {
        const long long o = x - u0 - lead;
        return o >= n ? n : o <= 0 || o < snap ? 0 : o > n - snap ? n : (int)o;
    }
    ATTN_HD long long length(Work w) const { return w.tiles + lead * w.units; }
    // Block that takes the last tile of the unit of n tiles that begins at u0.
    ATTN_HD int last_block(long long u0, int n) const {
        const long long last = (u0 + lead + n - 1) / share;
        return (int)(tile(last * share, u0, n) == n ? last - 1 : last);
    }
    // Block b's part of a line of that much work, cut for `blocks` blocks (see find_stretch);
    // false: nothing.
    ATTN_HD bool take(Work total, unsigned blocks, unsigned b, int turn, int unit_lead, int lead_share) {
        const bool long_enough = total.tiles >= (long long)lead_share * blocks;
        lead = long_enough ? unit_lead : 0;
        snap = long_enough && unit_lead ? 2 : 0;
        const long long all = length(total);
        share = all < 0x7fffffff - (long long)blocks ? (long long)(((unsigned)all + blocks - 1) / blocks)
                                                     : (all + blocks - 1) / blocks;
        if (share > turn) share = (share + turn - 1) / turn * turn;
        at = b * share;
        end = at + share < all ? at + share : all;
        return at < end;
    }
};

// sum over i < n of floor((a i + b) / 128), a >= 0, b >= 0 (the Euclid-like
// recursion; after the first step everything is below 128 n)
ATTN_HD long long floor_sum(int n0, int a0, int b0) {
    long long r = (long long)(a0 >> 7) * ((long long)n0 * (n0 - 1) / 2) + (long long)(b0 >> 7) * n0;
    unsigned n = n0, m = 128, a = a0 & 127, b = b0 & 127;
    for (;;) {
        const unsigned y = a * n + b;
        if (y < m) return r;
        n = y / m;
        b = y - n * m;
        const unsigned t = m;
        m = a;
        a = t;
        r += (long long)(a / m) * ((long long)n * (n - 1) / 2) + (long long)(b / m) * n;
        a %= m;
        b %= m;
    }
}

// Tiles of 128 keys that the first `tok` of an entry's T tokens need at most: of L keys,
// with `ordered` those up to ctx + the token's own place.  One at least.
ATTN_HD int tiles_to(bool ordered, int L, int ctx, int T, int tok) {
    if (ordered) {
        const int upto = ctx + (tok < T ? tok : T);
        L = upto < L ? upto : L;
    }
    const int n = (L + 127) / 128;
    return n > 1 ? n : 1;
}

// Key tiles of the first n of a key head's `units` units of `per` tokens.
ATTN_HD long long unit_tiles(bool ordered, int L, int ctx, int T, int units, int per, int n) {
    const int full = tiles_to(ordered, L, ctx, T, 1), last = tiles_to(ordered, L, ctx, T, T);
    if (full == last) return (long long)n * last;
    if (n <= 8) {
        long long r = 0;
        for (int i = 0; i < n; ++i) r += tiles_to(ordered, L, ctx, T, (i + 1) * per);
        return r;
    }
    // units before the entry's last one hold `per` tokens: ceil((ctx + (i + 1) per) / 128)
    const int whole = n < units - 1 ? n : units - 1;
    return floor_sum(whole, per, ctx + per + 127) + (n > whole ? last : 0);
}

}  // namespace attn
