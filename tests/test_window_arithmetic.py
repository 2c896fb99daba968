"""The arithmetic of sliding windows (csrc/window.h), compiled for the host: the key tiles
that a run of rows scans against the keys that the rows see, sums of them over units against
brute force, and the window of a tree's row."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from cache_model import seen_tree
from window_model import windowed

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "online_softmax_attention_gb300", "csrc")

SOURCE = r"""
#include "window.h"
using namespace attn;
extern "C" {
void t_list(int window, int sinks, int seen, int tile, int *r) {
    const TileList l = tile_list(window, sinks, seen, tile);
    r[0] = l.sinks; r[1] = l.skip;
}
int t_at(int sinks, int skip, int j) { return TileList{sinks, skip}.at(j); }
long long t_skipped(int window, int sinks, int ctx, int per, int n) { return skipped_tiles(window, sinks, ctx, per, n); }
int t_units(int ordered, int L, int ctx, int T, int units, int per, int window, int sinks, int piece, int i, int *r) {
    const WindowUnits u = {ordered != 0, L, ctx, T, units, per, window, sinks, piece};
    const KeyList l = u.list(i);
    r[0] = l.held; r[1] = l.shift; r[2] = u.tiles(i);
    return l.at(r[3]);
}
long long t_before(int ordered, int L, int ctx, int T, int units, int per, int window, int sinks, int piece, int n) {
    return WindowUnits{ordered != 0, L, ctx, T, units, per, window, sinks, piece}.before(n);
}
void t_row(const unsigned long long *mask, int T, int ctx, int window, int sinks, int *r) {
    const RowWindow w = tree_window(mask, T, ctx, window, sinks);
    r[0] = w.lo; r[1] = w.hi;
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("window")
    (d / "window.cpp").write_text(SOURCE)
    out = str(d / "window.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-ftrapv", "-fPIC", "-shared", "-I", CSRC, str(d / "window.cpp"), "-o", out],
                   check=True)
    lib = ctypes.CDLL(out)
    lib.t_skipped.restype = lib.t_before.restype = ctypes.c_longlong
    return lib


def tile_list(lib, window, sinks, seen, tile):
    r = (ctypes.c_int * 2)()
    lib.t_list(window, sinks, seen, tile, r)
    return r[0], r[1]


def test_the_list_holds_every_key_that_is_seen(lib):
    rng = random.Random(1)
    for _ in range(2000):
        tile, n = rng.choice([16, 32, 64, 128]), rng.randint(1, 700)
        window, sinks, seen = rng.randint(1, 800), rng.choice([0, 1, 4, rng.randint(0, 800)]), rng.randint(0, n)
        held, skip = tile_list(lib, window, sinks, seen, tile)
        count = -(-n // tile) - skip
        tiles = [lib.t_at(held, skip, j) for j in range(count)]
        assert count >= 1 and tiles == sorted(set(tiles)) and tiles[-1] == -(-n // tile) - 1 and tiles[0] >= 0
        # rows that would see `seen` keys or more
        need = {key // tile for row in {seen, min(seen + 5, n), n} for key in range(row) if key < sinks or key >= row - window}
        assert need <= set(tiles)
        # of the tiles before the rows' last ones, only those that the first row sees a key of
        first = {key // tile for key in range(seen) if key < sinks or key >= seen - window}
        assert all(t in first or t >= seen // tile or t * tile < sinks for t in tiles)


def test_sums_over_units(lib):
    rng = random.Random(2)
    for _ in range(3000):
        per, n = rng.choice([2, 4, 32, 64, 85, 256]), rng.randint(0, 60)
        ctx, window, sinks = rng.choice([0, rng.randint(0, 5000)]), rng.randint(1, 6000), rng.choice([0, 1, 200, rng.randint(0, 6000)])
        want = sum(tile_list(lib, window, sinks, ctx + i * per + 1, 128)[1] for i in range(n))
        assert lib.t_skipped(window, sinks, ctx, per, n) == want, (window, sinks, ctx, per, n)


def test_lengths_near_32_bits(lib):
    most = 2 ** 31 - 2 ** 16
    for window, sinks in ((1, 0), (4096, 4), (most - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1), (most - 1, 0)):
        held, skip = tile_list(lib, window, sinks, most, 128)
        first = (most - window) // 128
        assert held + skip == first and held == min(first, -(-sinks // 128))
        units = most // 256
        last = [tile_list(lib, window, sinks, 256 * i + 1, 128)[1] for i in (units - 3, units - 2, units - 1)]
        assert lib.t_skipped(window, sinks, 0, 256, units) - lib.t_skipped(window, sinks, 0, 256, units - 3) == sum(last)


def test_units_hold_every_key_that_is_seen(lib):
    """The places of a unit's tiles against the keys that its rows see: all of them once, in order, the
    last place being the last key; sums over units against brute force; pages in whole pieces."""
    rng = random.Random(4)
    for _ in range(1500):
        ordered, piece = rng.random() < 0.7, rng.choice([0, 0, 8, 16, 64, 128])
        ctx = rng.choice([0, rng.randint(0, 3000)]) if piece else 0
        T, per = rng.randint(1, 1500 if ordered else 120), rng.choice([2, 64, 84, 256])
        L, units = ctx + T, -(-T // per)
        window, sinks = rng.randint(1, 1200), rng.choice([0, 1, 4, rng.randint(0, 600)])
        total, r = 0, (ctypes.c_int * 4)()
        args = (int(ordered), L, ctx, T, units, per, window, sinks, piece)
        for i in range(units):
            lib.t_units(*args, i, r)
            held, shift, tiles = r[0], r[1], r[2]
            assert lib.t_before(*args, i) == total, (args, i)
            total += tiles
            first = ctx + i * per + 1 if ordered else ctx
            end = min(L, ctx + min((i + 1) * per, T)) if ordered else L
            places = end - shift  # that the unit's rows may see
            assert 128 * (tiles - 1) < max(places, 1) <= 128 * tiles
            keys = [p if p < held else p + shift for p in range(places)]
            assert keys == sorted(set(keys)) and (not keys or keys[-1] == end - 1)
            rows = {first, end}
            need = {k for n in rows for k in range(n) if k < sinks or k >= n - window}
            assert need <= set(keys), args
            if shift:
                grain = 128 if piece and ordered and units > 8 else piece or 16
                assert held % grain == 0 and held >= sinks and (not piece or shift % piece == 0)
                assert len(keys) < window + (end - first) + sinks + 2 * grain + 1
            else:
                assert held == 0
        assert lib.t_before(*args, units) == total, args


def test_unit_sums_of_long_rows(lib):
    most = 2 ** 31 - 2 ** 16
    r = (ctypes.c_int * 4)()
    for window, sinks, piece, ctx in ((1, 0, 0, 0), (4096, 4, 0, 0), (most - 1, 2 ** 31 - 1, 0, 0), (4096, 4, 64, 0),
                                      (100000, 5000, 0, 0), (1000, 10, 16, most // 2)):
        T = most - ctx
        units = -(-T // 256)
        args = (1, most, ctx, T, units, 256, window, sinks, piece)
        for n in (units, units - 1, units // 2, 10):
            tail = 0
            for i in range(n - 3, n):
                lib.t_units(*args, i, r)
                tail += r[2]
            assert lib.t_before(*args, n) - lib.t_before(*args, n - 3) == tail, (args, n)


def test_windows_of_tree_rows(lib):
    rng = random.Random(3)
    for _ in range(1500):
        T, words, ctx = rng.choice([1, 5, 63, 64, 65, 130]), 3, rng.choice([0, 1, 7, 200])
        bits = [rng.getrandbits(64) & rng.choice([2 ** 64 - 1, rng.getrandbits(64), 0]) for _ in range(words)]
        window, sinks = rng.randint(1, 260), rng.choice([0, 1, 4, rng.randint(0, 300)])
        mask = (ctypes.c_ulonglong * words)(*bits)
        r = (ctypes.c_int * 2)()
        lib.t_row(mask, T, ctx, window, sinks, r)
        row = seen_tree(ctx + T, T, [bits] * T)[:1]
        at = np.arange(ctx + T)
        assert (row & ((at >= r[0]) | (at < r[1])) == windowed(row, window, sinks)).all(), (T, ctx, window, sinks, bits)
