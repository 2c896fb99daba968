"""The arithmetic by which the packed and cached attention kernels cut their work
(csrc/line.h), compiled for the host: sums of key tiles against brute force, cuts that
take every tile once, and totals past 2^36 tiles."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "online_softmax_attention_gb300", "csrc")

SOURCE = r"""
#include "line.h"
using namespace attn;
static Stretch of(const long long *s) {
    Stretch r = {};
    r.at = s[0]; r.end = s[1]; r.share = s[2]; r.lead = (int)s[3]; r.snap = (int)s[4];
    return r;
}
extern "C" {
long long t_floor_sum(int n, int a, int b) { return floor_sum(n, a, b); }
int t_tiles_to(int ordered, int L, int ctx, int T, int tok) { return tiles_to(ordered != 0, L, ctx, T, tok); }
long long t_unit_tiles(int ordered, int L, int ctx, int T, int units, int per, int n) {
    return unit_tiles(ordered != 0, L, ctx, T, units, per, n);
}
int t_take(long long units, long long tiles, unsigned blocks, unsigned b, int turn, int lead, long long *s) {
    Stretch r = {};
    const bool any = r.take(Work{units, tiles} + Work{0, 0}, blocks, b, turn, lead, 12);
    s[0] = r.at; s[1] = r.end; s[2] = r.share; s[3] = r.lead; s[4] = r.snap;
    return any;
}
long long t_length(const long long *s, long long units, long long tiles) { return of(s).length(Work{units, tiles}); }
int t_tile(const long long *s, long long x, long long u0, int n) { return of(s).tile(x, u0, n); }
int t_last_block(const long long *s, long long u0, int n) { return of(s).last_block(u0, n); }
}
"""

i32, i64 = ctypes.c_int, ctypes.c_longlong


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("line")
    (d / "line.cpp").write_text(SOURCE)
    out = str(d / "line.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-ftrapv", "-fPIC", "-shared", "-I", CSRC, str(d / "line.cpp"), "-o", out],
                   check=True)
    lib = ctypes.CDLL(out)
    lib.t_floor_sum.restype = lib.t_unit_tiles.restype = lib.t_length.restype = i64
    lib.t_take.argtypes = [i64, i64, ctypes.c_uint, ctypes.c_uint, i32, i32, ctypes.c_void_p]
    lib.t_length.argtypes = [ctypes.c_void_p, i64, i64]
    lib.t_tile.argtypes = [ctypes.c_void_p, i64, i64, i32]
    lib.t_last_block.argtypes = [ctypes.c_void_p, i64, i32]
    return lib


def take(lib, units, tiles, blocks, b, turn, lead):
    s = (i64 * 5)()
    return s, bool(lib.t_take(units, tiles, blocks, b, turn, lead, s))


def test_sums_of_floors(lib):
    r = random.Random(1)
    for _ in range(300):
        n, a, b = r.randint(0, 200), r.randint(0, 600), r.randint(0, 5000)
        assert lib.t_floor_sum(n, a, b) == sum((a * i + b) // 128 for i in range(n))
    # a row of 2^24 units, and a context of almost 2^31 tokens before them
    for n, a, b in ((1 << 24, 2, 2 + 127), (1 << 23, 128, 127), (99991, 254, (1 << 31) - (1 << 16))):
        assert lib.t_floor_sum(n, a, b) == sum((a * i + b) // 128 for i in range(n))


def test_tiles_of_the_first_units(lib):
    r = random.Random(2)
    for _ in range(400):
        T = r.choice([1, 2, r.randint(1, 40), r.randint(1, 6000)])
        ordered = r.random() < 0.8
        L = T + r.choice([0, 0, r.randint(0, 9000)])
        ctx = L - T if ordered else L
        per = r.choice([256, 128, 84, 64, 50, 42, 2])
        units = -(-T // per)
        each = [max(1, -(-(min(L, ctx + min((u + 1) * per, T)) if ordered else L) // 128)) for u in range(units)]
        assert lib.t_tiles_to(ordered, L, ctx, T, per) == each[0]
        for n in {0, 1, units // 2, units - 1, units}:
            assert lib.t_unit_tiles(ordered, L, ctx, T, units, per, n) == sum(each[:n]), (T, L, per, n)


def check_cuts(lib, units, blocks, turn, lead):
    total = sum(units)
    parts = [[] for _ in units]
    at = 0
    for b in range(blocks):
        s, any_ = take(lib, len(units), total, blocks, b, turn, lead)
        length = lib.t_length(s, len(units), total)
        assert any_ == (s[0] < s[1]) and s[0] == b * s[2]
        if not any_:
            continue
        assert s[0] == at and s[1] <= length
        at, u0 = s[1], 0
        for i, n in enumerate(units):
            if u0 + n + s[3] > s[0] and u0 < s[1]:
                t0, t1 = lib.t_tile(s, s[0], u0, n), lib.t_tile(s, s[1], u0, n)
                if t0 < t1:
                    parts[i].append((b, t0, t1))
            u0 += n + s[3]
    assert at == length
    u0 = 0
    for n, p in zip(units, parts):
        assert [x for _, a, b in p for x in range(a, b)] == list(range(n))
        assert [b for b, _, _ in p] == list(range(p[0][0], p[-1][0] + 1))
        assert lib.t_last_block(s, u0, n) == p[-1][0]
        u0 += n + s[3]


@pytest.mark.parametrize("turn,lead", [(1, 1), (1, 2), (4, 0)])
def test_every_tile_is_taken_once(lib, turn, lead):
    r = random.Random(3)
    for _ in range(60):
        blocks = r.choice([1, 2, 7, 152])
        check_cuts(lib, [r.choice([1, 1, 2, 3, r.randint(1, 60)]) for _ in range(r.randint(1, 200))], blocks, turn, lead)
    for n in range(1, 30):  # one-tile units whose ends meet the cuts
        check_cuts(lib, [1] * (24 * n), 2 * n, turn, lead)


@pytest.mark.parametrize("turn,lead", [(1, 1), (1, 2), (4, 0)])
@pytest.mark.parametrize("units,tiles", [(1 << 20, 1 << 36), (1 << 20, (1 << 36) + 5), (8 << 18, 1 << 40), (1 << 28, 1 << 52)])
def test_totals_past_2_36_tiles(lib, units, tiles, turn, lead):
    """Chunks of 2^19 tokens whose 16-row units scan 2^15 tiles for each of 8 key heads, and beyond:
    the line has its whole length, and the blocks' stretches cover it in order."""
    at = 0
    for b in range(152):
        s, any_ = take(lib, units, tiles, 152, b, turn, lead)
        assert any_ and s[0] == at and s[2] >= tiles // 152
        assert lib.t_length(s, units, tiles) == tiles + lead * units
        at = s[1]
    assert at == tiles + lead * units
