"""The rule for lengths of cached sequences (csrc/pages.h), compiled for the host, at
every kind of 32-bit value that ``lens`` may hold."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "online_softmax_attention_gb300", "csrc")
SOURCE = """
#include "pages.h"
extern "C" {
int t_pages(int tokens, int shift) { return attn::pages_of(tokens, shift); }
int t_fits(int len, int max_pages, int shift) { return attn::length_fits(len, max_pages, shift); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("pages")
    (d / "pages.cpp").write_text(SOURCE)
    out = str(d / "pages.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-ftrapv", "-fPIC", "-shared", "-I", CSRC, str(d / "pages.cpp"), "-o", out],
                   check=True)
    return ctypes.CDLL(out)


@pytest.mark.parametrize("shift", [0, 3, 4, 10])
def test_lengths_at_the_edges_of_32_bits(lib, shift):
    page = 1 << shift
    for max_pages in (1, 8, 1000, ((1 << 31) - (1 << 16)) // page):
        most = max_pages * page
        for n in {0, 1, page - 1, page, page + 1, most - 1, most, most + 1, (1 << 31) - 1, (1 << 31) - page,
                  (1 << 31) - page + 1, -1, -page, -(1 << 31)}:
            if n < 1 << 31:
                assert bool(lib.t_fits(n, max_pages, shift)) == (0 <= n <= most), (n, max_pages)
            if 0 <= n < 1 << 31:
                assert lib.t_pages(n, shift) == -(-n // page)
