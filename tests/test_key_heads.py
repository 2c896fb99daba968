"""The key head of a query head (csrc/heads.h), compiled for the host, against the division."""
import ctypes
import os
import random
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "online_softmax_attention_gb300", "csrc")
SOURCE = """
#include "heads.h"
extern "C" int t_key_head(int h, int group) { return attn::key_head(h, attn::group_inverse(group)); }
"""


def test_as_the_division(tmp_path):
    (tmp_path / "heads.cpp").write_text(SOURCE)
    out = str(tmp_path / "heads.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", CSRC, str(tmp_path / "heads.cpp"), "-o", out],
                   check=True)
    f = ctypes.CDLL(out).t_key_head
    most = (1 << 31) - 1
    for group in range(1, 200):
        for h in range(3 * group + 2):
            assert f(h, group) == h // group
    r = random.Random(1)
    for _ in range(20000):
        group = r.choice([1, 2, 3, 7, r.randint(1, 1 << 10), r.randint(1, most)])
        k = r.randint(0, most // group)
        for h in (k * group - 1, k * group, k * group + group - 1, r.randint(0, most), most):
            if 0 <= h <= most:
                assert f(h, group) == h // group, (h, group)
