"""Lengths that no sequence can have are refused by every operation of the cache."""
import pytest
import torch

import online_softmax_attention_gb300 as attn
from online_softmax_attention_gb300 import _abi
from test_gpu_cache import fill, make, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [(1 << 31) - 1, (1 << 31) - 16, (1 << 31) - 15, 321, -1, -(1 << 31)])
def test_lengths_that_do_not_fit_are_refused(bad):
    """20 pages of 16 rows a sequence: 320 tokens."""
    c, m = make()
    fill(c, m, [40, 17, 32])
    c.lens[1] = bad
    m.lens[1] = bad
    k, v = (torch.ones(1, 3, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    one = torch.zeros(1, 1, dtype=torch.int32)
    remap = torch.full_like(c.refs, -1)
    attn.device_status()
    for call in (lambda: c.extend([0, 1], [1, 1]), lambda: c.extend([1], [0]), lambda: c.fork([0, 1], [5, 6]),
                 lambda: c.fork([0], [1]), lambda: c.keep([0, 1], [1, 1], one.repeat(2, 1), [0, 1]),
                 lambda: c.keep([1], [4], one + 1, [1]), lambda: c.write([1], [0, 1], k, v), lambda: c.free([1]),
                 lambda: c.free([1, 1]), lambda: c.compact(remap=remap)):
        call()
        assert attn.device_status() == _abi.ATTN_EINVAL
        same(c, m)
    assert torch.equal(remap.cpu(), torch.arange(97, dtype=torch.int32))
    for heads, dtype in ((3, torch.float16), (96, torch.float16)):  # few rows a key head, and many
        call = attn.TreeCall(torch.ones(1, heads, 64, dtype=dtype, device="cuda"), c, [1], [0, 1])
        call.o.fill_(5.0)
        assert (call.run()[0] == 5).all()
        assert attn.device_status() == _abi.ATTN_EINVAL
    # the others go on
    c.free([0])
    m.free([0])
    same(c, m)
    c.lens[1] = 17
    m.lens[1] = 17
    c.compact()
    m.compact()
    same(c, m)
    assert attn.device_status() == 0


def test_a_full_sequence_fits():
    c, m = make()
    fill(c, m, [320, 5])
    c.free([1])
    m.free([1])
    c.fork([0], [3])
    m.fork([0], [3])
    same(c, m)
    assert attn.device_status() == 0
