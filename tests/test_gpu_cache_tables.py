"""A page index outside the pool, met in a table, is reported and never followed."""
import pytest
import torch

import online_softmax_attention_gb300 as attn
from online_softmax_attention_gb300 import _abi
from test_gpu_cache import fill, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [97, -1, -7, (1 << 31) - 1, -(1 << 31)])
def test_every_operation_meets_it(bad):
    c, m = make()
    fill(c, m, [40, 17, 32])
    before = c.k.clone()
    c.table[0, 1] = bad
    attn.device_status()
    c.fork([0], [5])  # carried out, but for the count of the page that is none
    assert attn.device_status() == _abi.ATTN_EINVAL
    assert int(c.lens[5]) == 40 and int(c.table[5, 1]) == bad and int(c.refs[c.table[0, 0]]) == 2
    assert int(c.refs.sum()) == 3 + 2 + 2 + 2
    k, v = (torch.ones(25, 3, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    c.write([0], [0, 25], k, v)  # rows 15 (shared page), 16 to 31 (no page) stay, 32 to 39 are written
    assert attn.device_status() == _abi.ATTN_EINVAL
    changed = (c.k != before).flatten(2).any(2)  # (layers, pages); the child's last page is a copy of its own
    own, child = int(c.table[0, 2]), int(c.table[5, 2])
    assert bool(changed[0, own]) and set(changed.nonzero()[:, 1].tolist()) <= {own, child} and not changed[1, own]
    c.keep([0], [30], torch.tensor([[1, 8]]), [2])  # row 11 to 10 (shared), refused before anything moves
    assert attn.device_status() == _abi.ATTN_EINVAL and int(c.lens[0]) == 40
    for heads in (6, 96):
        attn.tree_fwd(torch.ones(1, heads, 64, dtype=torch.float16, device="cuda"), c, [0], [0, 1])
        assert attn.device_status() == _abi.ATTN_EINVAL
    c.free([0, 5])
    assert attn.device_status() == _abi.ATTN_EINVAL
    # (the page that the table lost is still counted)
    assert int(c.refs.sum()) == 2 + 2 + 1 and int(c.lens[0]) == int(c.lens[5]) == 0
    c.table[1, 1] = bad
    c.compact()
    assert attn.device_status() in (0, _abi.ATTN_EINVAL)
    assert int(c.table[1, 1]) == bad
