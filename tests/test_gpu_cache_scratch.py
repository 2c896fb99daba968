"""The cache's operations need nothing of the ``Cache`` object once they are launched or
captured: it may be dropped, and memory may be allocated in its place."""
import gc

import pytest
import torch

import online_softmax_attention_gb300 as attn
from test_gpu_cache import fill, make, same

pytestmark = pytest.mark.gpu


def junk():
    """Blocks of the sizes that scratch has, on the default stream, full of bad page indices."""
    return [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in (256, 1 << 10, 1 << 12, 1 << 14, 1 << 16) for _ in range(40)]


def lists(*xs):
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in xs]


def test_the_handle_holds_the_callers_tensors_only():
    c, _ = make()
    theirs = {t.data_ptr() for t in (c.k, c.v, c.table, c.lens, c.refs)}
    assert {t.data_ptr() for t in vars(c).values() if isinstance(t, torch.Tensor)} == theirs


@pytest.mark.parametrize("on_device", [True, False])
def test_dropped_while_another_stream_runs(on_device):
    c, m = make()
    fill(c, m, [40, 17])
    view = attn.Cache(c.k, c.v, c.table, c.lens, c.refs)  # made on the default stream
    seqs, counts, draft, keep, n_keep = lists([1, 0], [30, 9], [3, 4], [[1, 2], [0, 3]], [2, 2]) if on_device else (
        [1, 0], [30, 9], [3, 4], torch.tensor([[1, 2], [0, 3]]), [2, 2])
    parent, child = lists([0], [4]) if on_device else ([0], [4])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms: the operations wait behind it
        view.extend(seqs, counts)
        view.keep(seqs, draft, keep, n_keep)
        view.fork(parent, child)
        view.compact()
    del view
    gc.collect()
    held = junk()
    torch.cuda.synchronize()
    m.extend([1, 0], [30, 9])
    m.keep([1, 0], [3, 4], [[1, 2], [0, 3]], [2, 2])
    m.fork([0], [4])
    m.compact()
    same(c, m)
    assert attn.device_status() == 0 and len(held) == 200


def test_dropped_while_a_graph_holds_its_operations():
    c, m = make(n_pages=200, per_seq=40)
    fill(c, m, [20, 7, 33])
    view = attn.Cache(c.k, c.v, c.table, c.lens, c.refs)
    seqs, counts, keep, n_keep = lists([2, 0, 1], [4, 4, 4], [[0, 2], [1, 3], [0, 0]], [2, 2, 0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        view.extend(seqs, counts)
        view.keep(seqs, counts, keep, n_keep)
    del view
    gc.collect()
    held = junk()
    for _ in range(5):
        g.replay()
        m.extend([2, 0, 1], [4, 4, 4])
        m.keep([2, 0, 1], [4, 4, 4], [[0, 2], [1, 3], [0, 0]], [2, 2, 0])
    same(c, m)
    assert attn.device_status() == 0 and all(int(x.max()) == 0x7f for x in held)
