"""The windowed backward where values are not finite: pairs that a window hides, or that are of two sequences, add
nothing to the gradients of rows and keys that have nothing else to do with them."""
import pytest
import torch

import online_softmax_attention_gb300 as attn
from test_gpu_grouped import make
from window_model import causal

pytestmark = pytest.mark.gpu

LENS = [400, 90, 300]
KERNELS = [("tc", torch.bfloat16, 128), ("tc", torch.float16, 64), ("simt", torch.float32, 64), ("simt", torch.float16, 128)]


def seen(window, sinks):
    """(T, T): whether row i sees key j."""
    out = torch.zeros(sum(LENS), sum(LENS), dtype=torch.bool)
    at = 0
    for n in LENS:
        out[at:at + n, at:at + n] = torch.from_numpy(causal(n, window, sinks))
        at += n
    return out.cuda()


def step(kernel, dtype, d, window, sinks):
    x, cu = make(LENS, 4, 2, d, dtype, 120, True)
    c = {n: t.cuda() for n, t in x.items()}
    w = dict(causal=True, cu_seqlens_q=cu, kernel=kernel, window=window, sinks=sinks)
    o, lse = attn.fwd(c["q"], c["k"], c["v"], **w)
    return c, w, o, lse, attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], **w)


@pytest.mark.parametrize("kernel,dtype,d", KERNELS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (30, 3), (100, 0), (130, 140), (260, 5)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_values_of_keys(kernel, dtype, d, window, sinks, value):
    """Beside the sinks, in the middle, a sequence's last key and another's first ones."""
    c, w, o, lse, want = step(kernel, dtype, d, window, sinks)
    keys = torch.tensor([5, 150, 389, 400, 401, 490], device="cuda")
    v = c["v"].clone()
    v[keys, 1] = value
    got = attn.bwd(c["q"], c["k"], v, o, lse, c["do"], **w)
    rows = ~seen(window, sinks)[:, keys].any(1)
    assert rows.any() and torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[0][:, :2], want[0][:, :2])
    others = torch.ones(sum(LENS), dtype=torch.bool, device="cuda")
    others[keys] = False
    assert torch.equal(got[1][others], want[1][others]) and torch.equal(got[1][:, 0], want[1][:, 0])
    assert torch.equal(got[2], want[2])
    assert attn.device_status() == 0


@pytest.mark.parametrize("kernel,dtype,d", KERNELS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (30, 3), (100, 0), (130, 140), (260, 5)])
@pytest.mark.parametrize("value", [float("nan"), float("-inf")])
def test_rows_of_nan(kernel, dtype, d, window, sinks, value):
    """A row whose lse is NaN, or -inf though it sees keys (forwards of NaN scores), has no gradient, nor have the keys that
    it sees."""
    c, w, o, lse, want = step(kernel, dtype, d, window, sinks)
    rows = torch.tensor([0, 200, 399, 430, 700], device="cuda")
    bad = lse.clone()
    bad[3, rows] = value  # of the second key head
    dq, dk, dv = attn.bwd(c["q"], c["k"], c["v"], o, bad, c["do"], **w)
    keys = seen(window, sinks)[rows].any(0)
    for got, ref in ((dk, want[1]), (dv, want[2])):
        assert (value == value or got[keys, 1].isnan().all()) and torch.equal(got[~keys], ref[~keys]) and torch.equal(got[:, 0], ref[:, 0])
    others = torch.ones(sum(LENS), dtype=torch.bool, device="cuda")
    others[rows] = False
    assert (value == value or dq[rows, 3].isnan().all()) and torch.equal(dq[others], want[0][others]) and torch.equal(dq[:, :3], want[0][:, :3])
    assert attn.device_status() == 0
