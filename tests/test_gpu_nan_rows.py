"""A row of NaN scores has O and lse of NaN; lse = -inf means that a row sees nothing."""
import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from test_gpu_grouped import make as make_packed
from test_gpu_tree import make

pytestmark = pytest.mark.gpu


def same_rows(o, lse, want):
    """NaN in every column of o, and in lse, at `want` (tokens, heads) and nowhere else."""
    assert torch.equal(o.isnan().all(2).cpu(), want) and torch.equal(o.isnan().any(2).cpu(), want)
    assert torch.equal(lse.isnan().t().cpu(), want) and not torch.isinf(lse).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,news,heads,mask", [(9000, 1, 4, False), (9000, 40, 8, False), (50, 3, 2, False),
                                               (300, 30, 8, True)])
def test_queries_of_nan_over_the_cache(dtype, n, news, heads, mask):
    """Whole units and cut ones, few and many rows a key head."""
    cache, _, seqs, g = make([n, 20], 16, 1, 64, dtype, 101)
    q = torch.randn(news + 1, heads, 64, generator=g).to(dtype)
    q[0, 1] = q[news - 1, heads - 1] = float("nan")
    bits = torch.full((news + 1, 1), -1, device="cuda") if mask else None
    o, lse = attn.tree_fwd(q.cuda(), cache, seqs, [0, news, news + 1], mask=bits)
    want = torch.zeros(news + 1, heads, dtype=torch.bool)
    want[0, 1] = want[news - 1, heads - 1] = True
    same_rows(o, lse, want)
    assert attn.device_status() == 0


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("lens,at", [([6000], 4500), ([40, 200, 3], 150)])
def test_queries_and_keys_of_nan_in_prompts(lens, at, dtype, d):
    x, cu = make_packed(lens, 8, 2, d, dtype, 102)
    q, k, v = (x[n].cuda() for n in "qkv")
    q2, k2 = q.clone(), k.clone()
    q2[at, 3] = float("nan")
    want = torch.zeros(sum(lens), 8, dtype=torch.bool)
    want[at, 3] = True
    same_rows(*attn.fwd(q2, k, v, causal=True, cu_seqlens_q=cu), want)
    k2[at, 1] = float("nan")  # seen by the rows from its own to its sequence's end
    end = next(int(c) for c in cu if c > at)
    want = torch.zeros(sum(lens), 8, dtype=torch.bool)
    want[at:end, 4:] = True
    same_rows(*attn.fwd(q, k2, v, causal=True, cu_seqlens_q=cu), want)


def test_a_key_of_nan_reaches_the_gradients():
    """p is NaN in every row that sees the key, so dv is NaN at every key that such a row sees."""
    x, cu = make_packed([200, 90], 8, 2, 128, torch.bfloat16, 103, True)
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    k[150, 1] = float("nan")
    o, lse = attn.fwd(q, k, v, causal=True, cu_seqlens_q=cu)
    _, _, dv = attn.bwd(q, k, v, o, lse, do, causal=True, cu_seqlens_q=cu)
    want = torch.zeros(290, 2, dtype=torch.bool)
    want[:200, 1] = True
    assert torch.equal(dv.isnan().all(2).cpu(), want) and torch.equal(dv.isnan().any(2).cpu(), want)


def test_rows_that_see_nothing_keep_their_mark():
    cache, _, seqs, g = make([6, 40], 16, 2, 64, torch.bfloat16, 104)
    q = torch.randn(9, 4, 64, generator=g).bfloat16()
    bits = np.zeros((9, 1), np.int64)
    bits[1, 0] = 1
    o, lse = attn.tree_fwd(q.cuda(), cache, seqs, [0, 6, 9], mask=torch.from_numpy(bits).cuda())
    none = [0, 2, 3, 4, 5]
    assert (o[none] == 0).all() and (lse[:, none] == -torch.inf).all() and torch.isfinite(lse[:, [1, 6, 7, 8]]).all()
