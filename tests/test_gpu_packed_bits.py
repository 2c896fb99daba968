"""A sequence's results of the packed kernel depend, bit for bit, on its own queries and keys
only: not on other rows of their tiles, which may be another sequence's, nor on what an
earlier kernel left in shared memory for rows that no query fills."""
import pytest
import torch

import online_softmax_attention_gb300 as attn
from test_gpu_grouped import make
from test_gpu_tree import make as make_cache

pytestmark = pytest.mark.gpu


def leave_large_scores(d, dtype):
    """A forward whose queries fill every tile row and whose scores grow from key tile to key tile."""
    q = torch.full((2048, 8, d), 4.0, device="cuda", dtype=dtype)
    k = torch.linspace(0, 4, 2048, device="cuda").to(dtype)[:, None, None].expand(2048, 2, d).contiguous()
    attn.fwd(q, k, k)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("hq,hkv", [(6, 2), (10, 2), (7, 1), (8, 2)])
def test_rows_of_the_next_sequence_have_no_say(hq, hkv, dtype, d):
    """Queries that raise their own running max at every key tile beside ones that hardly do."""
    lens = [700, 300]
    x, cu = make(lens, hq, hkv, d, dtype, 91)
    q, k, v = (x[n].cuda() for n in "qkv")
    q[:700] *= 0.5
    ramp = torch.linspace(1, 40, 1000, device="cuda").to(dtype)[:, None, None]
    got = []
    for other in (torch.zeros_like(q[700:]), q[700:] * 30, torch.full_like(q[700:], float("nan"))):
        q2, k2 = q.clone(), k.clone()
        q2[700:] = other
        k2[700:] = k2[700:] * ramp[700:]
        got.append(attn.fwd(q2, k2, v, cu_seqlens_q=cu))
    for o, lse in got[1:]:
        assert torch.equal(o[:700], got[0][0][:700]) and torch.equal(lse[:, :700], got[0][1][:, :700])


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("hq,hkv", [(3, 1), (10, 2), (7, 1), (33, 1)])
def test_rows_that_no_query_fills_have_no_say(hq, hkv, dtype, d):
    """Groups that do not divide 128 leave rows of every tile unwritten."""
    lens = [900, 41, 1500]
    x, cu = make(lens, hq, hkv, d, dtype, 92)
    q, k, v = (x[n].cuda() for n in "qkv")
    cache, _, seqs, g = make_cache([1400, 700], 64, hkv, d, dtype, 93)
    new = torch.randn(60, hq, d, generator=g).to(dtype).cuda()
    first = None
    for dirty in (False, True, False, True):
        if dirty:
            leave_large_scores(d, dtype)
        else:
            attn.fwd(torch.zeros(2048, 8, d, device="cuda", dtype=dtype), *(torch.zeros(2048, 2, d, device="cuda", dtype=dtype),) * 2)
        got = (*attn.fwd(q, k, v, causal=True, cu_seqlens_q=cu), *attn.tree_fwd(new, cache, seqs, [0, 20, 60]))
        first = first or [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(got, first))
