"""Token counts so near 2^31 that rounding up to a tile would overflow are refused before any
launch (no GPU: the pointers are numbers that are never followed)."""
import ctypes

import pytest

from online_softmax_attention_gb300 import _abi
from test_abi import FAKE
from test_cache_refusals import _no_launch, _tree  # noqa: F401

MOST = (1 << 31) - (1 << 16)


def calls(n_q, n_k, H, H_kv, relation):
    f, b = _abi.FwdArgs(), _abi.BwdArgs()
    for a in (f, b):
        for n in ("q", "k", "v", "o"):
            setattr(a, n, _abi.AttnTensor(FAKE, H * 64, 64))
        a.lse, a.n_q, a.n_k, a.H, a.D, a.n_seq, a.H_kv = FAKE, n_q, n_k, H, 64, 1, H_kv
        a.scale, a.relation, a.workspace, a.workspace_bytes = 0.125, relation, None, 0
        a.dtype = a.o_dtype = _abi.ATTN_BF16
    for n in ("dout", "dq", "dk", "dv"):
        setattr(b, n, _abi.AttnTensor(FAKE, H * 64, 64))
    b.grad_dtype = _abi.ATTN_BF16
    lib = _abi.load()
    return lib.attn_fwd(ctypes.byref(f), None), lib.attn_bwd(ctypes.byref(b), None)


@pytest.mark.parametrize("n_q,n_k,H,H_kv,relation", [
    (64, MOST + 1, 2, 1, _abi.ATTN_FULL), (64, (1 << 31) - 1, 2, 1, _abi.ATTN_FULL), (64, MOST + 1, 1, 1, _abi.ATTN_FULL),
    (MOST + 1, 64, 1, 1, _abi.ATTN_FULL), ((1 << 31) - 1, (1 << 31) - 1, 1, 1, _abi.ATTN_CAUSAL),
    ((1 << 30) - 100, 64, 2, 1, _abi.ATTN_FULL)])
def test_prompts(n_q, n_k, H, H_kv, relation):
    assert calls(n_q, n_k, H, H_kv, relation) == (_abi.ATTN_EUNSUPPORTED, _abi.ATTN_EUNSUPPORTED)


def test_the_largest_counts_get_as_far_as_their_workspace():
    for n_q, n_k, H, H_kv in ((64, MOST, 2, 1), (MOST, 64, 1, 1), (MOST // 2, 64, 2, 1)):
        assert calls(n_q, n_k, H, H_kv, _abi.ATTN_FULL) == (_abi.ATTN_EWORKSPACE, _abi.ATTN_EWORKSPACE)


@pytest.mark.parametrize("n_q,H", [((1 << 29) - 1, 4), ((1 << 31) // 8 - 1, 8), (MOST // 4 + 1, 4)])
def test_rows_over_the_cache(n_q, H):
    """(token, head) rows of a unit's tile are counted in 32 bits."""
    assert _abi.load().attn_tree_fwd(ctypes.byref(_tree(n_q=n_q, H=H)), None) == _abi.ATTN_EUNSUPPORTED
    ok = _tree(n_q=MOST // H, H=H, workspace=None)
    assert _abi.load().attn_tree_fwd(ctypes.byref(ok), None) == _abi.ATTN_EWORKSPACE
