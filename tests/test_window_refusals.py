"""Arguments of windowed attention, of attention weights and of eviction that the host refuses
before any launch (no GPU: the pointers are numbers that are never followed)."""
import ctypes

import pytest

from online_softmax_attention_gb300 import _abi, _host
from test_abi import FAKE, _fwd_args
from test_cache_refusals import A, CACHE_REFUSALS, _cache


@pytest.fixture(autouse=True)
def _no_launch():
    lib = _abi.load()
    before = lib.attn_launch_count()
    yield
    assert lib.attn_launch_count() == before


BAD_WINDOWS = [({"window": -1}, _abi.ATTN_EINVAL), ({"window": 8, "sinks": -1}, _abi.ATTN_EINVAL),
               ({"sinks": 4}, _abi.ATTN_EINVAL)]


@pytest.mark.parametrize("kw,code", BAD_WINDOWS + [
    ({"window": 8, "relation": _abi.ATTN_FULL}, _abi.ATTN_EUNSUPPORTED),
    ({"window": 8, "qk_fp8": 1}, _abi.ATTN_EUNSUPPORTED)])
def test_forward_windows_that_are_refused(kw, code):
    lib = _abi.load()
    a = _fwd_args(**({"D": 128} if "qk_fp8" in kw else {}))
    for n, x in kw.items():
        setattr(a, n, x)
    a.workspace_bytes = 1 << 40
    assert lib.attn_fwd(ctypes.byref(a), None) == code


def _bwd_args(**kw):
    b = _abi.BwdArgs()
    for name in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
        setattr(b, name, _abi.AttnTensor(FAKE, 128, 64))
    b.lse = b.workspace = FAKE
    b.n_q = b.n_k = 256
    b.H, b.D, b.scale, b.n_seq, b.relation = 2, 64, 0.125, 1, _abi.ATTN_CAUSAL
    b.workspace_bytes = 1 << 40
    for n, x in kw.items():
        setattr(b, n, x)
    return b


@pytest.mark.parametrize("kw,code", BAD_WINDOWS + [
    ({"window": 8, "relation": _abi.ATTN_FULL}, _abi.ATTN_EUNSUPPORTED),
    ({"window": 8, "dq_mode": _abi.ATTN_DQ_FUSED}, _abi.ATTN_EUNSUPPORTED)])
def test_backward_windows_that_are_refused(kw, code):
    lib = _abi.load()
    b = _bwd_args(**kw)
    for fn in (lib.attn_bwd, lib.attn_bwd_preprocess, lib.attn_bwd_dkdv, lib.attn_bwd_dq):
        assert fn(ctypes.byref(b), None) == code


def _tree_args(**kw):
    a = _abi.TreeArgs()
    a.cache = _cache()
    a.H, a.q, a.o, a.lse = 4, _abi.AttnTensor(A, 256, 64), _abi.AttnTensor(A, 256, 64), A
    a.seqs = a.cu = a.workspace = A
    a.n, a.n_q, a.scale, a.o_dtype, a.workspace_bytes = 2, 8, 0.125, _abi.ATTN_BF16, 1 << 40
    for n, x in kw.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("kw,code", BAD_WINDOWS)
def test_cached_windows_that_are_refused(kw, code):
    lib = _abi.load()
    a = _tree_args(**kw)
    assert lib.attn_tree_fwd(ctypes.byref(a), None) == code
    assert lib.attn_tree_workspace_bytes(ctypes.byref(a)) == 0


def _weigh_args(**kw):
    a = _abi.WeighArgs()
    a.cache = kw.pop("cache", None) or _cache()
    a.H, a.q, a.lse, a.weights, a.weights_stride, a.cols = 4, _abi.AttnTensor(A, 256, 64), A, A, 128, 128
    a.n, a.n_q, a.scale, a.seqs, a.cu = 2, 8, 0.125, A, A
    for n, x in kw.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("kw,code", BAD_WINDOWS + [
    ({"layer": 2}, _abi.ATTN_EINVAL), ({"layer": -1}, _abi.ATTN_EINVAL), ({"H": 5}, _abi.ATTN_EINVAL),
    ({"H": 0}, _abi.ATTN_EINVAL), ({"n": -1}, _abi.ATTN_EINVAL), ({"n_q": -1}, _abi.ATTN_EINVAL),
    ({"cols": -1}, _abi.ATTN_EINVAL), ({"weights_stride": 127}, _abi.ATTN_EINVAL), ({"weights": None}, _abi.ATTN_EINVAL),
    ({"weights": A + 2}, _abi.ATTN_EINVAL), ({"lse": None}, _abi.ATTN_EINVAL), ({"lse": A + 1}, _abi.ATTN_EINVAL),
    ({"seqs": None}, _abi.ATTN_EINVAL), ({"cu": A + 2}, _abi.ATTN_EINVAL), ({"fresh": A + 1}, _abi.ATTN_EINVAL),
    ({"q": _abi.AttnTensor(A + 8, 256, 64)}, _abi.ATTN_EINVAL), ({"q": _abi.AttnTensor(A, 250, 64)}, _abi.ATTN_EINVAL),
    ({"scale": float("nan")}, _abi.ATTN_EINVAL), ({"scale": float("inf")}, _abi.ATTN_EINVAL),
    ({"n_q": 1 << 30}, _abi.ATTN_EUNSUPPORTED)])
def test_weigh_arguments_that_are_refused(kw, code):
    assert _abi.load().attn_cache_weigh(ctypes.byref(_weigh_args(**kw)), None) == code


def test_weights_of_no_entries():
    lib = _abi.load()
    assert lib.attn_cache_weigh(None, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_weigh(ctypes.byref(_weigh_args(n=0, seqs=None, cu=None)), None) == _abi.ATTN_OK


def _evict(c=None, w=None, seqs=A, budgets=A, n=3, sinks=0, recent=0, ws=A, size=None):
    lib = _abi.load()
    c = c or _cache()
    w = w or _abi.Weights(A, 4 * 128, 128, 2, 128)
    if size is None:
        size = max(lib.attn_cache_evict_workspace_bytes(ctypes.byref(c), n, w.cols), 256)
    return lib.attn_cache_evict(ctypes.byref(c), seqs, budgets, n, ctypes.byref(w), sinks, recent, ws, size, None)


@pytest.mark.parametrize("kw", [
    dict(seqs=None), dict(budgets=A + 2), dict(n=-1), dict(sinks=-1), dict(recent=-1), dict(w=_abi.Weights(None, 512, 128, 2, 128)),
    dict(w=_abi.Weights(A + 1, 512, 128, 2, 128)), dict(w=_abi.Weights(A, 512, 127, 2, 128)),
    dict(w=_abi.Weights(A, -512, 128, 2, 128)), dict(w=_abi.Weights(A, 512, 128, 0, 128)), dict(w=_abi.Weights(A, 512, 128, 2, -1))])
def test_evictions_that_are_refused(kw):
    assert _evict(**kw) == _abi.ATTN_EINVAL


def test_eviction_workspaces_that_are_refused():
    lib, c = _abi.load(), _cache()
    need = lib.attn_cache_evict_workspace_bytes(ctypes.byref(c), 3, 128)
    assert need > 3 * 128 * 4 and need % 256 == 0
    for ws, size in ((None, need), (A + 16, need), (A, need - 1)):
        assert _evict(ws=ws, size=size) == _abi.ATTN_EWORKSPACE
    assert lib.attn_cache_evict_workspace_bytes(ctypes.byref(c), -1, 128) == 0
    assert lib.attn_cache_evict_workspace_bytes(ctypes.byref(c), 1, -1) == 0
    assert lib.attn_cache_evict(ctypes.byref(c), A, A, 1, None, 0, 0, A, 1 << 20, None) == _abi.ATTN_EINVAL
    assert _evict(n=0, seqs=None, budgets=None) == _abi.ATTN_OK


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS)
def test_cache_descriptions_that_are_refused(kw, code):
    c = _cache(**kw)
    assert _abi.load().attn_cache_weigh(ctypes.byref(_weigh_args(cache=c)), None) == code
    assert _evict(c=c, size=1 << 20) == code
    assert _abi.load().attn_cache_evict_workspace_bytes(ctypes.byref(c), 1, 128) == 0


def test_windows_as_python_gives_them():
    assert _host.window(None, 0) == (0, 0) and _host.window(5, 3) == (5, 3) and _host.window(2 ** 31 - 1, 0)
    for bad in ((0, 0), (-3, 0), (2 ** 31, 0), (4, -1), (4, 2 ** 31), (None, 2)):
        with pytest.raises(ValueError, match="window|sinks"):
            _host.window(*bad)
    for bad in ((4.0, 0), (True, 0), (4, None), (4, 1.5), ("4", 0)):
        with pytest.raises(TypeError, match="whole number"):
            _host.window(*bad)


@pytest.mark.parametrize("layer,seq", [(0, 128), (511, 128), (600, 200)])
def test_weights_whose_layers_overlap_are_refused(layer, seq):
    """4 sequences' rows a layer, moved at the same time as the other layer's."""
    assert _cache().max_seqs == 4
    assert _evict(w=_abi.Weights(A, layer, seq, 2, 128)) == _abi.ATTN_EINVAL
    assert _evict(w=_abi.Weights(A, layer, seq, 1, 128), n=0) == _abi.ATTN_OK
