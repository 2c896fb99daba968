"""The library builds and its calls work without the compiled torch binding, which only
saves host time."""
import os
import warnings

import pytest
import torch

import online_softmax_attention_gb300 as attn
from online_softmax_attention_gb300 import _abi, _host, build


def no_torch(name, package=None):
    return None


@pytest.mark.parametrize("missing", ["torch", "headers", "compiler"])
def test_the_binding_is_left_out_of_the_build(missing, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_native.so"))
    (tmp_path / "_native.so").write_bytes(b"another torch's")
    if missing == "torch":
        monkeypatch.setattr(build.importlib.util, "find_spec", no_torch)
    elif missing == "headers":
        monkeypatch.setattr(build, "_torch_dir", lambda: str(tmp_path))
    else:
        monkeypatch.setenv("CXX", "no-such-compiler")
    assert not build._binding(False)
    assert not os.path.exists(build.NATIVE)


@pytest.fixture
def without(monkeypatch):
    monkeypatch.setattr(_host, "_native", None)
    monkeypatch.setattr(_host, "_NATIVE", os.path.join(os.path.dirname(_abi.LIB_PATH), "no_such_binding.so"))
    with pytest.warns(RuntimeWarning, match="not built"):
        _host.native()


def test_calls_take_the_python_path(without):
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # said once
        assert _host.native().fwd(1, 2, 3) is None
        with pytest.raises(ValueError, match="CUDA"):
            attn.fwd(*(torch.zeros(4, 2, 64) for _ in range(3)))


@pytest.mark.gpu
def test_results_without_the_binding(without):
    q, k, v = (torch.randn(40, h, 64, device="cuda").half() for h in (4, 2, 2))
    o, lse = attn.fwd(q, k, v, causal=True)
    dq, dk, dv = attn.bwd(q, k, v, o, lse, q, causal=True)
    cache = attn.Cache.empty(1, 8, 16, 2, 64, max_seqs=2, max_pages=4, dtype=torch.float16)
    one, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([1], [0, 40]))
    cache.extend(one, cu[1:])
    cache.write(one, cu, k, v)
    o2, lse2 = attn.tree_fwd(q, cache, one, cu)
    cache.fork(one, one - 1)
    cache.keep(one, cu[1:], cu[:1].view(1, 1), one)
    cache.free(one)
    assert attn.device_status() == 0 and cache.lens.tolist() == [40, 0]
    _host._native = None
    _host._NATIVE = os.path.join(os.path.dirname(_abi.LIB_PATH), "_native.so")
    assert not isinstance(_host.native(), _host._NoBinding)
    for a, b in zip((o, lse, dq, dk, dv), (*attn.fwd(q, k, v, causal=True), *attn.bwd(q, k, v, o, lse, q, causal=True))):
        assert torch.equal(a, b)
    cache.extend(one, cu[1:])
    cache.write(one, cu, k, v)
    got = attn.tree_fwd(q, cache, one, cu)
    assert torch.equal(got[0], o2) and torch.equal(got[1], lse2)
