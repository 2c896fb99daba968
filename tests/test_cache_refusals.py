"""Arguments of the grouped-head and cache entry points that the host refuses
before any launch (no GPU: the pointers are numbers that are never followed)."""
import ctypes

import pytest

import online_softmax_attention_gb300 as attn
from online_softmax_attention_gb300 import _abi

A = 1 << 20


@pytest.fixture(autouse=True)
def _no_launch():
    lib = _abi.load()
    before = lib.attn_launch_count()
    yield
    assert lib.attn_launch_count() == before


def _cache(**kw):
    c = _abi.Cache()
    c.k, c.v, c.table, c.lens, c.refs = A, A, A, A, A
    c.n_layers, c.n_pages, c.page_size, c.H_kv, c.D = 2, 64, 16, 2, 64
    c.dtype, c.max_seqs, c.max_pages, c.table_stride = _abi.ATTN_BF16, 4, 8, 8
    c.stride_head, c.stride_tok, c.stride_page, c.stride_layer = 64, 128, 2048, 131072
    for n, x in kw.items():
        setattr(c, n, x)
    return c


CACHE_REFUSALS = [
    ({"dtype": 5}, _abi.ATTN_EINVAL), ({"n_layers": 0}, _abi.ATTN_EINVAL), ({"n_pages": 0}, _abi.ATTN_EINVAL),
    ({"H_kv": 0}, _abi.ATTN_EINVAL), ({"max_seqs": 0}, _abi.ATTN_EINVAL), ({"max_pages": 0}, _abi.ATTN_EINVAL),
    ({"table_stride": 7}, _abi.ATTN_EINVAL), ({"k": None}, _abi.ATTN_EINVAL), ({"v": A + 2}, _abi.ATTN_EINVAL),
    ({"table": None}, _abi.ATTN_EINVAL), ({"lens": A + 1}, _abi.ATTN_EINVAL), ({"refs": None}, _abi.ATTN_EINVAL),
    ({"stride_tok": 132}, _abi.ATTN_EINVAL), ({"stride_head": 0}, _abi.ATTN_EINVAL),
    ({"stride_page": -2048}, _abi.ATTN_EINVAL),
    ({"D": 96}, _abi.ATTN_EUNSUPPORTED), ({"page_size": 24}, _abi.ATTN_EUNSUPPORTED),
    ({"page_size": 0}, _abi.ATTN_EUNSUPPORTED), ({"page_size": 2048}, _abi.ATTN_EUNSUPPORTED),
    ({"max_seqs": 262145}, _abi.ATTN_EUNSUPPORTED), ({"H_kv": 5000}, _abi.ATTN_EUNSUPPORTED),
    ({"max_pages": 1 << 28, "table_stride": 1 << 28}, _abi.ATTN_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS)
def test_cache_descriptions_that_are_refused(kw, code):
    lib, c = _abi.load(), _cache(**kw)
    r, t = ctypes.byref(c), ctypes.byref(_abi.AttnTensor(A, 128, 64))
    assert lib.attn_cache_workspace_bytes(r, 1) == 0
    assert lib.attn_cache_extend(r, A, A, 1, A, 1 << 20, None) == code
    assert lib.attn_cache_fork(r, A, A, 1, A, 1 << 20, None) == code
    assert lib.attn_cache_keep(r, A, A, A, 4, A, 1, A, 1 << 20, None) == code
    assert lib.attn_cache_free(r, A, 1, None) == code
    assert lib.attn_cache_compact(r, None, A, 1 << 20, None) == code
    assert lib.attn_cache_write(r, 0, A, A, 1, t, t, 1, None) == code


def test_cache_list_arguments_that_are_refused():
    lib, c = _abi.load(), _cache()
    r = ctypes.byref(c)
    need = lib.attn_cache_workspace_bytes(r, 3)
    assert need > lib.attn_cache_workspace_bytes(r, 0) > 0 or need == lib.attn_cache_workspace_bytes(r, 0)
    assert lib.attn_cache_workspace_bytes(r, -1) == 0 and lib.attn_cache_workspace_bytes(None, 1) == 0
    for ws, size in ((None, need), (A + 16, need), (A, need - 1)):
        assert lib.attn_cache_extend(r, A, A, 3, ws, size, None) == _abi.ATTN_EWORKSPACE
        assert lib.attn_cache_fork(r, A, A, 3, ws, size, None) == _abi.ATTN_EWORKSPACE
        assert lib.attn_cache_keep(r, A, A, A, 2, A, 3, ws, size, None) == _abi.ATTN_EWORKSPACE
    assert lib.attn_cache_compact(r, None, A, 16, None) == _abi.ATTN_EWORKSPACE
    assert lib.attn_cache_extend(r, A, A, -1, A, need, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_extend(r, None, A, 1, A, need, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_fork(r, A, A + 2, 1, A, need, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_keep(r, A, A, None, 2, A, 1, A, need, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_keep(r, A, A, A, -1, A, 1, A, need, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_free(r, None, 1, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_free(r, A, -1, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_compact(r, A + 1, A, need, None) == _abi.ATTN_EINVAL
    # empty lists are no work and no error
    assert lib.attn_cache_extend(r, None, None, 0, A, need, None) == _abi.ATTN_OK
    assert lib.attn_cache_free(r, None, 0, None) == _abi.ATTN_OK


def test_cache_write_arguments_that_are_refused():
    lib, c = _abi.load(), _cache()
    r, good = ctypes.byref(c), ctypes.byref(_abi.AttnTensor(A, 128, 64))
    bad = ctypes.byref(_abi.AttnTensor(A, 129, 64))
    assert lib.attn_cache_write(r, 2, A, A, 1, good, good, 1, None) == _abi.ATTN_EINVAL  # layer
    assert lib.attn_cache_write(r, -1, A, A, 1, good, good, 1, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_write(r, 0, A, A, 1, good, bad, 1, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_write(r, 0, A, None, 1, good, good, 1, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_write(r, 0, A, A, 1, None, good, 1, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_write(r, 0, A, A, 1, good, good, -1, None) == _abi.ATTN_EINVAL
    assert lib.attn_cache_write(r, 0, A, A, 1, good, good, 0, None) == _abi.ATTN_OK


def _tree(cache=None, **kw):
    a = _abi.TreeArgs()
    a.cache = cache or _cache()
    a.layer, a.H, a.n, a.n_q, a.mask_words = 0, 4, 2, 6, 0
    a.q = a.o = _abi.AttnTensor(A, 256, 64)
    a.lse, a.seqs, a.cu = A, A, A
    a.scale, a.o_dtype = 0.125, _abi.ATTN_BF16
    a.workspace, a.workspace_bytes = A, 1 << 30
    for n, x in kw.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("kw,code", [
    ({"layer": 2}, _abi.ATTN_EINVAL), ({"layer": -1}, _abi.ATTN_EINVAL), ({"H": 3}, _abi.ATTN_EINVAL),
    ({"H": 0}, _abi.ATTN_EINVAL), ({"n": -1}, _abi.ATTN_EINVAL), ({"n_q": -1}, _abi.ATTN_EINVAL),
    ({"o_dtype": _abi.ATTN_F16}, _abi.ATTN_EINVAL), ({"scale": float("nan")}, _abi.ATTN_EINVAL),
    ({"scale": float("inf")}, _abi.ATTN_EINVAL), ({"seqs": None}, _abi.ATTN_EINVAL), ({"cu": A + 2}, _abi.ATTN_EINVAL),
    ({"q": _abi.AttnTensor(A, 257, 64)}, _abi.ATTN_EINVAL), ({"o": _abi.AttnTensor(None, 256, 64)}, _abi.ATTN_EINVAL),
    ({"mask": A, "mask_words": 0}, _abi.ATTN_EINVAL), ({"mask": A + 4, "mask_words": 1}, _abi.ATTN_EINVAL),
    ({"mask_words": -1}, _abi.ATTN_EINVAL), ({"lse": A + 2}, _abi.ATTN_EINVAL),
    ({"n_q": 1 << 30}, _abi.ATTN_EUNSUPPORTED),
    ({"workspace": None}, _abi.ATTN_EWORKSPACE), ({"workspace": A + 64}, _abi.ATTN_EWORKSPACE),
    ({"workspace_bytes": 256}, _abi.ATTN_EWORKSPACE),
])
def test_tree_arguments_that_are_refused(kw, code):
    assert _abi.load().attn_tree_fwd(ctypes.byref(_tree(**kw)), None) == code


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS)
def test_tree_refuses_bad_caches(kw, code):
    lib, a = _abi.load(), _tree(_cache(**kw))
    assert lib.attn_tree_fwd(ctypes.byref(a), None) == code
    assert lib.attn_tree_workspace_bytes(ctypes.byref(a)) == 0
    assert lib.attn_tree_fwd(None, None) == _abi.ATTN_EINVAL


@pytest.mark.parametrize("H_kv", [-1, 3, 8])
def test_head_counts_that_do_not_divide_are_refused(H_kv):
    lib = _abi.load()
    f, b = _abi.FwdArgs(), _abi.BwdArgs()
    for a in (f, b):
        for n in ("q", "k", "v", "o"):
            setattr(a, n, _abi.AttnTensor(A, 256, 64))
        a.lse, a.n_q, a.n_k, a.H, a.D, a.n_seq, a.H_kv = A, 64, 64, 4, 64, 1, H_kv
        a.scale, a.relation, a.workspace, a.workspace_bytes = 0.125, _abi.ATTN_CAUSAL, A, 1 << 30
    for n in ("dout", "dq", "dk", "dv"):
        setattr(b, n, _abi.AttnTensor(A, 256, 64))
    assert lib.attn_fwd(ctypes.byref(f), None) == _abi.ATTN_EINVAL
    assert lib.attn_bwd(ctypes.byref(b), None) == _abi.ATTN_EINVAL


def test_no_pages_has_a_message():
    assert attn.strerror(_abi.ATTN_ENOPAGES) == "too few free cache pages"


def test_the_python_cache_needs_cuda_tensors():
    import torch
    k = torch.zeros(1, 4, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.Cache(k, k.clone(), i, i[:, 0].contiguous(), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="layers, pages"):
        attn.Cache(k[0], k[0], i, i[:, 0].contiguous(), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        attn.Cache(k.to(torch.int8), k.to(torch.int8), i, i[:, 0].contiguous(), torch.zeros(4, dtype=torch.int32))


def test_k_and_v_of_two_shapes_are_refused():
    import torch
    q, k, v = (torch.zeros(8, h, 64, dtype=torch.float16) for h in (4, 2, 4))
    with pytest.raises(ValueError, match="k and v must both"):
        attn.fwd(q, k, v, causal=True)


@pytest.mark.parametrize("page", [1, 16, 1024])
def test_positions_keep_clear_of_32_bits(page):
    """A sequence of almost 2^31 tokens: rounding its length up to a tile or a page would overflow."""
    lib, most = _abi.load(), ((1 << 31) - (1 << 16)) // page
    for pages, ok in ((most, True), (most + 1, False), (((1 << 31) - 1) // page, False)):
        c = _cache(page_size=page, max_pages=pages, table_stride=pages)
        assert (lib.attn_cache_workspace_bytes(ctypes.byref(c), 1) > 0) == ok
        assert lib.attn_cache_free(ctypes.byref(c), A, 0, None) == (0 if ok else _abi.ATTN_EUNSUPPORTED)
