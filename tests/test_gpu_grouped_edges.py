"""Grouped heads and the cache at their edges: many and long sequences, wide
groups, empty keys, stale rows, offsets past 32 bits, bad offsets, streams,
graphs, bounded waits; and the compiled binding beside the Python one."""
import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import assert_output, attention, seen_tree
from online_softmax_attention_gb300 import _abi
from test_gpu_grouped import make as make_packed
from test_gpu_grouped import reference
from test_gpu_tree import make, run

pytestmark = pytest.mark.gpu


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def cross(lens_q, lens_k, hq, hkv, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(lens_q), hq, d, generator=g).to(dtype)
    k, v = (torch.randn(sum(lens_k), hkv, d, generator=g).to(dtype) for _ in range(2))
    return q, k, v


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("lens_q,lens_k", [([5, 70, 0, 33], [0, 300, 7, 129]), ([200], [1]), ([1, 1, 1], [128, 0, 257])])
def test_cross_lengths_and_empty_keys(lens_q, lens_k, dtype, d):
    q, k, v = cross(lens_q, lens_k, 6, 2, d, dtype, 51)
    o, lse = attn.fwd(q.cuda(), k.cuda(), v.cuda(), cu_seqlens_q=cu_of(lens_q), cu_seqlens_k=cu_of(lens_k))
    cq, ck = np.cumsum([0] + lens_q), np.cumsum([0] + lens_k)
    for i, (n, m) in enumerate(zip(lens_q, lens_k)):
        rq, rk = slice(cq[i], cq[i + 1]), slice(ck[i], ck[i + 1])
        assert_output(o[rq], lse[:, rq], attention(q[rq], k[rk], v[rk], np.ones((n, m), bool), d ** -0.5), dtype, f"{i}")
        if m == 0:
            assert (o[rq] == 0).all() and (lse[:, rq] == -torch.inf).all()
    assert attn.device_status() == 0


@pytest.mark.parametrize("n_seq", [500, 2048, 2100])
def test_many_sequences(n_seq):
    """More sequences than one scan step, and the most and more than the packed kernel takes."""
    r = np.random.default_rng(52)
    lens = [int(x) for x in r.integers(0, 40, n_seq)]
    x, cu = make_packed(lens, 4, 2, 64, torch.float16, 52)
    c = {n: t.cuda() for n, t in x.items()}
    o, lse = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu)
    for i in list(r.choice(n_seq, 40, replace=False)) + [0, n_seq - 1]:
        m = slice(int(cu[i]), int(cu[i + 1]))
        n = lens[i]
        want = attention(x["q"][m], x["k"][m], x["v"][m], np.tril(np.ones((n, n), bool)), 0.125)
        assert_output(o[m], lse[:, m], want, torch.float16, f"sequence {i}")
    assert attn.device_status() == 0


@pytest.mark.parametrize("hq,hkv", [(128, 1), (127, 1), (160, 1), (65, 1), (96, 2)])
def test_wide_groups(hq, hkv):
    """Groups that fill a tile, do not divide it, and are wider than it."""
    lens = [3, 40]
    x, cu = make_packed(lens, hq, hkv, 64, torch.bfloat16, 53)
    o, lse = attn.fwd(*(x[n].cuda() for n in "qkv"), causal=True, cu_seqlens_q=cu)
    assert_output(o, lse, reference(x, lens, 0.125), torch.bfloat16)
    cache, model, seqs, g = make([70, 5], 16, hkv, 64, torch.bfloat16, 54)
    for news in ([1, 1], [3, 2]):
        q = torch.randn(sum(news), hq, 64, generator=g).bfloat16()
        run(cache, model, seqs, news, q, what=f"{news}")


@pytest.mark.parametrize("hq,hkv,n", [(6, 2, 9000), (20, 4, 5003), (8, 1, 4096)])
def test_long_prompts(hq, hkv, n):
    """Many units a head (their tiles are summed in closed form), cut between blocks: sampled rows."""
    lens = [n, 700]
    x, cu = make_packed(lens, hq, hkv, 128, torch.bfloat16, 55)
    c = {k: t.cuda() for k, t in x.items()}
    o, lse = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu)
    rows = [0, 1, 31, 32, 63, 64, 127, 128, 1000, 2047, 2048, n // 2, n - 130, n - 2, n - 1]
    k, v = x["k"][:n], x["v"][:n]
    seen = np.arange(n)[None, :] <= np.array(rows)[:, None]
    assert_output(o[rows], lse[:, rows], attention(x["q"][rows], k, v, seen, 128 ** -0.5), torch.bfloat16)
    m = slice(n, n + 700)
    want = attention(x["q"][m], x["k"][m], x["v"][m], np.tril(np.ones((700, 700), bool)), 128 ** -0.5)
    assert_output(o[m], lse[:, m], want, torch.bfloat16)


@pytest.mark.parametrize("tree", [False, True])
def test_long_chunks_over_the_cache(tree):
    cache, model, seqs, g = make([1000, 730, 65], 16, 2, 64, torch.float16, 56)
    news = [700, 0, 65]
    q = torch.randn(765, 10, 64, generator=g).half()
    r = np.random.default_rng(57)
    run(cache, model, seqs, news, q, r.integers(0, 1 << 63, (765, 11)).astype(np.uint64) if tree else None)


def test_rows_of_others_do_not_leak():
    """NaN behind the last sequence and in another one: the rest is as without it."""
    lens = [100, 60, 33]
    x, cu = make_packed(lens + [64], 8, 2, 64, torch.bfloat16, 58)
    clean = {n: t.cuda() for n, t in x.items()}
    want = attn.fwd(clean["q"], clean["k"], clean["v"], causal=True, cu_seqlens_q=cu[:4])
    dirty = {n: t.clone() for n, t in clean.items()}
    for t in dirty.values():
        t[193:] = float("nan")
        t[100:160] = float("nan")
    got = attn.fwd(dirty["q"], dirty["k"], dirty["v"], causal=True, cu_seqlens_q=cu[:4])
    for rows in (slice(0, 100), slice(160, 193)):
        assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][:, rows], want[1][:, rows])


@pytest.mark.parametrize("cq,ck", [([0, 30, 64], [0, 20, 64]), ([0, 70, 64], [0, 70, 64]), ([0, 30, 90], [0, 30, 90]),
                                   ([-5, 30, 64], [-5, 30, 64])])
def test_bad_offsets_are_reported(cq, ck):
    x, _ = make_packed([64], 4, 2, 64, torch.float16, 59)
    c = {n: t.cuda() for n, t in x.items()}
    attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=torch.tensor(cq, dtype=torch.int32).cuda(),
             cu_seqlens_k=torch.tensor(ck, dtype=torch.int32).cuda())
    assert attn.device_status() == _abi.ATTN_EINVAL
    assert attn.device_status() == 0


def test_offsets_past_32_bits_in_a_cache():
    """Pools of more than 2^32 bytes, the sequences' pages at their end; and the operations there."""
    page, heads, d, n_pages = 128, 8, 128, 20000
    k, v = (torch.empty(1, n_pages, page, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 31
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[:19000] = 1
    table = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    cache = attn.Cache(k, v, table, torch.zeros(4, dtype=torch.int32, device="cuda"), refs)
    lens = [300, 77]
    g = torch.Generator().manual_seed(60)
    kr, vr = (torch.randn(377, heads, d, generator=g).bfloat16() for _ in range(2))
    cache.extend([0, 1], lens)
    cache.write([0, 1], [0, 300, 377], kr.cuda(), vr.cuda())
    assert int(table[0, 0]) == 19000
    cache.fork([0], [2])
    cache.keep([0], [4], torch.tensor([[1, 3]]), [2])  # rows 297, 299 follow row 295
    kept = list(range(296)) + [297, 299]
    for seq, rows in ((0, kept), (2, list(range(300))), (1, list(range(300, 377)))):
        for t in (1, 12):  # few and many query rows: both kernels
            q = torch.randn(t, 32, d, generator=g).bfloat16()
            o, lse = attn.tree_fwd(q.cuda(), cache, [seq], [0, t])
            want = attention(q, kr[rows], vr[rows], seen_tree(len(rows), t), d ** -0.5)
            assert_output(o, lse, want, torch.bfloat16, f"{seq} {t}")
    refs[:19000] = 0
    cache.compact()
    assert int(table[[0, 1, 2]].max()) < 8
    q = torch.randn(1, 32, d, generator=g).bfloat16()
    o, lse = attn.tree_fwd(q.cuda(), cache, [0], [0, 1])
    assert_output(o, lse, attention(q, kr[kept], vr[kept], seen_tree(298, 1), d ** -0.5), torch.bfloat16)
    assert attn.device_status() == 0


def test_offsets_past_32_bits_in_a_prompt():
    """Heads 2^31 elements apart."""
    T, hq, hkv, d = 200, 4, 2, 64
    far = (1 << 31) + 64

    def spread(t):
        buf = torch.empty((t.shape[1] - 1) * far + t.shape[0] * d, dtype=t.dtype, device="cuda")
        view = buf.as_strided(t.shape, (d, far, 1))
        view.copy_(t)
        return view

    x, _ = make_packed([T], hq, hkv, d, torch.float16, 61)
    q, k, v = (spread(x[n].cuda()) for n in "qkv")
    out = spread(torch.zeros(T, hq, d, dtype=torch.float16))
    call = attn.FwdCall(q, k, v, causal=True, out=out)
    o, lse = call.run()
    assert_output(o.contiguous(), lse, reference(x, [T], 0.125), torch.float16)
    do = spread(torch.randn(T, hq, d, generator=torch.Generator().manual_seed(62)).half())
    got = attn.bwd(q, k, v, o, lse, do, causal=True)
    near = attn.bwd(*(t.contiguous() for t in (q, k, v, o)), lse, do.contiguous(), causal=True)
    assert all(torch.equal(a, b) for a, b in zip(got, near))


def test_streams_and_graphs():
    lens = [200, 90]
    x, cu = make_packed(lens, 8, 2, 128, torch.bfloat16, 63)
    c, dcu = {n: t.cuda() for n, t in x.items()}, cu.cuda()
    want = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=dcu)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=dcu))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(lse, want[1]) for o, lse in got)
    call = attn.FwdCall(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=dcu)
    call.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    for cut in (200, 1, 289):
        dcu.copy_(torch.tensor([0, cut, 290], dtype=torch.int32))
        graph.replay()
        assert_output(call.o, call.lse, reference(x, [cut, 290 - cut], 128 ** -0.5), torch.bfloat16, f"cut {cut}")


def test_bounded_waits_of_the_packed_kernel():
    """As for the other tensor-core kernels: a tiny budget runs out, is reported, and the next calls are whole."""
    lib = _abi.load()
    x, cu = make_packed([2000, 300], 8, 2, 128, torch.bfloat16, 64)
    c = {n: t.cuda() for n, t in x.items()}
    cache, _, seqs, g = make([900, 400], 64, 2, 128, torch.bfloat16, 65)
    q = torch.randn(60, 8, 128, generator=g).bfloat16().cuda()
    want = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu)
    want_tree = attn.tree_fwd(q, cache, seqs, [0, 30, 60])
    assert attn.device_status() == 0
    prev = lib.attn_set_watchdog_cycles(64)
    try:
        attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu)
        assert attn.device_status() == _abi.ATTN_ETIMEOUT
        attn.tree_fwd(q, cache, seqs, [0, 30, 60])
        assert attn.device_status() == _abi.ATTN_ETIMEOUT
    finally:
        lib.attn_set_watchdog_cycles(prev if prev != 4000000000 else 0)
    got = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu)
    got_tree = attn.tree_fwd(q, cache, seqs, [0, 30, 60])
    assert attn.device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got_tree[0], want_tree[0])


def test_both_bindings_make_the_same_calls():
    """Tensors take the compiled binding, lists the Python one."""
    lens = [50, 14]
    x, cu = make_packed(lens, 6, 2, 64, torch.float16, 66, True)
    c, dcu = {n: t.cuda() for n, t in x.items()}, cu.cuda()
    for kw in ({}, {"scale": 0.2}, {"out_dtype": torch.float32}):
        a = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=dcu, **kw)
        b = attn.fwd(c["q"], c["k"], c["v"], causal=1, cu_seqlens_q=cu.tolist(), **kw)
        assert all(torch.equal(p, q) and p.dtype == q.dtype for p, q in zip(a, b))
    o, lse = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=dcu)
    for kw in ({}, {"grad_dtype": torch.float32}):
        a = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], causal=True, cu_seqlens_q=dcu, **kw)
        b = attn.bwd(c["q"], c["k"], c["v"], o, lse, c["do"], causal=1, cu_seqlens_q=cu.tolist(), **kw)
        assert all(torch.equal(p, q) and p.dtype == q.dtype for p, q in zip(a, b))
    cache, _, seqs, g = make([60, 70], 16, 2, 64, torch.float16, 67)
    q = torch.randn(7, 6, 64, generator=g).half().cuda()
    ds, dc = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in (seqs, [0, 3, 7]))
    mask = torch.full((7, 1), 0b1011, device="cuda")
    for kw in ({}, {"mask": mask}, {"scale": 0.3, "out_dtype": torch.float32}):
        a, b = attn.tree_fwd(q, cache, ds, dc, **kw), attn.tree_fwd(q, cache, seqs, [0, 3, 7], **kw)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    # errors of the library come through either
    for lists in ((ds, dc), (seqs, [0, 3, 7])):
        with pytest.raises(attn.AttnError) as e:
            attn.tree_fwd(q[:, :5], cache, *lists)
        assert e.value.code == _abi.ATTN_EINVAL
    with pytest.raises(attn.AttnError):
        attn.fwd(c["q"][:, :5], c["k"], c["v"], cu_seqlens_q=dcu)
    with pytest.raises((TypeError, ValueError)):
        attn.tree_fwd(q.bfloat16(), cache, ds, dc)
    with pytest.raises(ValueError):
        attn.tree_fwd(q, cache, ds, dc[:2])
    with pytest.raises(ValueError):
        cache.write(ds, dc, q, q)  # six heads, not two
    with pytest.raises(ValueError):
        cache.extend(ds, dc)


@pytest.mark.parametrize("page,news", [(256, [40, 1]), (1024, [40, 30]), (8, [33, 64])])
def test_page_sizes_around_a_key_tile(page, news):
    cache, model, seqs, g = make([1500, 130], page, 2, 128, torch.bfloat16, 68, layout="hnd")
    q = torch.randn(sum(news), 8, 128, generator=g).bfloat16()
    run(cache, model, seqs, news, q, what=f"page {page}")


def test_fp8_and_pruned_forwards_with_shared_heads():
    """The forward's other options map key heads too: as on repeated heads, bit for bit."""
    x, _ = make_packed([300], 8, 2, 128, torch.bfloat16, 69)
    q, k, v = (x[n].cuda() for n in "qkv")
    k4, v4 = k.repeat_interleave(4, 1), v.repeat_interleave(4, 1)
    e4m3 = torch.float8_e4m3fn
    a = attn.fwd(q.to(e4m3), k.to(e4m3), v, causal=True)
    b = attn.fwd(q.to(e4m3), k4.to(e4m3), v4, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = attn.fwd(q, k, v, prune_threshold=0.5), attn.fwd(q, k4, v4, prune_threshold=0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_the_allocation_free_forward_with_shared_heads():
    import ctypes
    lib = _abi.load()
    lens = [200, 30]
    x, cu = make_packed(lens, 8, 2, 64, torch.float16, 70)
    c = {n: t.cuda() for n, t in x.items()}
    want = attn.fwd(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu, num_splits=1)
    call = attn.FwdCall(c["q"], c["k"], c["v"], causal=True, cu_seqlens_q=cu)
    call.args.workspace, call.args.workspace_bytes = None, 0
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.attn_fwd_noalloc(ctypes.byref(call.args), s) == 0
    assert torch.equal(call.o, want[0]) and torch.equal(call.lse, want[1])


def test_one_sequence_in_two_entries():
    """Reads may name a sequence twice: the same queries give the same rows."""
    cache, _, seqs, g = make([500, 60], 16, 2, 64, torch.float16, 71)
    q = torch.randn(3, 8, 64, generator=g).half().cuda()
    o, lse = attn.tree_fwd(torch.cat([q, q]), cache, [seqs[0], seqs[0]], [0, 3, 6])
    one = attn.tree_fwd(q, cache, [seqs[0]], [0, 3])
    # (cuts differ with the number of entries: equal up to rounding)
    assert torch.allclose(o[:3].float(), one[0].float(), atol=2e-3, rtol=2e-3)
    assert torch.allclose(o[3:].float(), one[0].float(), atol=2e-3, rtol=2e-3)
    assert torch.allclose(lse[:, :3], one[1], atol=1e-4) and torch.allclose(lse[:, 3:], one[1], atol=1e-4)


def test_caches_that_are_refused():
    k = torch.zeros(1, 4, 16, 2, 64, dtype=torch.float16, device="cuda")
    i = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    n, r = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (2, 4))
    with pytest.raises(ValueError, match="same strides"):
        attn.Cache(k, k.permute(0, 1, 3, 2, 4).contiguous().permute(0, 1, 3, 2, 4), i, n, r)
    with pytest.raises(ValueError, match="contiguous rows"):
        attn.Cache(k, k.clone(), i.t(), r, r)
    with pytest.raises(TypeError):
        attn.Cache(k, k.clone(), i.long(), n, r)
    with pytest.raises(ValueError, match="unsupported"):
        attn.Cache(k[:, :, :12], k.clone()[:, :, :12], i, n, r)
    with pytest.raises(ValueError, match="one CUDA device"):
        attn.Cache(k, k.clone(), i.cpu(), n, r)
    c = attn.Cache(k, k.clone(), i, n, r)
    with pytest.raises(ValueError, match="32 bits"):
        c.free([1 << 32])
    with pytest.raises(ValueError):
        c.compact(remap=i)


LOW = -2 ** 31


@pytest.mark.parametrize("cq,ck,causal", [([0, 64, LOW], [0, 64, LOW], True), ([0, 1, LOW], [0, 64, 64], False),
                                          ([0, 64, 64], [0, 1, LOW], False), ([LOW, 64], [LOW, 64], True),
                                          ([3, 64], [3, 64], True)])
def test_offsets_whose_difference_wraps_are_refused(cq, ck, causal):
    x, _ = make_packed([64], 4, 2, 64, torch.float16, 71)
    c = {n: t.cuda() for n, t in x.items()}
    attn.fwd(c["q"], c["k"], c["v"], causal=causal, cu_seqlens_q=torch.tensor(cq, dtype=torch.int32).cuda(),
             cu_seqlens_k=torch.tensor(ck, dtype=torch.int32).cuda())
    assert attn.device_status() == _abi.ATTN_EINVAL
    assert attn.device_status() == 0


@pytest.mark.parametrize("cu", [[LOW, 3, 40], [-5, 3, 40], [0, LOW, 40], [0, 1, LOW]])
def test_cache_offsets_below_zero_are_refused(cu):
    cache, _, seqs, g = make([50, 60], 16, 2, 64, torch.float16, 72)
    before = cache.k.clone()
    offsets = torch.tensor(cu, dtype=torch.int32).cuda()
    rows = torch.randn(40, 2, 64, generator=g).half().cuda()
    free = torch.tensor([i for i in range(4) if i not in seqs][:2], dtype=torch.int32).cuda()  # of length 0
    for list_ in (free, torch.tensor(seqs, dtype=torch.int32).cuda()):
        attn.device_status()
        cache.write(list_, offsets, rows, rows)
        entry = range(2) if list_ is free else [i for i in range(2) if not 0 <= cu[i] <= cu[i + 1] <= 40]
        for i in entry:  # (a valid entry's rows are written)
            for page in cache.table[int(list_[i])].tolist():
                if 0 <= page < cache.k.shape[1]:
                    assert torch.equal(cache.k[:, page].view(torch.int16), before[:, page].view(torch.int16))
        if list_ is free or cu[2] == 40:
            assert attn.device_status() == _abi.ATTN_EINVAL
        for heads in (2, 8):  # the 16-row kernel, the packed one
            call = attn.TreeCall(torch.randn(40, heads, 64, generator=g).half().cuda(), cache, list_, offsets)
            call.o.fill_(5.0)
            o, _ = call.run()
            for i in entry:
                if 0 <= cu[i] < cu[i + 1]:
                    assert (o[cu[i]:cu[i + 1]] == 5).all()
            assert attn.device_status() == _abi.ATTN_EINVAL


@pytest.mark.parametrize("dtype,n,news,heads", [(torch.bfloat16, 9000, 1, 4), (torch.float32, 9000, 1, 4),
                                                (torch.float16, 9000, 40, 8)])
def test_a_query_of_nan_gives_nan_in_cut_units(dtype, n, news, heads):
    """One long sequence, whose units are cut between blocks: its parts are merged."""
    cache, _, seqs, g = make([n], 16, 1, 64, dtype, 73)
    q = torch.randn(news, heads, 64, generator=g).to(dtype)
    q[0, 1] = float("nan")
    o, _ = attn.tree_fwd(q.cuda(), cache, seqs, [0, news])
    want = torch.zeros(news, heads, dtype=torch.bool)
    want[0, 1] = True
    assert torch.equal(o.isnan().all(2).cpu(), want) and torch.equal(o.isnan().any(2).cpu(), want)


def test_a_query_of_nan_gives_nan_in_a_cut_prompt():
    x, cu = make_packed([6000], 8, 1, 128, torch.bfloat16, 74)
    x["q"][4500, 3] = float("nan")
    o, _ = attn.fwd(*(x[n].cuda() for n in "qkv"), causal=True, cu_seqlens_q=cu)
    want = torch.zeros(6000, 8, dtype=torch.bool)
    want[4500, 3] = True
    assert torch.equal(o.isnan().all(2).cpu(), want) and torch.equal(o.isnan().any(2).cpu(), want)


def test_as_many_units_as_heads_and_sequences_allow():
    """2048 sequences of one token and 4096 key heads, a unit each: the output is the token's value row."""
    n, hkv = 2048, 4096
    g = torch.Generator(device="cuda").manual_seed(75)
    q = torch.randn(n, 2 * hkv, 64, generator=g, device="cuda", dtype=torch.float16)
    k, v = (torch.randn(n, hkv, 64, generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    call = attn.FwdCall(q, k, v, causal=True, cu_seqlens_q=cu, out=torch.full_like(q, 5.0))
    o, _ = call.run()
    assert attn.device_status() == 0
    # one key: p = 1 and l = 1 exactly
    assert torch.equal(o.view(n, hkv, 2, 64), v.unsqueeze(2).expand(n, hkv, 2, 64))


def test_more_key_heads_than_the_packed_kernel_takes():
    hkv = (1 << 14) + 1
    x, cu = make_packed([1, 1], 2, 1, 64, torch.float16, 76)
    q, k, v = (x[n].cuda().repeat(1, hkv, 1) for n in "qkv")
    o, _ = attn.fwd(q, k, v, causal=True, cu_seqlens_q=cu)
    assert torch.equal(o, v.repeat_interleave(2, 1)) and attn.device_status() == 0
