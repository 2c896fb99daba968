"""Attention of new tokens over the cache, with a sliding window and sinks, against f64."""
import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import assert_output, attention, seen_tree
from online_softmax_attention_gb300 import _abi
from test_gpu_tree import make, random_mask
from window_model import windowed

pytestmark = pytest.mark.gpu


def run(cache, model, seqs, news, q, window, sinks, mask=None, what="", **kw):
    cu = [0] + [int(x) for x in np.cumsum(news)]
    tm = None if mask is None else torch.from_numpy(mask.view(np.int64)).cuda()
    o, lse = attn.tree_fwd(q.cuda(), cache, seqs, cu, mask=tm, window=window, sinks=sinks, **kw)
    for i, s in enumerate(seqs):
        rows = slice(cu[i], cu[i + 1])
        k, v = model.rows(s, 0)
        seen = windowed(seen_tree(len(k), news[i], None if mask is None else mask[rows]), window, sinks)
        want = attention(q[rows], k, v, seen, kw.get("scale", q.shape[2] ** -0.5))
        assert_output(o[rows], lse[:, rows], want, q.dtype, f"{what} {window}+{sinks} entry {i}")
    assert attn.device_status() == 0
    return o, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,page,heads,group", [([1], 16, 1, 1), ([700], 16, 2, 4), ([5, 1, 64, 333, 31, 32, 33], 8, 2, 3),
                                                   ([2000, 3], 128, 1, 8), ([40] * 20, 1, 1, 5), ([400], 1024, 2, 16)])
def test_decoding(lens, page, heads, group, d, dtype):
    cache, model, seqs, g = make(lens, page, heads, d, dtype, 71)
    q = torch.randn(len(lens), heads * group, d, generator=g).to(dtype)
    for window, sinks in ((1, 0), (1, 1), (33, 4), (32, 0), (100, 40), (5, 2 ** 31 - 1)):
        run(cache, model, seqs, [1] * len(lens), q, window, sinks, what=f"{lens}")


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 64)])
@pytest.mark.parametrize("lens,news,page,heads,group", [
    ([7], [7], 16, 1, 2), ([300, 41, 9], [5, 41, 1], 32, 2, 4), ([64, 65], [64, 63], 64, 1, 3), ([500, 130], [130, 65], 16, 2, 1),
    ([90, 1000, 4], [0, 17, 2], 8, 1, 8), ([257], [33], 128, 4, 5), ([900, 70], [3, 2], 16, 2, 2), ([900, 70], [9, 2], 4, 2, 4)])
@pytest.mark.parametrize("tree", [False, True])
def test_chunks_and_trees(lens, news, page, heads, group, d, dtype, tree):
    cache, model, seqs, g = make(lens, page, heads, d, dtype, 72)
    q = torch.randn(sum(news), heads * group, d, generator=g).to(dtype)
    mask = random_mask(news, 3, np.random.default_rng(73)) if tree else None
    for window, sinks in ((1, 0), (3, 2), (20, 9), (64, 130), (140, 1)):
        run(cache, model, seqs, news, q, window, sinks, mask, what=f"{lens} {news}")


@pytest.mark.parametrize("dtype,group", [(torch.bfloat16, 2), (torch.bfloat16, 8), (torch.float32, 2)])
def test_rows_that_see_nothing(dtype, group):
    """No prefix and an empty mask row; a prefix alone still counts, its last tokens and the sinks."""
    news = [6, 3]
    cache, model, seqs, g = make([6, 40], 16, 2, 64, dtype, 74)
    q = torch.randn(9, 2 * group, 64, generator=g).to(dtype)
    mask = np.zeros((9, 1), np.uint64)
    mask[1, 0], mask[4, 0] = 1, 0b101
    o, lse = run(cache, model, seqs, news, q, 2, 1, mask)
    assert (o[[0, 2, 3, 5]] == 0).all() and (lse[:, [0, 2, 3, 5]] == -torch.inf).all()


def test_long_contexts_are_read_only_in_the_window():
    """Pages between the sinks' tile and the window's first one may be gone: their entries in the
    table are not followed."""
    cache, model, seqs, g = make([5000, 4000], 64, 2, 128, torch.bfloat16, 75)
    q1, q2 = torch.randn(2, 8, 128, generator=g).bfloat16(), torch.randn(40, 8, 128, generator=g).bfloat16()
    cache.table[seqs[0], 2:50] = -1
    cache.table[seqs[1], 2:40] = -1
    first = run(cache, model, seqs, [1, 1], q1, 1000, 4)
    run(cache, model, seqs, [30, 10], q2, 1000, 4)
    for _ in range(2):
        again = attn.tree_fwd(q1.cuda(), cache, seqs, [0, 1, 2], window=1000, sinks=4)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("t", [1, 20])
def test_a_window_as_long_as_a_sequence_can_be_is_none(t):
    cache, model, seqs, g = make([300], 16, 2, 64, torch.float16, 76)
    q = torch.randn(t, 8, 64, generator=g).half().cuda()
    plain = attn.tree_fwd(q, cache, seqs, [0, t])
    for window in (16 * cache.table.shape[1], 2 ** 31 - 1):
        wide = attn.tree_fwd(q, cache, seqs, [0, t], window=window, sinks=9)
        assert all(torch.equal(a, b) for a, b in zip(plain, wide))
    run(cache, model, seqs, [t], q.cpu(), 300, 0)


def test_layouts_scales_and_graphs():
    cache, model, seqs, g = make([210, 77], 32, 2, 128, torch.bfloat16, 77, layout="hnd")
    q = torch.randn(9, 8, 128, generator=g).bfloat16()
    run(cache, model, seqs, [4, 5], q, 40, 3, out_dtype=torch.float32, scale=-0.2)
    call = attn.TreeCall(q.cuda(), cache, seqs, [0, 4, 9], window=40, sinks=3)
    call.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    cache.lens[seqs[0]], cache.lens[seqs[1]] = 150, 9
    graph.replay()
    want = attn.tree_fwd(q.cuda(), cache, seqs, [0, 4, 9], window=40, sinks=3)
    assert torch.equal(call.o, want[0]) and torch.equal(call.lse, want[1])
    for bad in (dict(window=0), dict(sinks=1), dict(window=5, sinks=-1)):
        with pytest.raises(ValueError):
            attn.tree_fwd(q.cuda(), cache, seqs, [0, 4, 9], **bad)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_a_prompt_and_its_decoding_are_one_attention(dtype, d):
    """The prompt through the windowed forward, then tokens over the cache: the rows of one windowed prompt."""
    n, more, window, sinks = 150, 6, 50, 3
    g = torch.Generator().manual_seed(78)
    q, k, v = (torch.randn(n + more, h, d, generator=g).to(dtype).cuda() for h in (8, 2, 2))
    whole = attn.fwd(q, k, v, causal=True, window=window, sinks=sinks)
    cache = attn.Cache.empty(1, 20, 16, 2, d, max_seqs=2, max_pages=12, dtype=dtype)
    o, lse = attn.fwd(q[:n], k[:n], v[:n], causal=True, window=window, sinks=sinks)
    cache.extend([1], [n])
    cache.write([1], [0, n], k[:n], v[:n])
    for t in range(n, n + more):
        cache.extend([1], [1])
        cache.write([1], [0, 1], k[t:t + 1], v[t:t + 1])
        a, b = attn.tree_fwd(q[t:t + 1], cache, [1], [0, 1], window=window, sinks=sinks)
        o, lse = torch.cat([o, a]), torch.cat([lse, b], 1)
    # both are within the type's bound of the same values
    step = 2 * (2.0 ** -8 if dtype == torch.bfloat16 else 1e-5)
    assert (o - whole[0]).abs().max() <= step * (1 + whole[0].abs().max()) and (lse - whole[1]).abs().max() <= 2e-3
    assert attn.device_status() == 0


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 64)])
@pytest.mark.parametrize("lens,news,page,heads,group", [([700, 95], [1, 1], 16, 2, 4), ([700, 400], [3, 2], 32, 2, 2),
                                                        ([900, 600], [40, 20], 64, 2, 4), ([700], [30], 8, 1, 2),
                                                        ([2000], [1100], 16, 1, 2), ([2100, 1700], [1100, 70], 128, 1, 3)])
@pytest.mark.parametrize("window,sinks", [(50, 0), (33, 5), (200, 130)])
def test_tokens_that_no_row_sees_may_hold_anything(lens, news, page, heads, group, window, sinks, dtype, d):
    cache, _, seqs, g = make(lens, page, heads, d, dtype, 78)
    q = torch.randn(sum(news), heads * group, d, generator=g).to(dtype).cuda()
    cu = [0] + [int(x) for x in np.cumsum(news)]
    mask = torch.from_numpy(random_mask(news, -(-max(news) // 64), np.random.default_rng(79)).view(np.int64)).cuda()
    calls = [dict(mask=m, window=window, sinks=sinks) for m in (None, mask)]
    want = [attn.tree_fwd(q, cache, seqs, cu, **kw) for kw in calls]
    for s, n, t in zip(seqs, lens, news):
        hidden = torch.arange(sinks, max(sinks, n - t - window), device="cuda")
        pages = cache.table[s].long()[hidden // page]
        cache.k[:, pages, hidden % page] = float("nan")
        cache.v[:, pages, hidden % page] = torch.inf
    for kw, w in zip(calls, want):
        got = attn.tree_fwd(q, cache, seqs, cu, **kw)
        assert torch.isfinite(got[0]).all()
        assert all(torch.equal(a, b) for a, b in zip(got, w)), kw["mask"] is None
    assert attn.device_status() == 0


def test_two_streams_at_once():
    """Prepared calls of both kernels, on two streams over one cache."""
    cache, _, seqs, g = make([3000, 1700, 900], 16, 2, 128, torch.bfloat16, 80)
    calls = []
    for t in (1, 40):
        q = torch.randn(3 * t, 8, 128, generator=g).bfloat16().cuda()
        calls += [attn.TreeCall(q, cache, seqs, [0, t, 2 * t, 3 * t], window=w, sinks=4) for w in (600, 90)]
    want = []
    for c in calls:
        c.run()
        want.append((c.o.clone(), c.lse.clone()))
        c.o.fill_(9)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    for c, (o, lse) in zip(calls, want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


def test_offsets_that_go_back():
    """Entries that fit are carried out, more units than offsets in order can have among them; the others are reported."""
    cache, model, seqs, g = make([700, 90], 16, 2, 64, torch.bfloat16, 96)
    a, b = seqs
    q = torch.randn(3, 32, 64, generator=g).bfloat16()
    o, lse = attn.tree_fwd(q.cuda(), cache, [a, b, a, b, a], [0, 3, 0, 3, 0, 3], window=100, sinks=3)
    assert attn.device_status() == _abi.ATTN_EINVAL
    k, v = model.rows(a, 0)
    assert_output(o, lse, attention(q, k, v, windowed(seen_tree(len(k), 3, None), 100, 3), 0.125), torch.bfloat16)


@pytest.mark.parametrize("n,heads,group", [(600, 2, 4), (512, 1, 4), (40, 1, 20), (33, 2, 2)])
def test_many_entries(n, heads, group):
    """Some without new tokens, some with several, more than a cluster counts at once."""
    r = np.random.default_rng(97)
    lens = [int(x) for x in r.integers(1, 90, n)]
    news = [int(min(x, y)) for x, y in zip(r.choice([0, 1, 1, 1, 2, 5], n), lens)]
    cache, model, seqs, g = make(lens, 16, heads, 64, torch.float16, 98)
    q = torch.randn(sum(news), heads * group, 64, generator=g).half()
    run(cache, model, seqs, news, q, 20, 2, what=f"{n}")
