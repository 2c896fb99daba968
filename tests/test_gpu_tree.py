"""Attention of new tokens over the paged cache against f64."""
import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import Model, assert_output, attention, seen_tree
from online_softmax_attention_gb300 import _abi

pytestmark = pytest.mark.gpu


def make(lens, page, heads, d, dtype, seed, layers=1, layout="nhd", spare=3, junk=float("nan")):
    """A cache whose sequences hold scattered pages of N(0, 1) rows; every other slot holds `junk`."""
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    order = r.permutation(n_pages)
    table = np.full((len(lens) + 2, max(need + [1]) + 1), -5, np.int32)
    ids = r.permutation(len(lens) + 2)[:len(lens)]
    all_lens = np.zeros(len(lens) + 2, np.int32)
    k = torch.full((layers, n_pages, page, heads, d), junk, dtype=dtype)
    v = k.clone()
    at = 0
    for s, n, m in zip(ids, lens, need):
        table[s, :m] = order[at:at + m]
        all_lens[s] = n
        at += m
        for t in range(0, n, page):
            p, rows = table[s, t // page], min(page, n - t)
            k[:, p, :rows], v[:, p, :rows] = (torch.randn(layers, rows, heads, d, generator=g).to(dtype) for _ in range(2))
    refs = np.zeros(n_pages, np.int32)
    refs[order[:at]] = 1
    model = Model(k.double().numpy(), v.double().numpy(), table, all_lens, refs)
    if layout == "hnd":
        k, v = (t.permute(0, 1, 3, 2, 4).contiguous().permute(0, 1, 3, 2, 4) for t in (k, v))
    cache = attn.Cache(k.cuda() if layout == "nhd" else k.permute(0, 1, 3, 2, 4).cuda().permute(0, 1, 3, 2, 4),
                       v.cuda() if layout == "nhd" else v.permute(0, 1, 3, 2, 4).cuda().permute(0, 1, 3, 2, 4),
                       torch.from_numpy(table).cuda(), torch.from_numpy(all_lens).cuda(), torch.from_numpy(refs).cuda())
    return cache, model, [int(s) for s in ids], g


def random_mask(news, words, r):
    rows = r.integers(0, 1 << 63, (sum(news), words)).astype(np.uint64)
    return rows


def run(cache, model, seqs, news, q, mask=None, layer=0, scale=None, out_dtype=None, dtype=None, what=""):
    cu = [0] + [int(x) for x in np.cumsum(news)]
    tm = None if mask is None else torch.from_numpy(mask.view(np.int64)).cuda()
    o, lse = attn.tree_fwd(q.cuda(), cache, seqs, cu, layer=layer, mask=tm, scale=scale, out_dtype=out_dtype)
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for i, s in enumerate(seqs):
        rows = slice(cu[i], cu[i + 1])
        k, v = model.rows(s, layer)
        seen = seen_tree(len(k), news[i], None if mask is None else mask[rows])
        assert_output(o[rows], lse[:, rows], attention(q[rows], k, v, seen, scale), q.dtype, f"{what} entry {i}")
    assert attn.device_status() == 0
    return o, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,page,heads,group", [([1], 16, 1, 1), ([700], 16, 2, 4), ([5, 1, 64, 333, 31, 32, 33], 8, 2, 3),
                                                   ([2000, 3], 128, 1, 8), ([40] * 20, 1, 1, 5), ([129], 1024, 2, 16)])
def test_decoding(lens, page, heads, group, d, dtype):
    cache, model, seqs, g = make(lens, page, heads, d, dtype, 31)
    q = torch.randn(len(lens), heads * group, d, generator=g).to(dtype)
    run(cache, model, seqs, [1] * len(lens), q, what=f"{lens}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,news,page,heads,group", [
    ([7], [7], 16, 1, 2), ([300, 41, 9], [5, 41, 1], 32, 2, 4), ([64, 65], [64, 63], 64, 1, 3),
    ([500, 130], [130, 65], 16, 2, 1), ([90, 1000, 4], [0, 17, 2], 8, 1, 8), ([257], [33], 128, 4, 5)])
@pytest.mark.parametrize("tree", [False, True])
def test_chunks_and_trees(lens, news, page, heads, group, d, dtype, tree):
    cache, model, seqs, g = make(lens, page, heads, d, dtype, 32)
    q = torch.randn(sum(news), heads * group, d, generator=g).to(dtype)
    mask = random_mask(news, 3, np.random.default_rng(33)) if tree else None
    run(cache, model, seqs, news, q, mask, what=f"{lens} {news}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_see_nothing(dtype):
    """No prefix and an empty mask row: o = 0, lse = -inf; a prefix alone still counts."""
    news = [6, 3]
    cache, model, seqs, g = make([6, 40], 16, 2, 64, dtype, 34)
    q = torch.randn(9, 4, 64, generator=g).to(dtype)
    mask = np.zeros((9, 1), np.uint64)
    mask[1, 0], mask[4, 0] = 1, 0b101
    o, lse = run(cache, model, seqs, news, q, mask)
    assert (o[[0, 2, 3, 5]] == 0).all() and (lse[:, [0, 2, 3, 5]] == -torch.inf).all()


@pytest.mark.parametrize("layout,out_dtype,scale", [("hnd", torch.float32, None), ("nhd", torch.bfloat16, -0.2),
                                                    ("hnd", torch.bfloat16, 0.0)])
def test_layouts_layers_and_scales(layout, out_dtype, scale):
    cache, model, seqs, g = make([210, 77], 32, 2, 128, torch.bfloat16, 35, layers=3, layout=layout)
    q = torch.randn(9, 8, 128, generator=g).bfloat16()
    for layer in (2, 0):
        run(cache, model, seqs, [4, 5], q, layer=layer, out_dtype=out_dtype, scale=scale)


def test_query_views_and_given_outputs():
    cache, model, seqs, g = make([90, 20], 16, 2, 64, torch.float16, 36)
    both = torch.randn(6, 12, 64, generator=g).half()
    q = both[:, 2:10]
    out = torch.full((6, 16, 64), 3.0, dtype=torch.float16, device="cuda")
    lse = torch.empty(8, 6, device="cuda")
    call = attn.TreeCall(both.cuda()[:, 2:10], cache, seqs, [0, 2, 5], out=out[:, 4:12], lse=lse)
    lse.fill_(9.0)
    call.run()
    o, l = attn.tree_fwd(q.contiguous().cuda(), cache, seqs, [0, 2, 5])
    assert torch.equal(out[:5, 4:12], o[:5]) and torch.equal(lse[:, :5], l[:, :5])
    assert (out[:, :4] == 3).all() and (out[:, 12:] == 3).all()
    assert (out[5] == 3).all() and (lse[:, 5] == 9).all()  # the row behind the last entry
    del model


@pytest.mark.parametrize("lens,heads,group", [([9000], 1, 2), ([5000, 100, 3000], 2, 4), ([64] * 300, 2, 4)])
def test_long_and_many(lens, heads, group):
    """Sequences cut over many blocks, and many short ones to a block."""
    cache, model, seqs, g = make(lens, 64, heads, 128, torch.bfloat16, 37)
    q = torch.randn(len(lens), heads * group, 128, generator=g).bfloat16()
    first = run(cache, model, seqs, [1] * len(lens), q)
    for _ in range(3):
        again = attn.tree_fwd(q.cuda(), cache, seqs, list(range(len(lens) + 1)))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_entries_that_do_not_fit_are_left():
    cache, model, seqs, g = make([50, 60], 16, 2, 64, torch.float16, 38)
    q = torch.randn(8, 4, 64, generator=g).half()
    for bad_seqs, cu, good in (([seqs[0], 99], [0, 3, 8], [0]), ([-1, seqs[1]], [0, 3, 8], [1]),
                               ([seqs[0], seqs[1]], [0, 3, 9], [0]), ([seqs[0], seqs[1]], [3, 0, 8], [1])):
        call = attn.TreeCall(q.cuda(), cache, bad_seqs, cu)
        call.o.fill_(5.0)
        o, lse = call.run()
        assert attn.device_status() == _abi.ATTN_EINVAL
        for i in range(2):
            rows = slice(cu[i], cu[i + 1]) if cu[i] <= cu[i + 1] <= 8 else slice(0, 0)
            if i in good:
                k, v = model.rows(bad_seqs[i], 0)
                want = attention(q[rows], k, v, seen_tree(len(k), rows.stop - rows.start), 0.125)
                assert_output(o[rows], lse[:, rows], want, torch.float16)
            elif cu[i] == 3:
                assert (o[rows] == 5).all()
    # more new tokens than the sequence has, or than the mask has bits
    for lens, words in (([8, 0], None), ([70, 0], 1)):
        c2, _, s2, g2 = make([lens[0] - 1 if words is None else 80], 16, 2, 64, torch.float16, 39)
        q2 = torch.randn(lens[0], 4, 64, generator=g2).half().cuda()
        mask = None if words is None else torch.full((lens[0], words), -1, device="cuda")
        call = attn.TreeCall(q2, c2, s2, [0, lens[0]], mask=mask)
        call.o.fill_(5.0)
        assert (call.run()[0] == 5).all()
        assert attn.device_status() == _abi.ATTN_EINVAL


def test_a_page_that_does_not_exist_is_reported():
    cache, _, seqs, g = make([50], 16, 2, 64, torch.float16, 40)
    for bad in (4000, -1):
        cache.table[seqs[0], 1] = bad
        attn.tree_fwd(torch.randn(1, 4, 64, generator=g).half().cuda(), cache, seqs, [0, 1])
        assert attn.device_status() == _abi.ATTN_EINVAL


def test_two_streams_and_a_graph():
    """Reads of one cache on two streams at once, and a captured call that follows the lengths."""
    cache, model, seqs, g = make([3000, 2500], 64, 2, 128, torch.bfloat16, 41)
    qs = [torch.randn(2, 8, 128, generator=g).bfloat16().cuda() for _ in range(2)]
    want = [attn.tree_fwd(q, cache, seqs, [0, 1, 2]) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    calls = [attn.TreeCall(q, cache, seqs, [0, 1, 2]) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c in zip(streams, calls):
            c.run(s)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c.o, w[0]) and torch.equal(c.lse, w[1])
    graph = torch.cuda.CUDAGraph()
    calls[0].run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls[0].run()
    for cut in (0, 700, 2499):
        cache.lens[seqs[0]], cache.lens[seqs[1]] = 3000 - cut, 2500 - cut
        model.lens[seqs] = [3000 - cut, 2500 - cut]
        graph.replay()
        for i, s in enumerate(seqs):
            k, v = model.rows(s, 0)
            want = attention(qs[0][i:i + 1].cpu(), k, v, seen_tree(len(k), 1), 128 ** -0.5)
            assert_output(calls[0].o[i:i + 1], calls[0].lse[:, i:i + 1], want, torch.bfloat16, f"cut {cut}")


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 64)])
def test_serving(dtype, d):
    """Prompts through the forward into the cache, a tree of drafts, the accepted path
    kept, a fork, decoding, compaction: as attention over the whole sequences."""
    hq, hkv, page = 6, 2, 16
    g = torch.Generator().manual_seed(42)
    rows = lambda n, h: torch.randn(n, h, d, generator=g).to(dtype)  # noqa: E731
    cache = attn.Cache.empty(1, 40, page, hkv, d, max_seqs=5, max_pages=12, dtype=dtype)
    lens = [37, 80]
    ks, vs = [rows(n, hkv) for n in lens], [rows(n, hkv) for n in lens]
    q, cu = rows(sum(lens), hq), [0, 37, 117]
    o, lse = attn.fwd(q.cuda(), torch.cat(ks).cuda(), torch.cat(vs).cuda(), causal=True, cu_seqlens_q=cu)
    cache.extend([3, 1], lens)
    cache.write([3, 1], cu, torch.cat(ks).cuda(), torch.cat(vs).cuda())
    # the whole prompt as one chunk over the cache is the same attention
    o2, lse2 = attn.tree_fwd(q.cuda(), cache, [3, 1], cu)
    for i in range(2):
        m = slice(cu[i], cu[i + 1])
        want = attention(q[m], ks[i], vs[i], seen_tree(lens[i], lens[i]), d ** -0.5)
        assert_output(o[m], lse[:, m], want, dtype, "prompt")
        assert_output(o2[m], lse2[:, m], want, dtype, "prompt over the cache")
    # drafts 0 - 1 - 3, 0 - 2 - 4; the path 0, 2, 4 is accepted by the first, 0 by the second
    bits = np.array([0b00001, 0b00011, 0b00101, 0b01011, 0b10101], np.uint64)
    mask = np.tile(bits, 2)[:, None]
    dk, dv, dq = [rows(5, hkv) for _ in range(2)], [rows(5, hkv) for _ in range(2)], rows(10, hq)
    cache.extend([3, 1], [5, 5])
    cache.write([3, 1], [0, 5, 10], torch.cat(dk).cuda(), torch.cat(dv).cuda())
    o, lse = attn.tree_fwd(dq.cuda(), cache, [3, 1], [0, 5, 10], mask=torch.from_numpy(mask.view(np.int64)).cuda())
    for i in range(2):
        m = slice(5 * i, 5 * i + 5)
        k, v = torch.cat([ks[i], dk[i]]), torch.cat([vs[i], dv[i]])
        assert_output(o[m], lse[:, m], attention(dq[m], k, v, seen_tree(lens[i] + 5, 5, mask[m]), d ** -0.5), dtype, "tree")
    cache.keep([3, 1], [5, 5], torch.tensor([[0, 2, 4], [0, 0, 0]]), [3, 1])
    ks, vs = ([torch.cat([x[0], y[0][[0, 2, 4]]]), torch.cat([x[1], y[1][[0]]])] for x, y in ((ks, dk), (vs, dv)))
    cache.fork([3], [0])
    cache.free([1])
    cache.compact()
    for s in (3, 0):  # the two continue apart
        k1, v1, q1 = rows(1, hkv), rows(1, hkv), rows(1, hq)
        cache.extend([s], [1])
        cache.write([s], [0, 1], k1.cuda(), v1.cuda())
        o, lse = attn.tree_fwd(q1.cuda(), cache, [s], [0, 1])
        want = attention(q1, torch.cat([ks[0], k1]), torch.cat([vs[0], v1]), np.ones((1, 41), bool), d ** -0.5)
        assert_output(o, lse, want, dtype, f"decode {s}")
    assert attn.device_status() == 0


def test_workspaces_that_are_refused():
    cache, _, seqs, g = make([50], 16, 2, 64, torch.float16, 47)
    q = torch.randn(1, 4, 64, generator=g).half().cuda()
    need = attn.TreeCall(q, cache, seqs, [0, 1]).workspace.numel()
    with pytest.raises(ValueError, match="workspace"):
        attn.TreeCall(q, cache, seqs, [0, 1], workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        attn.TreeCall(q, cache, seqs, [0, 1], workspace=torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])
    for ws in (torch.empty(need - 256, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 256, dtype=torch.uint8, device="cuda")[16:]):  # too small; not 256-byte aligned
        with pytest.raises(attn.AttnError):
            attn.TreeCall(q, cache, seqs, [0, 1], workspace=ws).run()
