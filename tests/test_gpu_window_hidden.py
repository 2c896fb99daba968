"""Windowed attention over the cache where tokens that no new one sees hold anything: what is hidden comes
from the masks themselves (chains, trees, random bits), for every kernel, type and page size."""
import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import assert_output, attention, seen_tree
from test_gpu_tree import make, random_mask
from window_model import windowed

pytestmark = pytest.mark.gpu


def masks(kind, news, words, r):
    """uint64 (rows, words): a chain or a random tree, whose tokens see themselves; random bits; or None."""
    if kind == "causal":
        return None
    if kind == "bits":
        return random_mask(news, words, r)
    out = np.zeros((sum(news), words), np.uint64)
    at = 0
    for t in news:
        for u in range(t):
            if u:
                out[at + u] = out[at + (u - 1 if kind == "chain" else r.integers(0, u))]
            out[at + u, u >> 6] |= np.uint64(1 << (u & 63))
        at += t
    return out


def setup(lens, news, page, heads, group, d, dtype, kind, window, sinks, seed):
    """Cache, model, call arguments and, per sequence, which tokens each new one sees."""
    cache, model, seqs, g = make(lens, page, heads, d, dtype, seed)
    q = torch.randn(sum(news), heads * group, d, generator=g).to(dtype)
    cu = [0] + [int(x) for x in np.cumsum(news)]
    mask = masks(kind, news, -(-max(news) // 64), np.random.default_rng(seed))
    rows = [None if mask is None else mask[cu[i]:cu[i + 1]] for i in range(len(lens))]
    seen = [windowed(seen_tree(n, t, m), window, sinks) for n, t, m in zip(lens, news, rows)]
    call = dict(mask=None if mask is None else torch.from_numpy(mask.view(np.int64)).cuda(), window=window, sinks=sinks)
    return cache, model, seqs, q, cu, call, seen


def check(o, lse, model, seqs, q, cu, seen, dtype, what):
    for i, s in enumerate(seqs):
        rows = slice(cu[i], cu[i + 1])
        k, v = model.rows(s, 0)
        assert_output(o[rows], lse[:, rows], attention(q[rows], k, v, seen[i], q.shape[2] ** -0.5), dtype, f"{what} entry {i}")


# clusters of 16-row units, stretches of them (long windows, pages of 4), 256-row units whole and cut, f32
SHAPES = [([700, 95], [1, 1], 16, 2, 4), ([700, 400], [4, 2], 32, 2, 2), ([9400], [5], 64, 1, 2), ([900, 300], [9, 2], 4, 2, 4),
          ([900, 600], [40, 20], 64, 2, 4), ([700], [70], 8, 1, 2), ([2500, 300], [200, 7], 16, 1, 3), ([1500], [130], 1024, 2, 1)]
WINDOWS = [(1, 0), (3, 2), (50, 0), (60, 200), (200, 17)]


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 64), (torch.float32, 128)])
@pytest.mark.parametrize("lens,news,page,heads,group", SHAPES)
@pytest.mark.parametrize("kind", ["causal", "chain", "tree", "bits"])
def test_tokens_that_no_row_sees(lens, news, page, heads, group, kind, dtype, d):
    for window, sinks in WINDOWS + ([(9000, 4)] if lens[0] > 9000 else []):
        cache, model, seqs, q, cu, call, seen = setup(lens, news, page, heads, group, d, dtype, kind, window, sinks, 110)
        want = attn.tree_fwd(q.cuda(), cache, seqs, cu, **call)
        check(*want, model, seqs, q, cu, seen, dtype, f"{kind} {window}+{sinks}")
        for s, rows in zip(seqs, seen):
            hidden = torch.from_numpy(np.flatnonzero(~rows.any(0))).cuda()
            at = cache.table[s].long()[hidden // page], hidden % page
            cache.k[:, at[0], at[1]] = float("nan")
            cache.v[:, at[0], at[1]] = torch.inf
            cache.v[:, at[0][::2], at[1][::2]] = float("nan")
        got = attn.tree_fwd(q.cuda(), cache, seqs, cu, **call)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (kind, window, sinks)
    assert attn.device_status() == 0


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)])
@pytest.mark.parametrize("lens,news,page,heads,group,window,sinks", [
    # the first token that a row of a chain sees is one of a multiple of 256, or the one behind it
    ([2000], [4], 16, 2, 2, 205, 0), ([2000], [4], 16, 2, 2, 204, 3), ([2000, 1400], [4, 1], 256, 2, 2, 205, 4), ([2000], [40], 128, 2, 4, 169, 4),
    ([2000], [40], 8, 2, 4, 168, 0), ([3000, 900], [400, 300], 64, 1, 2, 41, 300), ([9800], [5], 64, 1, 1, 9028, 300),
    ([1500], [20], 4, 1, 4, 201, 2), ([4500], [30], 1024, 1, 4, 375, 2)])
@pytest.mark.parametrize("kind", ["causal", "chain", "tree", "bits"])
def test_pages_that_no_row_sees_may_be_gone(lens, news, page, heads, group, window, sinks, kind, dtype, d):
    """Table entries of pages in runs of 256 tokens before the new ones that hold none which is seen."""
    cache, model, seqs, q, cu, call, seen = setup(lens, news, page, heads, group, d, dtype, kind, window, sinks, 111)
    gone = 0
    for s, rows, n, t in zip(seqs, seen, lens, news):
        live = rows.any(0)
        live[n - t:] = True
        table = cache.table[s].cpu()
        for i in range(-(-n // page)):
            a, b = i * page // 256 * 256, -(-(i + 1) * page // 256) * 256
            if not live[a:b].any():
                table[i] = -1
                gone += 1
        cache.table[s] = table.cuda()
    assert gone > 0
    o, lse = attn.tree_fwd(q.cuda(), cache, seqs, cu, **call)
    assert attn.device_status() == 0
    check(o, lse, model, seqs, q, cu, seen, dtype, f"{kind} {window}+{sinks}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,page", [(4, 16), (40, 16), (40, 256)])
def test_pages_that_a_row_sees_are_missed(t, page, dtype):
    """The page of the first token that a row of a chain sees."""
    cache, _, seqs, q, cu, call, seen = setup([2000], [t], page, 2, 2, 64, dtype, "chain", 300, 2, 112)
    first = int(np.flatnonzero(seen[0].any(0) & (np.arange(2000) >= 2))[0])
    cache.table[seqs[0], first // page] = -1
    attn.tree_fwd(q.cuda(), cache, seqs, cu, **call)
    assert attn.device_status() == attn._abi.ATTN_EINVAL


def test_trees_in_a_graph_and_on_streams_at_once():
    """Prepared calls of both kernels over one cache whose hidden tokens are NaN, replayed for other lengths and masks."""
    lens, streams = [3000, 1700, 900], []
    calls = []
    for t, window in ((4, 600), (40, 600), (70, 30)):
        cache, _, seqs, q, cu, call, seen = setup(lens, [t] * 3, 16, 2, 4, 128, torch.bfloat16, "tree", window, 4, 113)
        for s, rows in zip(seqs, seen):
            hidden = torch.from_numpy(np.flatnonzero(~rows.any(0))).cuda()
            cache.v[:, cache.table[s].long()[hidden // 16], hidden % 16] = float("nan")
        c = attn.TreeCall(q.cuda(), cache, seqs, cu, **call)
        c.run()
        torch.cuda.synchronize()
        assert torch.isfinite(c.o).all()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
        calls.append((c, graph, c.o.clone(), c.lse.clone(), cache, seqs, q, cu, call))
        streams.append(torch.cuda.Stream())
    for c, *_ in calls:
        c.o.fill_(9)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (c, graph, *_) in zip(streams, calls):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for c, graph, o, lse, cache, seqs, q, cu, call in calls:
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
        # every draft now sees the ones before it, of shorter sequences
        call["mask"].copy_(torch.from_numpy(masks("chain", [int(n) for n in np.diff(cu)], call["mask"].shape[1], None).view(np.int64)))
        cache.lens[seqs[0]], cache.v[...] = 500, torch.randn(cache.v.shape, device="cuda").bfloat16()
        graph.replay()
        want = attn.tree_fwd(q.cuda(), cache, seqs, cu, **call)
        assert torch.equal(c.o, want[0]) and torch.equal(c.lse, want[1])
    assert attn.device_status() == 0
