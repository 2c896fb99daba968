"""Eviction from the cache by accumulated attention weight, against a model in plain Python."""
import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import assert_output, attention, seen_tree
from online_softmax_attention_gb300 import _abi
from test_gpu_tree import make
from window_model import evict, kept, weigh

pytestmark = pytest.mark.gpu


def state(cache, w):
    return [t.cpu() for t in (cache.k, cache.v, cache.table, cache.lens, cache.refs, w)]


def check(cache, model, seqs, budgets, w, sinks=0, recent=0, what=""):
    after = w.cpu().numpy().copy()
    evict(model, seqs, budgets, after, sinks, recent)
    cache.evict(seqs, budgets, w, sinks=sinks, recent=recent)
    assert attn.device_status() == 0
    for x, y, name in ((cache.lens, model.lens, "lengths"), (cache.refs, model.refs, "counts"), (cache.table, model.table, "tables"),
                       (cache.k, model.k, "k"), (cache.v, model.v, "v"), (w, after, "weights")):
        assert np.array_equal(x.cpu().double().numpy(), np.asarray(y, dtype=np.float64), equal_nan=True), f"{what}: {name}"


def weights(cache, seed, kind="normal", layers=None):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(cache.new_weights(layers).shape, generator=g)
    if kind == "heavy":
        w = (3 * w).exp()
    elif kind == "ties":
        w = w.round()
    elif kind == "same":
        w = torch.full_like(w, 0.25)
    elif kind == "odd":  # zeros of both signs, infinities, NaN, the smallest and largest numbers
        odd = torch.tensor([0.0, -0.0, torch.inf, -torch.inf, torch.nan, -torch.nan, 1e-45, -1e-45, 3e38, -3e38, 1.0])
        w = odd[torch.randint(0, 11, w.shape, generator=g)]
    return w.cuda()


@pytest.mark.parametrize("kind", ["normal", "heavy", "ties", "same", "odd"])
@pytest.mark.parametrize("lens,budgets,page,sinks,recent", [
    ([1], [0], 16, 0, 0), ([1], [1], 16, 1, 0), ([40], [39], 16, 4, 8), ([700, 33, 100], [100, 33, 99], 16, 4, 20),
    ([257, 5, 129], [64, 2, 128], 64, 0, 0), ([300, 300], [10, 290], 8, 3, 7), ([2100], [600], 1, 1, 64), ([1300], [1025], 1024, 4, 0),
    ([90, 91], [30, 31], 32, 10, 20)])
def test_sequences_cut_to_a_budget(lens, budgets, page, sinks, recent, kind):
    cache, model, seqs, _ = make(lens, page, 2, 64, torch.float16, 91, layers=2)
    one = kind == "odd"  # (sums of infinities: one layer)
    check(cache, model, seqs, budgets, weights(cache, 92, kind, 1 if one else 2), sinks, recent, f"{lens} {budgets}")


@pytest.mark.parametrize("dtype,d,heads,layers,layout", [(torch.bfloat16, 128, 8, 3, "nhd"), (torch.float32, 128, 3, 1, "hnd"),
                                                         (torch.float16, 64, 5, 2, "hnd"), (torch.float32, 64, 1, 4, "nhd")])
def test_layouts_and_layers(dtype, d, heads, layers, layout):
    lens = [500, 64, 333]
    cache, model, seqs, _ = make(lens, 16, heads, d, dtype, 93, layers=layers, layout=layout)
    check(cache, model, seqs, [200, 30, 332], weights(cache, 94, layers=layers), 4, 16)
    check(cache, model, seqs, [100, 30, 20], weights(cache, 95, layers=layers + 1), 0, 0, "again, more layers of weights")


def test_more_tokens_than_shared_memory_numbers():
    cache, model, seqs, _ = make([45000, 41000], 256, 1, 64, torch.float16, 96)
    check(cache, model, seqs, [2000, 40900], weights(cache, 97, "ties"), 4, 30)


def test_weights_of_other_strides():
    cache, model, seqs, _ = make([200, 100], 16, 2, 64, torch.float16, 98, layers=2)
    big = torch.randn(3, cache.max_seqs, 230, generator=torch.Generator().manual_seed(99)).cuda()
    inside = big[::2, :, 5:225]
    check(cache, model, seqs, [50, 60], inside, 2, 3)
    assert inside.shape == (2, cache.max_seqs, 220)


def test_shared_pages():
    """A prefix that both hold stays; rows that would move into it are refused."""
    cache, model, seqs, g = make([96, 5], 16, 2, 64, torch.float16, 100, spare=20)
    a, child = seqs[0], next(s for s in range(4) if s not in seqs)
    cache.fork([a], [child])
    model.fork([a], [child])
    w = weights(cache, 101)
    w[:, [a, child], :64] = 100.0  # the first four pages' tokens are the heaviest
    check(cache, model, [a], [64], w)  # nothing moves: the pages behind are released
    cache.extend([a], [30])
    model.extend([a], [30])
    before = state(cache, w)
    w[:, a, 0] = -5.0  # now a shared page's row would go
    before[5] = w.cpu()
    cache.evict([a], [70], w)
    assert attn.device_status() == _abi.ATTN_EINVAL
    assert all(torch.equal(x, y) for x, y in zip(before[2:5], state(cache, w)[2:5])) and torch.equal(before[5], w.cpu())


def test_lists_that_are_refused_change_nothing():
    cache, model, seqs, _ = make([200, 100, 40], 16, 2, 64, torch.float16, 102, junk=0.0)
    w = weights(cache, 103)
    before = state(cache, w)
    a, b, c = seqs

    def refused(ids, budgets, **kw):
        cache.evict(ids, budgets, kw.pop("w", w), **kw)
        assert attn.device_status() == _abi.ATTN_EINVAL, (ids, budgets, kw)
        assert all(torch.equal(x, y) for x, y in zip(before, state(cache, w))), (ids, budgets, kw)

    refused([a, 77], [10, 10])
    refused([a, -1], [10, 10])
    refused([a, b, a], [10, 10, 10])
    refused([a, b], [10, -1])
    refused([a, b], [50, 20], sinks=10, recent=11)
    refused([a, b], [50, 20], sinks=2 ** 31 - 1, recent=2 ** 31 - 1)
    refused([c, a], [10, 10], w=w[..., :150])  # too few columns for the second
    for bad in (-1, cache.refs.numel()):
        cache.table[a, 11] = bad
        before = state(cache, w)
        refused([b, a], [10, 10])
    # what is shorter than its budget is not looked at any further
    cache.evict([c], [40], w, sinks=30, recent=30)
    assert attn.device_status() == 0 and all(torch.equal(x, y) for x, y in zip(before, state(cache, w)))
    cache.evict([], [], w)
    assert attn.device_status() == 0


def test_arguments_that_are_refused():
    cache, _, seqs, _ = make([50], 16, 2, 64, torch.float16, 104)
    w = cache.new_weights()
    for args, kw in ((([0], [1, 2], w), {}), (([0], [1], w.cpu()), {}), (([0], [1], w.half()), {}), (([0], [1], w), dict(sinks=-1)),
                     (([0], [1], w), dict(recent=-1)), (([0], [1], w), dict(recent=1.5)), (([0], [1], w[:, :, ::2]), {}),
                     (([0.5], [1], w), {}), (([0], [2 ** 31], w), {})):
        with pytest.raises(ValueError):
            cache.evict(*args, **kw)


def test_a_captured_loop():
    """Decoding at a budget, captured: room, rows, attention, weights, eviction; as the same steps called."""
    lens, budget = [150, 90], 80

    def build():
        cache, model, seqs, g = make(lens, 16, 2, 64, torch.float16, 105, spare=12)
        return cache, seqs, weights(cache, 106, "heavy"), [torch.randn(2, h, 64, generator=g).half().cuda() for h in (8, 2, 2)]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def step(cache, seqs, w, rows, cu, ones, budgets):
        q, k, v = rows
        cache.extend(seqs, ones)
        cache.write(seqs, cu, k, v)
        o, lse = attn.tree_fwd(q, cache, seqs, cu)
        cache.weigh(seqs, cu, q, lse, w)
        cache.evict(seqs, budgets, w, sinks=2, recent=10)
        return o, lse

    lists = [ints([0, 1, 2]), ints([1, 1]), ints([budget, budget])]
    cache, seqs, w, rows = build()
    called = [step(cache, ints(seqs), w, rows, *lists) for _ in range(4)]
    again, seqs, w2, rows = build()
    ids = ints(seqs)
    step(again, ids, w2, rows, *lists)  # (warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(again, ids, w2, rows, *lists)
    for i in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, called[i][0]) and torch.equal(lse, called[i][1])
    assert attn.device_status() == 0
    live = slice(0, budget)
    assert torch.equal(cache.lens, again.lens) and torch.equal(w[:, seqs, live], w2[:, seqs, live])
    assert (cache.lens[seqs] == budget).all()


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_serving_at_a_budget(dtype, d):
    """A prompt, its tokens' weights, eviction, and decoding over what was kept: against attention over the kept rows."""
    n, budget, sinks, recent = 120, 40, 2, 12
    g = torch.Generator().manual_seed(107)
    q, k, v = (torch.randn(n + 1, h, d, generator=g).to(dtype) for h in (6, 2, 2))
    cache = attn.Cache.empty(1, 12, 16, 2, d, max_seqs=3, max_pages=10, dtype=dtype)
    w = cache.new_weights()
    cache.extend([2], [n])
    cache.write([2], [0, n], k[:n].cuda(), v[:n].cuda())
    o, lse = attn.tree_fwd(q[:n].cuda(), cache, [2], [0, n])
    cache.weigh([2], [0, n], q[:n].cuda(), lse, w)
    mass = weigh(q[:n], k[:n], lse.cpu(), seen_tree(n, n), d ** -0.5)
    assert np.abs(w[0, 2, :n].cpu().double().numpy() - mass).max() <= 2.0 ** -11 * mass.max()
    keep = kept(w[:, 2].cpu().numpy(), n, budget, sinks, recent)
    cache.evict([2], [budget], w, sinks=sinks, recent=recent)
    assert int(cache.lens[2]) == budget and int((cache.refs > 0).sum()) == 3
    cache.extend([2], [1])
    cache.write([2], [0, 1], k[n:].cuda(), v[n:].cuda())
    o, lse = attn.tree_fwd(q[n:].cuda(), cache, [2], [0, 1])
    rows = [*keep, n]
    assert_output(o, lse, attention(q[n:], k[rows], v[rows], np.ones((1, budget + 1), bool), d ** -0.5), dtype)
    assert attn.device_status() == 0
