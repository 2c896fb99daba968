"""Accumulated attention weights of cached tokens against f64."""
import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import seen_tree
from online_softmax_attention_gb300 import _abi
from test_gpu_tree import make
from window_model import weigh, windowed

pytestmark = pytest.mark.gpu


def check(cache, model, seqs, news, q, window=None, sinks=0, fresh=None, layer=0, scale=None, seed=0, what=""):
    """Per token, all terms are positive: |w - ref| <= 2^-12 of the new ones' sum (the scores'
    f32 error, below 1e-4, and 2^x to 2^-21, as in the attention's own bound) and the f32
    additions', 2^-16 of everything (fewer than 2^8 roundings of half a step, 2^-24, in a row)."""
    cu = [0] + [int(x) for x in np.cumsum(news)]
    dev = q.cuda()
    lse = attn.tree_fwd(dev, cache, seqs, cu, layer=layer, window=window, sinks=sinks, scale=scale)[1]
    w = torch.rand(cache.new_weights().shape, generator=torch.Generator().manual_seed(seed)).cuda()
    w[..., -1] = float("nan")  # behind every sequence
    before = w.cpu().double().numpy()
    cache.weigh(seqs, cu, dev, lse, w, layer=layer, window=window, sinks=sinks, fresh=fresh, scale=scale)
    assert attn.device_status() == 0
    got, want, off = w.cpu().double().numpy(), before.copy(), np.zeros_like(before)
    for i, s in enumerate(seqs):
        rows = slice(cu[i], cu[i + 1])
        k, _ = model.rows(s, layer)
        n, new = len(k), news[i] if fresh is None else fresh[i]
        seen = windowed(seen_tree(n, news[i]), window, sinks)
        mass = weigh(q[rows], k, lse[:, rows].cpu(), seen, q.shape[2] ** -0.5 if scale is None else scale)
        want[layer, s, n - new:n] = 0
        want[layer, s, :n] += mass
        off[layer, s, :n] = mass * 2.0 ** -12 + want[layer, s, :n] * 2.0 ** -16
    touched = off > 0
    assert np.array_equal(got[~touched], want[~touched], equal_nan=True), f"{what}: weights that nothing is added to"
    assert (np.abs(got - want) <= off)[touched].all(), f"{what}: {np.max((np.abs(got - want) / off)[touched]):.2f} of the bound"
    return w


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,page,heads,group", [([1], 16, 1, 1), ([700], 16, 2, 4), ([5, 1, 64, 333, 31, 32, 33], 8, 3, 3),
                                                   ([2000, 3], 128, 1, 8), ([40] * 20, 1, 5, 2), ([129], 1024, 8, 4),
                                                   ([500], 64, 9, 1)])
def test_decoding(lens, page, heads, group, d, dtype):
    cache, model, seqs, g = make(lens, page, heads, d, dtype, 81)
    q = torch.randn(len(lens), heads * group, d, generator=g).to(dtype)
    check(cache, model, seqs, [1] * len(lens), q, what=f"{lens}")


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64), (torch.float32, 64)])
@pytest.mark.parametrize("lens,news,page,heads,group", [
    ([7], [7], 16, 1, 2), ([300, 41, 9], [5, 41, 1], 32, 2, 4), ([64, 65], [64, 63], 64, 1, 3), ([500, 130], [130, 65], 16, 2, 1),
    ([90, 1000, 4], [0, 17, 2], 8, 1, 8), ([257], [33], 128, 4, 5), ([300], [300], 16, 8, 4)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (20, 3), (1, 0), (140, 40)])
def test_chunks_and_windows(lens, news, page, heads, group, d, dtype, window, sinks):
    cache, model, seqs, g = make(lens, page, heads, d, dtype, 82)
    q = torch.randn(sum(news), heads * group, d, generator=g).to(dtype)
    check(cache, model, seqs, news, q, window, sinks, what=f"{lens} {news}")
    check(cache, model, seqs, news, q, window, sinks, fresh=lens, seed=1, what=f"{lens} {news} fresh")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layers_scales_and_layouts(dtype):
    cache, model, seqs, g = make([210, 77], 32, 2, 128, dtype, 83, layers=3, layout="hnd")
    q = torch.randn(9, 8, 128, generator=g).to(dtype)
    for layer, scale in ((2, 0.3), (0, -0.2), (1, 0.0)):
        check(cache, model, seqs, [4, 5], q, layer=layer, scale=scale, fresh=[0, 6])


def test_long_contexts_and_many_sequences():
    for lens in ([20000], [64] * 300, [6000, 1, 3000]):
        cache, model, seqs, g = make(lens, 64, 2, 64, torch.float16, 84)
        q = torch.randn(len(lens), 8, 64, generator=g).half()
        first = check(cache, model, seqs, [1] * len(lens), q, what=f"{lens[:3]}")
        again = check(cache, model, seqs, [1] * len(lens), q)
        assert torch.equal(first[..., :-1], again[..., :-1])


def test_rows_that_saw_nothing_add_nothing():
    cache, model, seqs, g = make([40], 16, 2, 64, torch.bfloat16, 85)
    q = torch.randn(3, 8, 64, generator=g).bfloat16().cuda()
    lse = attn.tree_fwd(q, cache, seqs, [0, 3])[1]
    lse[:, 1] = -torch.inf
    w, one = cache.new_weights(), cache.new_weights()
    cache.weigh(seqs, [0, 3], q, lse, w)
    only = lse.clone()
    only[:, [0, 2]] = -torch.inf
    cache.weigh(seqs, [0, 3], q, only, one)
    assert torch.isfinite(w).all() and w.sum() > 10 and (one == 0).all()


def test_entries_that_do_not_fit_are_left():
    cache, model, seqs, g = make([50, 60], 16, 2, 64, torch.float16, 86)
    q = torch.randn(8, 4, 64, generator=g).half().cuda()
    lse = attn.tree_fwd(q, cache, seqs, [0, 3, 8])[1]
    good = cache.new_weights()
    cache.weigh(seqs, [0, 3, 8], q, lse, good)
    assert attn.device_status() == 0
    a, b = seqs
    for bad_seqs, cu, fresh, done in (([a, 99], [0, 3, 8], None, [a]), ([-1, b], [0, 3, 8], None, [b]), ([a, b], [0, 3, 9], None, [a]),
                                      ([a, b], [3, 0, 8], None, [b]), ([a, b], [0, 3, 8], [51, 5], [b]), ([a, b], [0, 3, 8], [3, -1], [a]),
                                      ([a, a], [0, 3, 8], None, []), ([b, b], [0, 3, 8], None, []), ([b, 2 ** 31 - 1], [0, 3, 8], None, [])):
        w = cache.new_weights()
        cache.weigh(bad_seqs, cu, q, lse, w, fresh=fresh)
        assert attn.device_status() == _abi.ATTN_EINVAL, (bad_seqs, cu, fresh)
        for s in seqs:
            if s in done and cu[1] == 3:
                assert torch.equal(w[:, s], good[:, s]), (bad_seqs, cu, fresh)
            elif s in done:  # (its offsets 0 and 8 fit: all the rows are its own)
                assert (w[:, s, :60] > 0).all() and (w[:, s, 60:] == 0).all()
            elif not (bad_seqs[0] == b and s == b):
                assert (w[:, s] == 0).all(), (bad_seqs, cu, fresh)
    short = torch.zeros(1, cache.max_seqs, 55, device="cuda")  # too few columns for the second
    cache.weigh(seqs, [0, 3, 8], q, lse, short)
    assert attn.device_status() == _abi.ATTN_EINVAL
    assert torch.equal(short[:, a, :50], good[:, a, :50]) and (short[:, b] == 0).all()
    cache.table[a, 1] = -1
    cache.weigh([a], [0, 3], q[:3], lse[:, :3].contiguous(), cache.new_weights())
    assert attn.device_status() == _abi.ATTN_EINVAL


def test_arguments_that_are_refused():
    cache, model, seqs, g = make([50], 16, 2, 64, torch.float16, 87)
    q = torch.randn(1, 4, 64, generator=g).half().cuda()
    lse, w = torch.zeros(4, 1, device="cuda"), cache.new_weights()
    for kw in (dict(lse=lse.double()), dict(lse=lse.t()), dict(lse=lse.cpu()), dict(weights=w.double()), dict(weights=w[:, 1:]),
               dict(weights=w.cpu()), dict(weights=w[0]), dict(weights=w.expand(2, -1, -1)), dict(cu=[0]), dict(fresh=[1, 2]),
               dict(layer=1), dict(layer=-1), dict(window=0), dict(sinks=3), dict(q=q[..., :32])):
        a = dict(cu=[0, 1], q=q, lse=lse, weights=w, layer=0, fresh=None, window=None, sinks=0)
        a.update(kw)
        with pytest.raises(ValueError):
            cache.weigh(seqs, a["cu"], a["q"], a["lse"], a["weights"], layer=a["layer"], fresh=a["fresh"], window=a["window"],
                        sinks=a["sinks"])
    with pytest.raises(TypeError):
        cache.weigh(seqs, [0, 1], q.float(), lse, w)
    cache.weigh(seqs, [0, 0], q[:0], lse[:, :0].contiguous(), w)  # no rows: nothing to add
    assert (w == 0).all() and attn.device_status() == 0


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("lens,news,page,heads,group", [
    ([1500], [1500], 16, 2, 4), ([900, 3, 700, 128], [300, 3, 0, 128], 8, 1, 3), ([2000, 1300], [64, 200], 64, 8, 4),
    ([127, 128, 129], [127, 128, 129], 128, 3, 1), ([300] * 40, [20] * 40, 32, 2, 5), ([5000], [77], 1024, 1, 128),
    ([600, 600], [1, 599], 16, 4, 16)])
def test_many_rows(lens, news, page, heads, group, d, dtype):
    """Tensor-core units: tiles of rows that the group does not fill, new tokens over several key tiles,
    units cut between blocks, entries without new tokens beside others."""
    cache, model, seqs, g = make(lens, page, heads, d, dtype, 88)
    q = torch.randn(sum(news), heads * group, d, generator=g).to(dtype)
    first = check(cache, model, seqs, news, q, what=f"{lens}")
    again = check(cache, model, seqs, news, q)
    assert torch.equal(first[..., :-1], again[..., :-1])
    check(cache, model, seqs, news, q, fresh=lens, what=f"{lens} fresh")
    check(cache, model, seqs, news, q, scale=-0.1, what=f"{lens} scaled")


def test_other_rows_and_stale_slots_may_hold_anything():
    """Query rows of no entry, and cached slots behind the sequences, with NaN in them."""
    cache, model, seqs, g = make([300, 70], 16, 2, 64, torch.bfloat16, 89)
    q = torch.randn(150, 8, 64, generator=g).bfloat16().cuda()
    lse = attn.tree_fwd(q[:110], cache, seqs, [0, 50, 110])[1]
    w, want = cache.new_weights(), cache.new_weights()
    cache.weigh(seqs, [0, 50, 110], q[:110], lse, want)
    q[110:] = float("nan")
    more = torch.full((8, 150), float("nan"), device="cuda")
    more[:, :110] = lse
    cache.weigh(seqs, [0, 50, 110], q, more, w)
    assert torch.equal(w, want) and torch.isfinite(w).all() and attn.device_status() == 0


def test_workspaces_streams_and_graphs():
    cache, model, seqs, g = make([700, 300], 16, 2, 64, torch.bfloat16, 90)
    q = torch.randn(200, 8, 64, generator=g).bfloat16().cuda()
    lse = attn.tree_fwd(q, cache, seqs, [0, 120, 200])[1]
    want = cache.new_weights()
    ids, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (seqs, [0, 120, 200]))
    cache.weigh(ids, cu, q, lse, want)
    torch.cuda.synchronize()
    outs = [cache.new_weights() for _ in range(3)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, w in zip(side, outs):
        with torch.cuda.stream(s):
            for _ in range(5):
                w.zero_()
                cache.weigh(ids, cu, q, lse, w)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs[2].zero_()
        cache.weigh(ids, cu, q, lse, outs[2])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(w, want) for w in outs)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [11, 22, 28, 37, 48, 65, 100, 128])
def test_groups_that_leave_a_part_of_a_query_tile(group, d):
    """The rows of whole tokens are fewer than a tile's; calls before leave infinite scores behind."""
    cache, model, seqs, g = make([300, 129], 16, 1, d, torch.bfloat16, 91)
    big, _, ids, _ = make([700], 16, 1, d, torch.bfloat16, 92)
    big.k.fill_(2.0 ** 120)
    q = torch.full((600, 8, d), 2.0 ** 100).bfloat16().cuda()
    for _ in range(2):
        big.weigh(ids, [0, 600], q, torch.zeros(8, 600, device="cuda"), big.new_weights())
    q = torch.randn(50, group, d, generator=g).bfloat16()
    check(cache, model, seqs, [20, 30], q, what=f"{group}")


@pytest.mark.parametrize("dtype,t", [(torch.bfloat16, 1), (torch.float16, 30), (torch.float32, 4)])
def test_tokens_that_a_window_hides_may_hold_anything(dtype, t):
    cache, _, seqs, g = make([700, 300], 16, 2, 64, dtype, 93)
    q = torch.randn(2 * t, 8, 64, generator=g).to(dtype).cuda()
    kw = dict(window=90, sinks=3)
    lse = attn.tree_fwd(q, cache, seqs, [0, t, 2 * t], **kw)[1]
    w, want = cache.new_weights(), cache.new_weights()
    cache.weigh(seqs, [0, t, 2 * t], q, lse, want, **kw)
    for s, n in zip(seqs, (700, 300)):
        hidden = torch.arange(3, n - t + 1 - 90, device="cuda")
        cache.k[:, cache.table[s].long()[hidden // 16], hidden % 16] = float("nan")
    cache.weigh(seqs, [0, t, 2 * t], q, lse, w, **kw)
    assert torch.equal(w, want) and torch.isfinite(w).all() and attn.device_status() == 0


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("lens,news,page,heads,group", [
    ([700], [700], 16, 2, 4), ([900, 3, 700, 128], [300, 3, 0, 128], 8, 1, 3), ([2000, 1300], [64, 20], 64, 2, 4),
    ([300] * 40, [5] * 40, 32, 2, 5), ([5000], [7], 1024, 1, 128), ([1300, 600], [1299, 1], 16, 1, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 3), (256, 0), (300, 300), (700, 2 ** 31 - 1), (900, 40)])
def test_many_rows_over_windows(lens, news, page, heads, group, d, dtype, window, sinks):
    """Units that a window hides, wholly or from the last rows; the sinks' ones; weights that start anew there."""
    cache, model, seqs, g = make(lens, page, heads, d, dtype, 94)
    q = torch.randn(sum(news), heads * group, d, generator=g).to(dtype)
    first = check(cache, model, seqs, news, q, window, sinks, what=f"{lens}")
    again = check(cache, model, seqs, news, q, window, sinks)
    assert torch.equal(first[..., :-1], again[..., :-1])
    check(cache, model, seqs, news, q, window, sinks, fresh=lens, what=f"{lens} fresh")
    check(cache, model, seqs, news, q, window, sinks, fresh=[(n + 1) // 2 for n in lens], what=f"{lens} half fresh")


@pytest.mark.parametrize("dtype,t", [(torch.bfloat16, 1), (torch.float16, 40), (torch.float32, 9)])
def test_pages_that_a_window_hides_may_be_gone(dtype, t):
    cache, _, seqs, g = make([3000, 1700], 64, 2, 64, dtype, 95)
    q = torch.randn(2 * t, 8, 64, generator=g).to(dtype).cuda()
    kw = dict(window=500, sinks=70)
    lse = attn.tree_fwd(q, cache, seqs, [0, t, 2 * t], **kw)[1]
    w, want = cache.new_weights(), cache.new_weights()
    cache.weigh(seqs, [0, t, 2 * t], q, lse, want, **kw)
    for s, n in zip(seqs, (3000, 1700)):
        cache.table[s, 2:(n - t + 1 - 500) // 64] = -1
    cache.weigh(seqs, [0, t, 2 * t], q, lse, w, **kw)
    assert torch.equal(w, want) and attn.device_status() == 0
    cache.weigh([seqs[0]] * 2, [0, t, 2 * t], q, lse, w, fresh=[3000, 3000], **kw)  # twice: nothing is touched
    assert torch.equal(w, want) and attn.device_status() == _abi.ATTN_EINVAL
