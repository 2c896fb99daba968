"""The paged cache's operations against a model of them, one entry at a time."""
import numpy as np
import pytest
import torch

import online_softmax_attention_gb300 as attn
from cache_model import Model
from online_softmax_attention_gb300 import _abi

pytestmark = pytest.mark.gpu


def make(n_pages=97, page=16, layers=2, heads=3, d=64, seqs=12, per_seq=20, dtype=torch.float16, seed=1, layout="nhd"):
    """A cache of random values (whole numbers, exact in every type) and its model."""
    g = torch.Generator().manual_seed(seed)
    def pool():
        t = torch.randint(-128, 128, (layers, n_pages, page, heads, d), generator=g).to(dtype).cuda()
        if layout == "hnd":  # pages as (heads, page, D)
            t = t.permute(0, 1, 3, 2, 4).contiguous().permute(0, 1, 3, 2, 4)
        return t
    table = torch.full((seqs, per_seq), -7, dtype=torch.int32, device="cuda")
    c = attn.Cache(pool(), pool(), table, torch.zeros(seqs, dtype=torch.int32, device="cuda"),
                   torch.zeros(n_pages, dtype=torch.int32, device="cuda"))
    m = Model(*(t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()
                for t in (c.k, c.v, c.table, c.lens, c.refs)))
    return c, m


def same(c, m):
    for n in ("table", "lens", "refs", "k", "v"):
        np.testing.assert_array_equal(getattr(c, n).float().cpu().numpy(), getattr(m, n).astype(np.float32), err_msg=n)


def fill(c, m, lens, seed=2):
    """Sequences 0, 1, ... of the given lengths, their rows written in every layer."""
    seqs = list(range(len(lens)))
    c.extend(seqs, lens)
    m.extend(seqs, lens)
    put(c, m, seqs, lens, seed)


def put(c, m, seqs, counts, seed):
    g = torch.Generator().manual_seed(seed)
    cu = [0] + [int(x) for x in np.cumsum(counts)]
    L, _, _, H, D = c.k.shape
    for layer in range(L):
        k, v = (torch.randint(-128, 128, (cu[-1], H, D), generator=g).to(c.k.dtype) for _ in range(2))
        c.write(seqs, cu, k.cuda(), v.cuda(), layer=layer)
        m.write(layer, seqs, cu, k.float().numpy(), v.float().numpy())


@pytest.mark.parametrize("page,dtype,d,layout", [(16, torch.float16, 64, "nhd"), (1, torch.bfloat16, 64, "nhd"),
                                                 (64, torch.bfloat16, 128, "hnd"), (8, torch.float32, 128, "nhd"),
                                                 (32, torch.float32, 64, "hnd"), (1024, torch.float16, 64, "nhd")])
def test_a_life_of_the_cache(page, dtype, d, layout):
    """Prompts, forks, drafts kept and dropped, frees, compaction, new prompts."""
    c, m = make(n_pages=260 if page < 8 else 60, page=page, dtype=dtype, d=d, layout=layout, per_seq=220 if page < 8 else 30,
                layers=2 if page < 1024 else 1, seqs=14)
    lens = [5, 1, page, 2 * page - 1, 33]
    fill(c, m, lens)
    same(c, m)
    c.fork([0, 3, 3, 2], [9, 6, 7, 8])
    m.fork([0, 3, 3, 2], [9, 6, 7, 8])
    same(c, m)
    seqs, counts = [6, 3, 0, 9, 2], [3, 4, 5, 0, 1]
    c.extend(seqs, counts)
    m.extend(seqs, counts)
    put(c, m, seqs, counts, 3)
    same(c, m)
    keep = [[1, 2, 0, 0], [0, 0, 0, 0], [0, 2, 4, 0], [0, 0, 0, 0], [0, 0, 0, 0]]
    n_keep = [2, 0, 3, 0, 1]
    c.keep(seqs, counts, torch.tensor(keep), n_keep)
    m.keep(seqs, counts, keep, n_keep)
    same(c, m)
    c.free([3, 1, 6])
    m.free([3, 1, 6])
    same(c, m)
    remap = torch.empty_like(c.refs)
    c.compact(remap=remap)
    np.testing.assert_array_equal(remap.cpu().numpy(), m.compact())
    same(c, m)
    c.compact()  # nothing left to move
    m.compact()
    same(c, m)
    c.extend([1, 3], [2 * page + 1, 7])
    m.extend([1, 3], [2 * page + 1, 7])
    put(c, m, [1, 3], [2 * page + 1, 7], 4)
    same(c, m)
    assert attn.device_status() == 0


def test_many_pages_and_entries():
    """More pages than one pass of the scan, more entries than one block has threads."""
    c, m = make(n_pages=70001, page=1, layers=1, heads=1, seqs=3000, per_seq=64, seed=5)
    r = np.random.default_rng(6)
    seqs = r.permutation(3000)[:2100]
    counts = r.integers(0, 25, 2100)
    c.extend(seqs, counts)
    m.extend(seqs, counts)
    same(c, m)
    gone = seqs[::3]
    c.free(gone)
    m.free(gone)
    c.compact()
    m.compact()
    same(c, m)
    c.extend(gone, counts[:700])
    m.extend(gone, counts[:700])
    same(c, m)
    assert attn.device_status() == 0


def test_a_shared_partial_page_is_copied_before_it_grows():
    c, m = make()
    fill(c, m, [40])
    for x in (c, m):
        x.fork([0, 0], [1, 2])       # full pages shared, partial ones copied
        x.free([0])
        x.extend([1], [8])           # 48 tokens: its last page is full
        x.fork([1], [3])             # so it is shared now
    cut = [3]
    c.keep(cut, [4], torch.zeros(1, 4, dtype=torch.int32), [0])  # and partial again
    m.keep(cut, [4], [[0]], [0])
    same(c, m)
    assert int(c.refs[c.table[3, 2]]) == 2
    for x in (c, m):
        x.extend([3, 1], [2, 2])
    put(c, m, [3, 1], [2, 2], 8)
    same(c, m)
    assert attn.device_status() == 0


def test_rows_through_views():
    """New rows as slices of one projection; a page table wider than its rows."""
    c, m = make(heads=2, d=64)
    wide = torch.full((12, 31), -3, dtype=torch.int32, device="cuda")
    c = attn.Cache(c.k, c.v, wide[:, :20], c.lens, c.refs)
    c.extend([4, 2], [30, 3])
    m.extend([4, 2], [30, 3])
    x = torch.randint(-9, 9, (33, 6, 64)).half().cuda()
    c.write([4, 2], torch.tensor([0, 30, 33], dtype=torch.int64), x[:, 2:4], x[:, 4:], layer=1)
    m.write(1, [4, 2], [0, 30, 33], x[:, 2:4].float().cpu().numpy(), x[:, 4:].float().cpu().numpy())
    np.testing.assert_array_equal(c.k.float().cpu().numpy(), m.k)
    np.testing.assert_array_equal(c.v.float().cpu().numpy(), m.v)
    assert (wide[:, 20:] == -3).all()


@pytest.mark.parametrize("call,code", [
    (lambda c: c.extend([0, 12], [1, 1]), _abi.ATTN_EINVAL),            # no such sequence
    (lambda c: c.extend([0, -1], [1, 1]), _abi.ATTN_EINVAL),
    (lambda c: c.extend([0, 0], [1, 1]), _abi.ATTN_EINVAL),             # listed twice
    (lambda c: c.extend([0, 5], [1, -1]), _abi.ATTN_EINVAL),
    (lambda c: c.extend([5], [321]), _abi.ATTN_EINVAL),                 # more than the table's row holds
    (lambda c: c.extend([5], [(1 << 31) - 1]), _abi.ATTN_EINVAL),
    (lambda c: c.extend([5, 6, 7, 8, 9], [320] * 5), _abi.ATTN_ENOPAGES),
    (lambda c: c.fork([0], [1]), _abi.ATTN_EINVAL),                     # a child that is not empty
    (lambda c: c.fork([0, 0], [5, 5]), _abi.ATTN_EINVAL),
    (lambda c: c.fork([0, 1], [5, 12]), _abi.ATTN_EINVAL),
    (lambda c: c.fork([12], [5]), _abi.ATTN_EINVAL),
    (lambda c: c.keep([0], [41], torch.zeros(1, 4), [0]), None),        # not whole numbers
    (lambda c: c.keep([0], [41], torch.zeros(1, 4, dtype=torch.int32), [0]), _abi.ATTN_EINVAL),
    (lambda c: c.keep([0, 1], [2, 2], torch.tensor([[0, 1], [0, 2]]), [2, 2]), _abi.ATTN_EINVAL),
    (lambda c: c.keep([0], [3], torch.tensor([[1, 1]]), [2]), _abi.ATTN_EINVAL),
    (lambda c: c.keep([0], [3], torch.tensor([[1, 0]]), [2]), _abi.ATTN_EINVAL),
    (lambda c: c.keep([0], [3], torch.tensor([[-1, 0]]), [2]), _abi.ATTN_EINVAL),
    (lambda c: c.keep([0], [3], torch.tensor([[0, 1]]), [3]), _abi.ATTN_EINVAL),
    (lambda c: c.keep([0, 0], [3, 3], torch.tensor([[0], [0]]), [1, 1]), _abi.ATTN_EINVAL),
    (lambda c: c.keep([2], [17], torch.tensor([[1]]), [1]), _abi.ATTN_EINVAL),  # into a shared page
    (lambda c: c.free([13]), _abi.ATTN_EINVAL),
])
def test_a_refused_list_changes_nothing(call, code):
    c, m = make()
    fill(c, m, [40, 17, 32])
    for x in (c, m):
        x.fork([2], [4])
    attn.device_status()
    if code is None:
        with pytest.raises(ValueError):
            call(c)
        return
    call(c)
    same(c, m)
    assert attn.device_status() == code
    assert attn.device_status() == 0


def test_writes_that_do_not_fit_are_skipped():
    c, m = make()
    fill(c, m, [40, 17, 32])
    for x in (c, m):
        x.fork([2], [4])
    attn.device_status()
    k, v = (torch.randint(-9, 9, (9, 3, 64)).half().cuda() for _ in range(2))
    kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
    # too long for its sequence; shared pages; a sequence out of range; one that fits; the same once more
    c.write([5, 2, 99, 1, 1], [0, 2, 4, 5, 7, 9], k, v)
    m.write(0, [1], [5, 7], kn, vn)
    same(c, m)
    assert attn.device_status() == _abi.ATTN_EINVAL
    # rows behind the last entry are not read
    c.write([0], [0, 3], k, v)
    m.write(0, [0], [0, 3], kn, vn)
    same(c, m)
    assert attn.device_status() == 0


def test_a_sequence_freed_twice_is_freed_once():
    c, m = make()
    fill(c, m, [40, 17])
    c.free([0, 0, 1, 0])
    m.free([0, 1])
    same(c, m)
    assert int(c.refs.sum()) == 0 and attn.device_status() == 0


def test_a_page_that_does_not_exist_is_reported():
    c, m = make()
    fill(c, m, [40, 17])
    c.table[0, 1] = 5000
    c.free([0])
    assert attn.device_status() == _abi.ATTN_EINVAL
    assert int(c.refs[int(m.table[0, 1])]) == 1 and int(c.refs[int(m.table[0, 0])]) == 0
    c.table[1, 1] = -1
    c.extend([1], [1])  # its last page cannot be looked at
    assert attn.device_status() == _abi.ATTN_EINVAL and int(c.lens[1]) == 17


def test_empty_lists_do_nothing():
    c, m = make()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    rows = torch.empty(0, 3, 64, dtype=torch.float16, device="cuda")
    c.extend(none, none)
    c.fork([], [])
    c.free(none)
    c.keep(none, none, torch.empty(0, 3, dtype=torch.int32), none)
    c.write(none, [0], rows, rows)
    same(c, m)


def test_a_captured_loop():
    """Room, rows and the kept ones of a draft step in a graph, replayed as the cache grows."""
    c, m = make(n_pages=200, per_seq=40)
    fill(c, m, [20, 7, 33])
    seqs, counts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([2, 0, 1], [4, 4, 4]))
    cu, keep, n_keep = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in
                        ([0, 4, 8, 12], [[0, 2], [1, 3], [0, 0]], [2, 2, 0]))
    k, v = (torch.randint(-9, 9, (12, 3, 64)).half().cuda() for _ in range(2))

    def step(x, seqs, counts, cu, keep, n_keep, write):
        x.extend(seqs, counts)
        write(x)
        x.keep(seqs, counts, keep, n_keep)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c, seqs, counts, cu, keep, n_keep, lambda x: x.write(seqs, cu, k, v))
    for _ in range(7):
        g.replay()
        step(m, [2, 0, 1], [4, 4, 4], None, [[0, 2], [1, 3], [0, 0]], [2, 2, 0],
             lambda x: x.write(0, [2, 0, 1], [0, 4, 8, 12], k.float().cpu().numpy(), v.float().cpu().numpy()))
    same(c, m)
    assert attn.device_status() == 0


@pytest.mark.parametrize("device", ["cuda", "cpu"])
def test_entries_past_32_bits_are_not_cut(device):
    """64-bit lists whose low 32 bits would be a good entry."""
    c, m = make()
    fill(c, m, [40, 17, 32])
    far = 1 << 32
    def refuses(f):
        attn.device_status()
        if device == "cpu":
            with pytest.raises(ValueError, match="32 bits"):
                f()
        else:
            f()
            assert attn.device_status() == _abi.ATTN_EINVAL
        same(c, m)
    def t(*x):
        return torch.tensor(x, device=device)
    k, v = (torch.ones(2, 3, 64).half().cuda() for _ in range(2))
    refuses(lambda: c.extend(t(far), t(1)))
    refuses(lambda: c.extend(t(0), t(far + 1)))
    refuses(lambda: c.fork(t(0), t(far + 5)))
    refuses(lambda: c.free(t(1 - far)))
    refuses(lambda: c.write(t(far), t(0, 2), k, v))
    refuses(lambda: c.write(t(0), t(0, far + 2), k, v))
    refuses(lambda: c.keep(t(0), t(3), t(far + 1).view(1, 1), t(1)))
    refuses(lambda: c.keep(t(0), t(3), t(1).view(1, 1), t(far + 1)))
    q = torch.ones(2, 3, 64).half().cuda()
    refuses(lambda: attn.tree_fwd(q, c, t(far), t(0, 2)))
    c.extend(t(0, 2), t(3, 1))  # 64-bit lists that fit
    m.extend([0, 2], [3, 1])
    same(c, m)
    assert attn.device_status() == 0
