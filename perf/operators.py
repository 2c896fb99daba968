"""Cases of the grouped-head and cache operators, their plain forms, and their values in 64 bits.

``run`` computes an operator in its plain form (elementary torch operations in
f32, rounded once) or, with ``own`` set, through this package's entry points.
``work`` counts what a pass cannot do without: each input read once, each output
written once, and the multiply-adds of the admitted pairs.

Kinds of case:
  prompt    attention over whole prompts: causal, packed sequences, grouped heads
  train     the same forward followed by its backward (dq, dk, dv)
  tree      new tokens (one, a chunk, a tree of drafts) over a paged cache
  fork      sequences forked into children, and the children freed again
  compact   the live pages of a fragmented pool moved to its front
  draft     room for drafted tokens, their rows written, the accepted ones kept
"""
from __future__ import annotations

import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a single short prompt: latency
        dict(name="prompt_one_short", kind="prompt", n_seq=1, lo=37, hi=37, hq=8, hkv=2, d=64, dtype="f16", mix=1),
        # a batch of chat turns, packed
        dict(name="prompt_chat_batch", kind="prompt", n_seq=48, lo=9, hi=420, hq=32, hkv=8, d=128, dtype="bf16", mix=2),
        # long documents: the largest prompt call
        dict(name="prompt_documents", kind="prompt", n_seq=3, lo=5000, hi=8192, hq=32, hkv=8, d=128, dtype="bf16", mix=3),
        # fine-tuning on packed short samples, every head of its own group size 4, f16
        dict(name="train_packed", kind="train", n_seq=24, lo=30, hi=1000, hq=16, hkv=4, d=64, dtype="f16", mix=4),
        # pre-training step on full-length rows
        dict(name="train_rows", kind="train", n_seq=2, lo=4096, hi=4096, hq=32, hkv=8, d=128, dtype="bf16", mix=5),
        # decoding for one user
        dict(name="decode_one", kind="tree", n_seq=1, lo=700, hi=700, t_lo=1, t_hi=1, tree=False, hq=32, hkv=8, d=128,
             page=16, dtype="bf16", mix=6),
        # decoding for a full batch of ragged contexts
        dict(name="decode_batch", kind="tree", n_seq=96, lo=64, hi=12000, t_lo=1, t_hi=1, tree=False, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", mix=7),
        # speculative decoding: small trees for a few users, ragged draft counts
        dict(name="tree_small", kind="tree", n_seq=6, lo=900, hi=5000, t_lo=5, t_hi=24, tree=True, hq=16, hkv=4, d=64,
             page=32, dtype="f16", mix=8),
        # speculative decoding: wide trees over long contexts
        dict(name="tree_wide", kind="tree", n_seq=8, lo=9000, hi=30000, t_lo=63, t_hi=63, tree=True, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", mix=9),
        # parallel sampling: each prompt forked into four continuations, the losers freed
        dict(name="fork_free", kind="fork", n_seq=40, children=4, lo=100, hi=1500, hkv=8, d=128, page=32, layers=4,
             dtype="bf16", mix=10),
        # an aged pool brought to its front
        dict(name="compact_pool", kind="compact", n_seq=120, drop=0.5, lo=40, hi=1200, hkv=8, d=128, page=32, layers=4,
             dtype="bf16", mix=11),
        # one verification step's cache work: drafts in, accepted path kept
        dict(name="draft_step", kind="draft", n_seq=32, t=48, kept=6, lo=200, hi=3000, hkv=8, d=128, page=16, layers=8,
             dtype="bf16", mix=12),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "train", "tree", "tree", "tree", "fork", "compact", "draft"])
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    c = dict(kind=kind, d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f16"]), mix=rng.randrange(1 << 30), hkv=hkv)
    if kind in ("prompt", "train"):
        n = _log(rng, 1, 48)
        hi = _log(rng, 1, min(6000, int(20000 / n ** 0.75)) if kind == "prompt" else min(3000, int(9000 / n ** 0.75)))
        c.update(n_seq=n, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, hq=hkv * g)
    elif kind == "tree":
        n = _log(rng, 1, 96)
        t = rng.choice([1, 1, _log(rng, 1, 64), _log(rng, 2, 100)])
        hi = _log(rng, t + 1, max(200, min(24000, int(260000 / n))))
        c.update(n_seq=n, lo=max(t, hi // rng.choice([1, 2, 16])), hi=hi, t_lo=max(1, t // rng.choice([1, 2, 4])), t_hi=t,
                 tree=t > 1 and rng.random() < 0.7, hq=hkv * g, page=rng.choice([8, 16, 32, 64, 128]))
    else:
        hi = _log(rng, 20, 2000)
        c.update(n_seq=_log(rng, 1, 100), lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, page=rng.choice([8, 16, 32, 64, 128]),
                 layers=rng.choice([1, 2, 3, 4]))
        if kind == "fork":
            c.update(children=rng.randrange(1, 6))
        elif kind == "compact":
            c.update(drop=rng.choice([0.1, 0.3, 0.5, 0.8]))
        else:
            t = _log(rng, 1, 64)
            c.update(t=t, kept=rng.randrange(0, t + 1))
    return c


# ---- sizes that follow from a case -------------------------------------------------


def _spread(case, lo, hi, n, salt):
    r = random.Random("%d %d" % (case["mix"], salt))
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case):
    """The sequences' lengths (in the tree cases with the new tokens)."""
    return _spread(case, case["lo"], case["hi"], case["n_seq"], 0)


def _news(case):
    """New tokens of each sequence of a tree case."""
    return [min(t, n) for t, n in zip(_spread(case, case["t_lo"], case["t_hi"], case["n_seq"], 1), _lens(case))]


def _kept(case):
    """Accepted drafts of each sequence: between one fewer and one more than usual."""
    return [max(0, min(case["t"], case["kept"] + x)) for x in _spread(case, -1, 1, case["n_seq"], 2)]


def _dropped(case):
    """Which sequences of the pool were freed before it is compacted."""
    r = random.Random("%d 3" % case["mix"])
    return [r.random() < case["drop"] for _ in range(case["n_seq"])]


def _pages(n, page):
    return -(-n // page)


def work(case):
    kind, d = case["kind"], case["d"]
    lens = _lens(case)
    if kind in ("prompt", "train"):
        rows, hq, hkv = sum(lens), case["hq"], case["hkv"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        q, kv, stat = 2 * rows * hq * d, 2 * rows * hkv * d, 4 * rows * hq
        if kind == "prompt":
            return {"bytes": 2 * q + 2 * kv + stat, "flops": 4 * d * hq * pairs}
        return {"bytes": 4 * q + 4 * kv + stat, "flops": 14 * d * hq * pairs}  # q, dO in; o, dq out; k, v; dk, dv
    if kind == "tree":
        news, hq, hkv = _news(case), case["hq"], case["hkv"]
        pairs = sum(t * (n - t) + t * (t + 1) // 2 for t, n in zip(news, lens))
        rows = sum(news)
        return {"bytes": 4 * sum(lens) * hkv * d + 4 * rows * hq * d + 4 * rows * hq + 4 * sum(_pages(n, case["page"]) for n in lens),
                "flops": 4 * d * hq * pairs}
    row = 2 * 2 * case["layers"] * case["hkv"] * d  # a token's k and v rows of all layers
    page = case["page"]
    if kind == "fork":
        moved = sum(n % page for n in lens) * case["children"]
        return {"bytes": 2 * moved * row + 8 * sum(_pages(n, page) for n in lens) * case["children"], "flops": 0}
    if kind == "compact":
        live, moved = _compact_counts(case)
        return {"bytes": 2 * moved * page * row + 8 * live, "flops": 0}
    moved = sum(max(0, k - 1) for k in _kept(case))  # the first accepted draft stays where it is
    return {"bytes": 2 * case["n_seq"] * case["t"] * row + 2 * moved * row, "flops": 0}


def _compact_counts(case):
    """(live pages, live pages that lie beyond them) of the pool of a compact case."""
    _, table, _, refs = _tables(case, _lens(case), 0)
    live = refs > 0
    n = int(live.sum())
    return n, int(live[n:].sum())


# ---- inputs ---------------------------------------------------------------------------


def _tables(case, lens, spare):
    """An aged pool: (pages, table, sequence ids, refs); each sequence's pages lie scattered over the pool."""
    r = np.random.RandomState(case["mix"] % (1 << 31))
    page, n = case["page"], len(lens)
    need = [_pages(x, page) for x in lens]
    n_pages = sum(need) + spare + max(4, sum(need) // 8)
    width = max(need) + _pages(case.get("t", 0), page) + 1
    slots = n * (1 + case.get("children", 0)) + 3
    order = r.permutation(n_pages)
    ids = r.permutation(slots).astype(np.int32)
    table = np.zeros((slots, width), np.int32)
    refs = np.zeros(n_pages, np.int32)
    dropped = _dropped(case) if case["kind"] == "compact" else [False] * n
    at = 0
    for i, k in enumerate(need):
        table[ids[i], :k] = order[at:at + k]
        refs[order[at:at + k]] = 0 if dropped[i] else 1
        at += k
    return n_pages, table, ids, refs


def _cache(case, gen, lens, spare=0):
    n_pages, table, ids, refs = _tables(case, lens, spare)
    dev = "cuda"
    shape = (case.get("layers", 1), n_pages, case["page"], case["hkv"], case["d"])
    dropped = _dropped(case) if case["kind"] == "compact" else [False] * len(lens)
    all_lens = np.zeros(table.shape[0], np.int32)
    all_lens[ids[:len(lens)]] = [0 if x else n for x, n in zip(dropped, lens)]
    s = {"k": torch.randn(shape, generator=gen, device=dev, dtype=_DT[case["dtype"]]),
         "v": torch.randn(shape, generator=gen, device=dev, dtype=_DT[case["dtype"]]),
         "table": torch.from_numpy(table).to(dev), "lens": torch.from_numpy(all_lens).to(dev),
         "refs": torch.from_numpy(refs).to(dev), "ids": torch.from_numpy(ids).to(dev)}
    s["seqs"] = s["ids"][:len(lens)].contiguous()
    if own:  # the handle of the cache, which a program keeps as long as the cache
        import online_softmax_attention_gb300 as attn
        s["cache"] = attn.Cache(s["k"], s["v"], s["table"], s["lens"], s["refs"])
    return s


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def _tree_mask(gen_np, news, words):
    """A random tree over each sequence's drafts: a draft sees its ancestors and itself."""
    out = np.zeros((sum(news), words), np.uint64)
    at = 0
    for t in news:
        for u in range(t):
            if u:
                out[at + u] = out[at + gen_np.randint(max(0, u - 6), u)]
            out[at + u, u >> 6] |= np.uint64(1) << np.uint64(u & 63)
        at += t
    return torch.from_numpy(out.view(np.int64)).to("cuda")


def prepare(case, seed):
    kind = case["kind"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = np.random.RandomState(seed % (1 << 31))
    lens, dt, d = _lens(case), _DT[case["dtype"]], case["d"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dt)

    if kind in ("prompt", "train"):
        rows = sum(lens)
        s = {"q": randn(rows, case["hq"], d), "k": randn(rows, case["hkv"], d), "v": randn(rows, case["hkv"], d),
             "cu": _cu(lens), "longest": max(lens)}
        if kind == "train":
            s["do"] = randn(rows, case["hq"], d)
    elif kind == "tree":
        news = _news(case)
        s = _cache(case, gen, lens)
        s.update(q=randn(sum(news), case["hq"], d), cu=_cu(news), longest=max(news), width=max(lens),
                 mask=_tree_mask(rnd, news, _pages(max(news), 64)) if case["tree"] else None)
    elif kind == "fork":
        n, c = len(lens), case["children"]
        s = _cache(case, gen, lens, spare=n * c)
        s["parents"] = s["seqs"].repeat_interleave(c)
        s["children"] = s["ids"][n:n + n * c].contiguous()
    elif kind == "compact":
        s = _cache(case, gen, lens)
    else:
        t, kept = case["t"], _kept(case)
        s = _cache(case, gen, lens, spare=len(lens) * (_pages(t, case["page"]) + 1))
        keep = np.zeros((len(lens), t), np.int32)
        for i, k in enumerate(kept):  # an accepted path starts at the first draft
            keep[i, :k] = [0] + sorted(rnd.choice(np.arange(1, t), k - 1, replace=False)) if k else []
        rows = len(lens) * t
        s.update(counts=torch.full((len(lens),), t, dtype=torch.int32, device="cuda"), cu=_cu([t] * len(lens)),
                 keep=torch.from_numpy(keep).to("cuda"), n_keep=torch.tensor(kept, dtype=torch.int32, device="cuda"),
                 new_k=[randn(rows, case["hkv"], d) for _ in range(case["layers"])],
                 new_v=[randn(rows, case["hkv"], d) for _ in range(case["layers"])])
    if kind in ("compact", "draft"):
        s["before"] = {n: s[n].clone() for n in ("table", "lens", "refs")}
    s["kind"] = kind
    return s


# ---- plain forms ------------------------------------------------------------------------


def _padded(x, cu, longest):
    """Packed rows (T, H, D) as (sequences, longest, H, D) f32 and which of them exist."""
    start, n = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    at = torch.arange(longest, device=x.device)
    live = at[None] < n[:, None]
    rows = torch.where(live, start[:, None] + at[None], 0)
    return torch.where(live[:, :, None, None], x[rows].float(), 0.0), live, rows


def _softmax(s, seen):
    """p, lse of scores where only `seen` pairs exist; a row without any has p = 0, lse = -inf."""
    s = s.masked_fill(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = (s - m).exp()
    total = p.sum(-1, keepdim=True)
    return p / total.clamp(min=1e-38), (m + total.log()).squeeze(-1)


def _plain_prompt(s):
    hkv, d = s["k"].shape[1:]
    g = s["q"].shape[1] // hkv
    q, live, rows = _padded(s["q"], s["cu"], s["longest"])
    k, v = _padded(s["k"], s["cu"], s["longest"])[0], _padded(s["v"], s["cu"], s["longest"])[0]
    b, n = live.shape
    q = q.view(b, n, hkv, g, d)
    scores = torch.einsum("bihgd,bjhd->bhgij", q, k) * d ** -0.5
    at = torch.arange(n, device=q.device)
    p, lse = _softmax(scores, (at[None, :] <= at[:, None]) & live[:, None, None, None, :])
    del scores
    o = torch.einsum("bhgij,bjhd->bihgd", p, v)
    packed_o = o.reshape(b, n, hkv * g, d)[live].to(s["q"].dtype)
    packed_lse = lse.permute(0, 3, 1, 2).reshape(b, n, hkv * g)[live].t().contiguous()
    if "do" not in s:
        return packed_o, packed_lse
    do = _padded(s["do"], s["cu"], s["longest"])[0].view(b, n, hkv, g, d)
    dv = torch.einsum("bhgij,bihgd->bjhd", p, do)
    dp = torch.einsum("bihgd,bjhd->bhgij", do, v)
    ds = p.mul_(dp.sub_((do * o).sum(-1).permute(0, 2, 3, 1)[..., None]))
    del dp
    dq = torch.einsum("bhgij,bjhd->bihgd", ds, k).reshape(b, n, hkv * g, d) * d ** -0.5
    dk = torch.einsum("bhgij,bihgd->bjhd", ds, q) * d ** -0.5
    return packed_o, packed_lse, dq[live].to(s["q"].dtype), dk[live].to(s["q"].dtype), dv[live].to(s["q"].dtype)


def _plain_tree(s):
    page, hkv, d = s["k"].shape[2:]
    q, live, _ = _padded(s["q"], s["cu"], s["longest"])
    b, t = live.shape
    g = s["q"].shape[1] // hkv
    slots = -(-s["width"] // page)
    held = s["table"][s["seqs"].long(), :slots].long()
    k = s["k"][0][held].reshape(b, slots * page, hkv, d).float()
    v = s["v"][0][held].reshape(b, slots * page, hkv, d).float()
    at = torch.arange(slots * page, device=q.device)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    n = s["lens"][s["seqs"].long()].long()
    draft = at[None] - (n - new)[:, None]  # a key's place among the new tokens; negative: before them
    if s["mask"] is None:
        seen = draft[:, None, :] <= torch.arange(t, device=q.device)[None, :, None]
    else:
        rows = torch.where(live, s["cu"][:-1].long()[:, None] + torch.arange(t, device=q.device)[None], 0)
        word = draft.clamp(0, 64 * s["mask"].shape[1] - 1)
        words = s["mask"][rows].gather(2, (word >> 6)[:, None, :].expand(b, t, -1))
        seen = (draft[:, None, :] < 0) | ((words >> (word & 63)[:, None, :]) & 1).bool()
    seen = seen & (at[None] < n[:, None])[:, None, :] & live[:, :, None]
    scores = torch.einsum("bihgd,bjhd->bhgij", q.view(b, t, hkv, g, d), k) * d ** -0.5
    p, lse = _softmax(scores, seen[:, None, None])
    v = torch.where((at[None] < n[:, None])[:, :, None, None], v, 0.0)
    o = torch.einsum("bhgij,bjhd->bihgd", p, v).reshape(b, t, hkv * g, d)
    return o[live].to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(b, t, hkv * g)[live].t().contiguous()


def _lowest_free(refs, ranks):
    """The free pages of the given ranks (0 = the lowest)."""
    return torch.searchsorted(torch.cumsum(refs == 0, 0), ranks + 1).clamp(max=refs.numel() - 1)


def _plain_fork(s):
    page = s["k"].shape[2]
    table, lens, refs, parents, children = s["table"], s["lens"], s["refs"], s["parents"].long(), s["children"].long()
    n = lens[parents].long()
    tail = n % page
    need = (tail > 0).long()
    new = _lowest_free(refs, torch.cumsum(need, 0) - need)
    slot = torch.arange(table.shape[1], device=refs.device)[None]
    shared, last = slot < (n // page)[:, None], slot == (n // page)[:, None]
    rows = table[parents].long()
    old = torch.where(need > 0, rows.gather(1, (n // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0], new)
    table[children] = torch.where(shared, rows, torch.where(last & (need > 0)[:, None], new[:, None], table[children].long())).int()
    refs.index_add_(0, rows.reshape(-1), shared.reshape(-1).int())
    refs.index_add_(0, new, need.int())
    lens[children] = n.int()
    has = need.nonzero()[:, 0]  # the forks that copy a page
    copied = (torch.arange(page, device=refs.device)[None] < tail[has][:, None])[None, :, :, None, None]
    s["k"][:, new[has]] = torch.where(copied, s["k"][:, old[has]], s["k"][:, new[has]])
    s["v"][:, new[has]] = torch.where(copied, s["v"][:, old[has]], s["v"][:, new[has]])
    forked = lens.clone(), refs.clone()
    held = slot < torch.ceil(n / page)[:, None]  # the children are freed again
    refs.index_add_(0, table[children].long().reshape(-1), -held.reshape(-1).int())
    lens[children] = 0
    return [*forked, table, lens, refs, s["k"], s["v"]]


def _plain_compact(s):
    page = s["k"].shape[2]
    table, lens, refs = s["table"], s["lens"], s["refs"]
    live = refs > 0
    at = torch.arange(refs.numel(), device=refs.device)
    front = at < live.sum()
    holes, movers = (~live & front).nonzero()[:, 0], (live & ~front).nonzero()[:, 0]
    s["k"][:, holes] = s["k"][:, movers]
    s["v"][:, holes] = s["v"][:, movers]
    to = at.int()
    to[movers] = holes.int()
    refs[holes] = refs[movers]
    refs[movers] = 0
    held = torch.arange(table.shape[1], device=refs.device)[None] < ((lens + page - 1) // page)[:, None]
    table.copy_(torch.where(held, to[table.long()], table))
    return [table, lens, refs, s["k"], s["v"]]


def _plain_draft(s):
    page = s["k"].shape[2]
    table, lens, refs, seqs = s["table"], s["lens"], s["refs"], s["seqs"].long()
    t = s["keep"].shape[1]
    # room
    n = lens[seqs].long()
    have, want = (n + page - 1) // page, (n + t + page - 1) // page
    need = want - have
    first = torch.cumsum(need, 0) - need
    slot = torch.arange(table.shape[1], device=refs.device)[None]
    fresh = (slot >= have[:, None]) & (slot < want[:, None])
    new = _lowest_free(refs, (first - have)[:, None] + slot)
    table[seqs] = torch.where(fresh, new.int(), table[seqs])
    refs.index_add_(0, torch.where(fresh, new, 0).reshape(-1), fresh.reshape(-1).int())
    # rows
    u = torch.arange(t, device=refs.device)[None]
    place = n[:, None] + u
    pages, rows = table[seqs].long().gather(1, place // page), place % page
    new_k, new_v = torch.stack(s["new_k"]), torch.stack(s["new_v"])
    s["k"][:, pages, rows] = new_k.view(new_k.shape[0], *place.shape, *new_k.shape[2:])
    s["v"][:, pages, rows] = new_v.view(new_v.shape[0], *place.shape, *new_v.shape[2:])
    # accepted ones follow the prefix; the places behind them keep what they hold
    source = torch.where(u < s["n_keep"].long()[:, None], n[:, None] + s["keep"].long(), place)
    from_pages, from_rows = table[seqs].long().gather(1, source // page), source % page
    s["k"][:, pages, rows] = s["k"][:, from_pages, from_rows]
    s["v"][:, pages, rows] = s["v"][:, from_pages, from_rows]
    after = n + s["n_keep"].long()
    dropped = (slot >= ((after + page - 1) // page)[:, None]) & (slot < want[:, None])
    refs.index_add_(0, torch.where(dropped, table[seqs].long(), 0).reshape(-1), -dropped.reshape(-1).int())
    lens[seqs] = after.int()
    return [table, lens, refs, s["k"], s["v"]]


def run(state):
    s, kind = state, state["kind"]
    if kind in ("compact", "draft"):  # the pool as it was before the pass
        s["table"].copy_(s["before"]["table"])
        s["lens"].copy_(s["before"]["lens"])
        s["refs"].copy_(s["before"]["refs"])
    if not own:
        plain = {"prompt": _plain_prompt, "train": _plain_prompt, "tree": _plain_tree, "fork": _plain_fork,
                 "compact": _plain_compact, "draft": _plain_draft}
        return plain[kind](s)

    import online_softmax_attention_gb300 as attn

    if kind in ("prompt", "train"):
        o, lse = attn.fwd(s["q"], s["k"], s["v"], causal=True, cu_seqlens_q=s["cu"])
        if kind == "prompt":
            return o, lse
        return (o, lse) + attn.bwd(s["q"], s["k"], s["v"], o, lse, s["do"], causal=True, cu_seqlens_q=s["cu"])
    cache = s["cache"]
    if kind == "tree":
        return attn.tree_fwd(s["q"], cache, s["seqs"], s["cu"], mask=s["mask"])
    if kind == "fork":
        cache.fork(s["parents"], s["children"])
        forked = [s["lens"].clone(), s["refs"].clone()]
        cache.free(s["children"])
        return forked + [s["table"], s["lens"], s["refs"], s["k"], s["v"]]
    if kind == "compact":
        cache.compact()
    else:
        cache.extend(s["seqs"], s["counts"])
        for layer, (k, v) in enumerate(zip(s["new_k"], s["new_v"])):
            cache.write(s["seqs"], s["cu"], k, v, layer=layer)
        cache.keep(s["seqs"], s["counts"], s["keep"], s["n_keep"])
    return [s["table"], s["lens"], s["refs"], s["k"], s["v"]]


# ---- 64 bits ----------------------------------------------------------------------------


def exact(case, seed):
    """The attention kinds from their definition, one sequence and head at a time, in f64."""
    kind = case["kind"]
    if kind not in ("prompt", "train", "tree"):
        return None  # values are moved, not computed
    s = prepare(case, seed)
    lens, hq, group, d = _lens(case), case["hq"], case["hq"] // case["hkv"], case["d"]
    news = _news(case) if kind == "tree" else lens
    rows = sum(news)
    o = torch.zeros(rows, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(hq, rows, dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros(rows, h, d, dtype=torch.float64, device="cuda") for h in (hq, case["hkv"], case["hkv"]))
    at = 0
    for i, (n, t) in enumerate(zip(lens, news)):
        mine = slice(at, at + t)
        at += t
        if kind == "tree":
            held = s["table"][int(s["seqs"][i]), :_pages(n, case["page"])].long()
            keys, values = (s[x][0][held].flatten(0, 1)[:n].double() for x in ("k", "v"))
            hidden = torch.ones(t, n, dtype=torch.bool, device="cuda").triu(n - t + 1)
            if s["mask"] is not None:
                bits = torch.arange(64, device="cuda")
                hidden[:, n - t:] = ((s["mask"][mine][:, :, None] >> bits) & 1).flatten(1)[:, :t] == 0
                hidden[:, :n - t] = False
        else:
            keys, values = s["k"][mine].double(), s["v"][mine].double()
            hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for h in range(hq):
            q, k, v = s["q"][mine, h].double(), keys[:, h // group], values[:, h // group]
            x = (q @ k.T) / d ** 0.5
            x[hidden] = -torch.inf
            lse[h, mine] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[h, mine][:, None])
            o[mine, h] = p @ v
            if kind == "train":
                do = s["do"][mine, h].double()
                dv[mine, h // group] += p.T @ do
                y = do @ v.T
                ds = p * (y - (p * y).sum(1, keepdim=True)) / d ** 0.5
                dq[mine, h] = ds @ k
                dk[mine, h // group] += ds.T @ q
    return (o, lse, dq, dk, dv) if kind == "train" else (o, lse)
