"""Cases of windowed attention with sinks and of eviction from the cache by attention weight, their plain forms, and their values in 64 bits.

``run`` computes an operator in its plain form (elementary torch operations in
f32, rounded once) or, with ``own`` set, through this package's entry points.
``work`` counts what a pass cannot do without: each input read once, each output
written once, and the multiply-adds of the admitted pairs.

Of the keys that a query would see without a window, in order, it sees the first
``sinks`` and the last ``window``.

Kinds of case:
  prompt    attention over whole prompts: causal, packed sequences, grouped heads, windowed
  train     the same forward followed by its backward (dq, dk, dv)
  tree      new tokens (one, a chunk, a tree of drafts) over a paged cache, windowed
  weigh     attention weight that the cached tokens get from new ones, accumulated
  evict     each sequence cut to its heaviest tokens, their rows moved together
"""
from __future__ import annotations

import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # a single short prompt: latency
        dict(name="window_prompt_short", kind="prompt", n_seq=1, lo=150, hi=150, hq=8, hkv=2, d=64, dtype="f16", window=64,
             sinks=4, mix=1),
        # a batch of chat turns, packed, in a layer of short windows
        dict(name="window_prompt_batch", kind="prompt", n_seq=48, lo=9, hi=420, hq=32, hkv=8, d=128, dtype="bf16", window=128,
             sinks=0, mix=2),
        # long documents, many windows long
        dict(name="window_prompt_long", kind="prompt", n_seq=2, lo=14000, hi=16384, hq=32, hkv=8, d=128, dtype="bf16",
             window=2048, sinks=4, mix=3),
        # fine-tuning on packed short samples
        dict(name="window_train_packed", kind="train", n_seq=24, lo=30, hi=1000, hq=16, hkv=4, d=64, dtype="f16", window=200,
             sinks=1, mix=4),
        # a training step on full-length rows
        dict(name="window_train_rows", kind="train", n_seq=2, lo=8192, hi=8192, hq=32, hkv=8, d=128, dtype="bf16", window=1024,
             sinks=4, mix=5),
        # decoding for one user, a long context behind the window
        dict(name="window_decode_one", kind="tree", n_seq=1, lo=21000, hi=21000, t_lo=1, t_hi=1, tree=False, hq=32, hkv=8,
             d=128, page=16, dtype="bf16", window=1024, sinks=4, mix=6),
        # decoding for a full batch of ragged contexts
        dict(name="window_decode_batch", kind="tree", n_seq=96, lo=64, hi=12000, t_lo=1, t_hi=1, tree=False, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", window=2048, sinks=4, mix=7),
        # speculative decoding: wide trees over long contexts
        dict(name="window_tree_wide", kind="tree", n_seq=8, lo=9000, hi=30000, t_lo=63, t_hi=63, tree=True, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", window=4096, sinks=4, mix=8),
        # a decoding step's weights, every sequence's new token
        dict(name="weigh_decode", kind="weigh", n_seq=64, lo=200, hi=6000, t_lo=1, t_hi=1, whole=False, hq=32, hkv=8, d=128,
             page=16, layers=2, dtype="bf16", window=0, sinks=0, mix=9),
        # the weights of fresh prompts, from their last tokens
        dict(name="weigh_prompt", kind="weigh", n_seq=4, lo=1500, hi=8000, t_lo=64, t_hi=64, whole=True, hq=32, hkv=8, d=128,
             page=64, layers=1, dtype="bf16", window=0, sinks=0, mix=10),
        # one user's conversation brought back to its budget
        dict(name="evict_one", kind="evict", n_seq=1, lo=1280, hi=1280, budget=1024, sinks=4, recent=128, hkv=8, d=128, page=16,
             layers=4, dtype="bf16", mix=11),
        # long prompts cut to a budget before they are decoded
        dict(name="evict_batch", kind="evict", n_seq=32, lo=900, hi=6000, budget=1024, sinks=4, recent=64, hkv=8, d=128, page=64,
             layers=8, dtype="bf16", mix=12),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "train", "train", "tree", "tree", "weigh", "weigh", "evict", "evict"])
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    c = dict(kind=kind, d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f16"]), mix=rng.randrange(1 << 30), hkv=hkv)
    if kind in ("prompt", "train"):
        if rng.random() < 0.15:
            c.update(dtype="f32")
        most = 2000 if c["dtype"] == "f32" else 8000 if kind == "prompt" else 4000
        n = _log(rng, 1, 48)
        hi = _log(rng, 1, max(1, min(most, int(2 * most / n ** 0.75))))
        c.update(n_seq=n, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, hq=hkv * g, window=_log(rng, 1, max(2, 2 * hi)),
                 sinks=rng.choice([0, 0, 1, 4, _log(rng, 1, 300)]))
    elif kind == "tree":
        n = _log(rng, 1, 96)
        t = rng.choice([1, 1, _log(rng, 1, 64), _log(rng, 2, 100)])
        hi = _log(rng, t + 1, max(200, min(24000, int(260000 / n))))
        c.update(n_seq=n, lo=max(t, hi // rng.choice([1, 2, 16])), hi=hi, t_lo=max(1, t // rng.choice([1, 2, 4])), t_hi=t,
                 tree=t > 1 and rng.random() < 0.7, hq=hkv * g, page=rng.choice([8, 16, 32, 64, 128]),
                 window=_log(rng, 1, min(4096, 2 * hi)), sinks=rng.choice([0, 1, 4, _log(rng, 1, 200)]))
    elif kind == "weigh":
        n = _log(rng, 1, 64)
        t = rng.choice([1, 1, _log(rng, 1, 64), _log(rng, 1, 200)])
        hi = _log(rng, t + 1, max(200, min(8000, int(200000 / n))))
        windowed = rng.random() < 0.3
        c.update(n_seq=n, lo=max(t, hi // rng.choice([1, 2, 16])), hi=hi, t_lo=max(1, t // rng.choice([1, 2, 4])), t_hi=t,
                 whole=rng.random() < 0.5, hq=hkv * g, page=rng.choice([8, 16, 32, 64, 128]), layers=rng.choice([1, 2, 3]),
                 window=_log(rng, 1, 2 * hi) if windowed else 0, sinks=rng.choice([0, 4]) if windowed else 0)
    else:
        hi = _log(rng, 20, 6000)
        budget = _log(rng, 1, hi)
        sinks = rng.choice([0, 0, 1, 4])
        c.update(n_seq=_log(rng, 1, 64), lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, budget=budget, sinks=min(sinks, budget),
                 recent=int((budget - min(sinks, budget)) * rng.choice([0, 0.1, 0.5, 1])), page=rng.choice([8, 16, 32, 64, 128]),
                 layers=rng.choice([1, 2, 3, 4]))
    return c


# ---- sizes that follow from a case -------------------------------------------------


def _spread(case, lo, hi, n, salt):
    r = random.Random("%d %d" % (case["mix"], salt))
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case):
    """The sequences' lengths (over a cache with the new tokens)."""
    return _spread(case, case["lo"], case["hi"], case["n_seq"], 0)


def _news(case):
    """New tokens of each sequence of a tree or weigh case."""
    return [min(t, n) for t, n in zip(_spread(case, case["t_lo"], case["t_hi"], case["n_seq"], 1), _lens(case))]


def _pages(n, page):
    return -(-n // page)


def _seen(case, first, last):
    """Pairs of the queries at places [first, last) of a sequence with the keys that they see."""
    n = np.arange(first + 1, last + 1)
    w, s = case["window"] or n[-1:].max(initial=0), case["sinks"]
    return int((np.minimum(n, w) + np.clip(n - w, 0, s)).sum())


def work(case):
    kind, d = case["kind"], case["d"]
    es = 4 if case["dtype"] == "f32" else 2
    lens = _lens(case)
    if kind in ("prompt", "train"):
        rows, hq, hkv = sum(lens), case["hq"], case["hkv"]
        pairs = sum(_seen(case, 0, n) for n in lens)
        q, kv, stat = es * rows * hq * d, es * rows * hkv * d, 4 * rows * hq
        if kind == "prompt":
            return {"bytes": 2 * q + 2 * kv + stat, "flops": 4 * d * hq * pairs}
        return {"bytes": 4 * q + 4 * kv + stat, "flops": 14 * d * hq * pairs}  # q, dO in; o, dq out; k, v; dk, dv
    if kind in ("tree", "weigh"):
        news, hq, hkv = _news(case), case["hq"], case["hkv"]
        pairs = sum(_seen(case, n - t, n) for t, n in zip(news, lens))
        # rows that some new token sees
        read = sum(min(n, t - 1 + case["window"] + case["sinks"]) if case["window"] else n for t, n in zip(news, lens))
        rows, table = sum(news), 4 * sum(_pages(n, case["page"]) for n in lens)
        if kind == "tree":
            return {"bytes": 2 * es * (read * hkv + rows * hq) * d + 4 * rows * hq + table, "flops": 4 * d * hq * pairs}
        fresh = sum(lens) if case["whole"] else rows
        return {"bytes": es * (read * hkv + rows * hq) * d + 4 * rows * hq + 4 * sum(lens) + 4 * (sum(lens) - fresh) + table,
                "flops": 2 * d * hq * pairs}
    row = 2 * es * case["layers"] * case["hkv"] * d  # a token's k and v rows of all layers
    moved = sum(case["budget"] - case["sinks"] for n in lens if n > case["budget"])
    weighed = sum(n for n in lens if n > case["budget"])
    return {"bytes": 2 * moved * (row + 4 * case["layers"]) + 4 * weighed * case["layers"], "flops": 0}


# ---- inputs ---------------------------------------------------------------------------


def _cache(case, gen, lens):
    """An aged pool: each sequence's pages lie scattered over it."""
    r = np.random.RandomState(case["mix"] % (1 << 31))
    page, n = case["page"], len(lens)
    need = [_pages(x, page) for x in lens]
    n_pages = sum(need) + max(4, sum(need) // 8)
    width, slots = max(need) + 1, n + 3
    order = r.permutation(n_pages)
    ids = r.permutation(slots).astype(np.int32)
    table = np.zeros((slots, width), np.int32)
    refs = np.zeros(n_pages, np.int32)
    all_lens = np.zeros(slots, np.int32)
    all_lens[ids[:n]] = lens
    refs[order[:sum(need)]] = 1
    for i, (k, end) in enumerate(zip(need, np.cumsum(need))):
        table[ids[i], :k] = order[end - k:end]
    shape = (case.get("layers", 1), n_pages, page, case["hkv"], case["d"])
    s = {"k": torch.randn(shape, generator=gen, device="cuda", dtype=_DT[case["dtype"]]),
         "v": torch.randn(shape, generator=gen, device="cuda", dtype=_DT[case["dtype"]]),
         "table": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(all_lens).cuda(),
         "refs": torch.from_numpy(refs).cuda(), "seqs": torch.from_numpy(ids[:n].copy()).cuda()}
    if own:  # the handle of the cache, which a program keeps as long as the cache
        import online_softmax_attention_gb300 as attn
        s["cache"] = attn.Cache(s["k"], s["v"], s["table"], s["lens"], s["refs"])
    return s


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def _tree_mask(rnd, news, words):
    """A random tree over each sequence's drafts: a draft sees its ancestors and itself."""
    out = np.zeros((sum(news), words), np.uint64)
    at = 0
    for t in news:
        for u in range(t):
            if u:
                out[at + u] = out[at + rnd.randint(max(0, u - 6), u)]
            out[at + u, u >> 6] |= np.uint64(1) << np.uint64(u & 63)
        at += t
    return torch.from_numpy(out.view(np.int64)).cuda()


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
    else:
        s = _cache(case, gen, lens)
    if kind in ("tree", "weigh"):
        news = _news(case)
        s.update(q=randn(sum(news), case["hq"], d), cu=_cu(news), longest=max(news), width=max(lens))
    if kind == "tree":
        s["mask"] = _tree_mask(rnd, news, _pages(max(news), 64)) if case["tree"] else None
    if kind == "weigh":
        # the rows' lse, which the attention over the cache gave
        s.update(window=case["window"], sinks=case["sinks"], layer=case["layers"] - 1)
        s["lse"] = _softmax(*_cached_scores(s))[1]
        shape = (case["layers"], *s["table"].shape[:1], s["table"].shape[1] * case["page"])
        s["weights"] = torch.rand(shape, generator=gen, device="cuda").pow_(8)
        s["fresh"] = torch.tensor(lens if case["whole"] else news, dtype=torch.int32, device="cuda")
        s["before"] = {"weights": s["weights"].clone()}
    if kind == "evict":
        # accumulated weights: few heavy tokens, many light ones, and some that nothing ever looked at
        shape = (case["layers"], *s["table"].shape[:1], s["table"].shape[1] * case["page"])
        s["weights"] = torch.randn(shape, generator=gen, device="cuda").mul_(2).exp_()
        s["weights"].mul_((torch.rand(shape[1:], generator=gen, device="cuda") < 0.9).float())
        s["budgets"] = torch.full((len(lens),), case["budget"], dtype=torch.int32, device="cuda")
        s.update(recent=case["recent"], width=max(lens), budget=case["budget"])
        s["before"] = {n: s[n].clone() for n in ("lens", "refs", "weights")}
    s.update(kind=kind, window=case.get("window", 0), sinks=case["sinks"])
    return s


# ---- plain forms ------------------------------------------------------------------------


def _softmax(s, seen):
    """p, lse (heads, rows packed) of scores (sequences, heads of keys, group, rows, keys) where only
    `seen` pairs exist; a row without any has p = 0, lse = -inf.  With `live`, of those rows alone."""
    live, seen = seen
    s = s.masked_fill_(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True).clamp_(min=-3.0e38)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    b, h, g, t = lse.shape
    return p.div_(total.clamp(min=1e-38)), lse.permute(0, 3, 1, 2).reshape(b, t, h * g)[live].t().contiguous()


def _blocks(s):
    """The sequences' rows in blocks of queries, and the places of the keys that each block may see: its
    window's, and the sinks.  (blocks, rows, heads, D) f32 queries' rows and (blocks, keys) keys' rows,
    with what exists and what is seen."""
    start, n = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    longest, w = s["longest"], min(s["window"], s["longest"])
    size = min(longest, 256)
    at = torch.arange(-(-longest // size) * size, device=n.device).view(-1, size)  # (blocks of a sequence, size)
    places = torch.cat([torch.arange(min(s["sinks"], longest), device=n.device).expand(at.shape[0], -1),
                        at[:, :1] - w + 1 + torch.arange(w + size - 1, device=n.device)], 1)
    window = torch.arange(places.shape[1], device=n.device) >= min(s["sinks"], longest)
    back = at[:, :, None] - places[:, None, :]
    seen = (back >= 0) & torch.where(window, (back < w) & (places[:, None, :] >= s["sinks"]), True)
    live, real = at[None] < n[:, None, None], (places[None] >= 0) & (places[None] < n[:, None, None])
    some = live[:, :, 0]  # blocks that hold a row
    seen = (seen[None] & live[..., None] & real[:, :, None])[some]
    rows = torch.where(live, start[:, None, None] + at[None], 0)[some]
    keys = torch.where(real, start[:, None, None] + places[None], 0)[some]
    return rows, live[some], keys, seen


def _plain_prompt(s):
    (_, hkv, d), hq = s["k"].shape, s["q"].shape[1]
    g = hq // hkv
    rows, live, keys, seen = _blocks(s)
    b, size = rows.shape
    q = s["q"][rows].float().view(b, size, hkv, g, d)
    k, v = s["k"][keys].float(), s["v"][keys].float()
    p, lse = _softmax(torch.einsum("bihgd,bjhd->bhgij", q, k) * d ** -0.5, (live, seen[:, None, None]))
    o = torch.einsum("bhgij,bjhd->bihgd", p, v)
    # (a block's rows that exist come in the order of the packed ones)
    packed_o = o.reshape(b, size, hq, d)[live].to(s["q"].dtype)
    if "do" not in s:
        return packed_o, lse
    do = torch.where(live[..., None, None], s["do"][rows].float(), 0.0).view(b, size, hkv, g, d)
    dv = torch.einsum("bhgij,bihgd->bjhd", p, do)
    dp = torch.einsum("bihgd,bjhd->bhgij", do, v)
    ds = p.mul_(dp.sub_((do * o).sum(-1).permute(0, 2, 3, 1)[..., None]))
    del dp
    dq = torch.einsum("bhgij,bjhd->bihgd", ds, k).reshape(b, size, hq, d) * d ** -0.5
    dk = torch.einsum("bhgij,bihgd->bjhd", ds, q) * d ** -0.5
    # a key's blocks added up
    dk, dv = (torch.zeros(s["k"].shape, device=k.device).index_add_(0, keys.flatten(), x.flatten(0, 1)) for x in (dk, dv))
    return packed_o, lse, dq[live].to(s["q"].dtype), dk.to(s["k"].dtype), dv.to(s["k"].dtype)


def _listed_places(s, live):
    """(sequences, new tokens, keys): whether a new token sees a cached place, without a window."""
    page = s["k"].shape[2]
    b, t = live.shape
    at = torch.arange(-(-s["width"] // page) * page, device=live.device)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    n = s["lens"][s["seqs"].long()].long()
    draft = at[None] - (n - new)[:, None]  # a key's place among the new tokens; negative: before them
    if s.get("mask") is None:
        seen = draft[:, None, :] <= torch.arange(t, device=at.device)[None, :, None]
    else:
        rows = torch.where(live, s["cu"][:-1].long()[:, None] + torch.arange(t, device=at.device)[None], 0)
        word = draft.clamp(0, 64 * s["mask"].shape[1] - 1)
        words = s["mask"][rows].gather(2, (word >> 6)[:, None, :].expand(b, t, -1))
        seen = (draft[:, None, :] < 0) | ((words >> (word & 63)[:, None, :]) & 1).bool()
    return seen & (at[None] < n[:, None])[:, None, :] & live[:, :, None]


def _cached_scores(s):
    """Scores of the new tokens over the cache, and (which of them exist, which pairs are seen)."""
    page, hkv, d = s["k"].shape[2:]
    start, new = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    at = torch.arange(s["longest"], device=new.device)
    live = at[None] < new[:, None]
    q = s["q"][torch.where(live, start[:, None] + at[None], 0)].float()
    b, t, hq, _ = q.shape
    held = s["table"][s["seqs"].long(), :-(-s["width"] // page)].long()
    k = s["k"][s.get("layer", 0)][held].reshape(b, -1, hkv, d).float()
    seen = _listed_places(s, live)
    if s["window"]:
        place = seen.cumsum(-1)  # in the list of what the token sees, from 1 on
        seen = seen & ((place > place[..., -1:] - s["window"]) | (place <= s["sinks"]))
    return torch.einsum("bihgd,bjhd->bhgij", q.view(b, t, hkv, hq // hkv, d), k) * d ** -0.5, (live, seen[:, None, None])


def _plain_tree(s):
    page, hkv, d = s["k"].shape[2:]
    scores, (live, seen) = _cached_scores(s)
    p, lse = _softmax(scores, (live, seen))
    held = s["table"][s["seqs"].long(), :-(-s["width"] // page)].long()
    v = s["v"][0][held].reshape(live.shape[0], -1, hkv, d).float()
    o = torch.einsum("bhgij,bjhd->bihgd", p, v).reshape(*live.shape, -1, d)
    return o[live].to(s["q"].dtype), lse


def _plain_weigh(s):
    scores, (live, seen) = _cached_scores(s)
    b, hkv, g, t, keys = scores.shape
    lse = torch.zeros(b, t, hkv * g, device=scores.device)
    lse[live] = s["lse"].t()
    p = scores.sub_(lse.view(b, t, hkv, g).permute(0, 2, 3, 1)[..., None]).exp_().masked_fill_(~seen, 0.0)
    got = p.sum((1, 2, 3))
    n, seqs = s["lens"][s["seqs"].long()].long(), s["seqs"].long()
    at = torch.arange(s["weights"].shape[2], device=n.device)[None]
    old = s["weights"][s["layer"]][seqs]
    base = torch.where(at < (n - s["fresh"].long())[:, None], old, 0.0)
    base[:, :keys] += got[:, :base.shape[1]]
    s["weights"][s["layer"], seqs] = torch.where(at < n[:, None], base, old)
    return s["weights"]


def _plain_evict(s):
    page = s["k"].shape[2]
    seqs, lens, refs, table = s["seqs"].long(), s["lens"], s["refs"], s["table"].long()
    n = lens[seqs].long()[:, None]
    at = torch.arange(s["width"], device=n.device)[None]
    total = s["weights"][:, seqs, :s["width"]].double().sum(0).float()
    # sinks and the last ones first of all, then by weight, the lowest place first among equals; none behind the end
    always = (at < s["sinks"]) | (at >= n - s["recent"])
    rank = torch.where(at < n, torch.where(always, float("inf"), total), float("-inf"))
    order = rank.sort(dim=1, descending=True, stable=True).indices
    after = torch.minimum(n, s["budgets"].long()[:, None])
    kept = torch.zeros(rank.shape, dtype=torch.bool, device=n.device).scatter_(1, order, at < after)
    # the kept ones' places, in order, and those that they go to
    i, source = kept.nonzero(as_tuple=True)
    to = (kept.cumsum(1) - 1)[i, source]
    from_page, to_page = table[seqs[i], source // page], table[seqs[i], to // page]
    for pool in (s["k"], s["v"]):
        pool[:, to_page, to % page] = pool[:, from_page, source % page]
    s["weights"][:, seqs[i], to] = s["weights"][:, seqs[i], source]
    slot = torch.arange(table.shape[1], device=n.device)[None]
    dropped = (slot * page >= after) & (slot * page < n) & (slot >= (after + page - 1) // page)
    refs.index_add_(0, torch.where(dropped, table[seqs], 0).reshape(-1), -dropped.reshape(-1).int())
    lens[seqs] = after[:, 0].int()
    return [s["table"], lens, refs, s["k"], s["v"], s["weights"]]


def run(state):
    s, kind = state, state["kind"]
    for name, x in s.get("before", {}).items():  # the cache as it was before the pass
        s[name].copy_(x)
    if not own:
        return {"prompt": _plain_prompt, "train": _plain_prompt, "tree": _plain_tree, "weigh": _plain_weigh,
                "evict": _plain_evict}[kind](s)

    import online_softmax_attention_gb300 as attn

    window = dict(window=s["window"] or None, sinks=s["sinks"])
    if kind in ("prompt", "train"):
        o, lse = attn.fwd(s["q"], s["k"], s["v"], causal=True, cu_seqlens_q=s["cu"], **window)
        if kind == "prompt":
            return o, lse
        return (o, lse) + attn.bwd(s["q"], s["k"], s["v"], o, lse, s["do"], causal=True, cu_seqlens_q=s["cu"], **window)
    cache = s["cache"]
    if kind == "tree":
        return attn.tree_fwd(s["q"], cache, s["seqs"], s["cu"], mask=s["mask"], **window)
    if kind == "weigh":
        cache.weigh(s["seqs"], s["cu"], s["q"], s["lse"], s["weights"], layer=s["layer"], fresh=s["fresh"], **window)
        return s["weights"]
    cache.evict(s["seqs"], s["budgets"], s["weights"], sinks=s["sinks"], recent=s["recent"])
    return [s["table"], s["lens"], s["refs"], s["k"], s["v"], s["weights"]]


# ---- 64 bits ----------------------------------------------------------------------------


def exact(case, seed):
    """The attention kinds from their definition, one sequence and head at a time, in f64."""
    kind = case["kind"]
    if kind == "evict":
        return None  # values are moved, not computed
    s = prepare(case, seed)
    lens, hq, group, d = _lens(case), case["hq"], case["hq"] // case["hkv"], case["d"]
    news = _news(case) if kind in ("tree", "weigh") else lens
    window, sinks = case["window"], case["sinks"]
    rows = sum(news)
    o = torch.zeros(rows, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(hq, rows, dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros(rows, h, d, dtype=torch.float64, device="cuda") for h in (hq, case["hkv"], case["hkv"]))
    weights = s["weights"].double() if kind == "weigh" else None
    at = 0
    for i, (n, t) in enumerate(zip(lens, news)):
        mine = slice(at, at + t)
        at += t
        if kind in ("tree", "weigh"):
            held = s["table"][int(s["seqs"][i]), :_pages(n, case["page"])].long()
            keys, values = (s[x][s.get("layer", 0)][held].flatten(0, 1)[:n].double() for x in ("k", "v"))
        else:
            keys, values = s["k"][mine].double(), s["v"][mine].double()
        seen = torch.ones(t, n, dtype=torch.bool, device="cuda").tril(n - t)
        if s.get("mask") is not None:
            bits = torch.arange(64, device="cuda")
            seen[:, n - t:] = ((s["mask"][mine][:, :, None] >> bits) & 1).flatten(1)[:, :t] == 1
            seen[:, :n - t] = True
        if window:
            nth = seen.long().cumsum(1)
            seen &= (nth <= sinks) | (nth > seen.sum(1, keepdim=True) - window)
        if kind == "weigh":
            j = int(s["seqs"][i])
            mass = torch.zeros(n, dtype=torch.float64, device="cuda")
            for h in range(hq):
                x = s["q"][mine, h].double() @ keys[:, h // group].T / d ** 0.5
                mass += (torch.exp(x - s["lse"][h, mine].double()[:, None]) * seen).sum(0)
            weights[s["layer"], j, n - int(s["fresh"][i]):n] = 0
            weights[s["layer"], j, :n] += mass
            continue
        for h in range(hq):
            q, k, v = s["q"][mine, h].double(), keys[:, h // group], values[:, h // group]
            x = (q @ k.T) / d ** 0.5
            x[~seen] = -torch.inf
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
    if kind == "weigh":
        return weights
    return (o, lse, dq, dk, dv) if kind == "train" else (o, lse)
