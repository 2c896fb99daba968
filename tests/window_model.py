"""What sliding windows with sinks, accumulated attention weights and eviction mean, in
plain Python and f64: the reference of their GPU tests."""
from __future__ import annotations

import numpy as np
import torch

from cache_model import attention


def windowed(seen, window, sinks):
    """Of the keys that each row of `seen` (T, L) sees, in order, the first `sinks` and the last `window`."""
    if window is None:
        return seen
    nth = np.cumsum(seen, 1)
    return seen & ((nth <= sinks) | (nth > nth[:, -1:] - window)) if seen.shape[1] else seen


def causal(n, window=None, sinks=0):
    return windowed(np.tril(np.ones((n, n), bool)), window, sinks)


def reference(x, lens, scale, window, sinks):
    """o, lse and sum p |v| of packed prompts."""
    parts = [[], [], []]
    at = 0
    for n in lens:
        m = slice(at, at + n)
        for p, y in zip(parts, attention(x["q"][m], x["k"][m], x["v"][m], causal(n, window, sinks), scale)):
            p.append(y)
        at += n
    return torch.cat(parts[0]), torch.cat(parts[1], 1), torch.cat(parts[2])


def gradients(x, lens, scale, window, sinks):
    """dq, dk, dv by autograd in f64 of the definition."""
    q, k, v = (x[n].double().requires_grad_() for n in "qkv")
    g = q.shape[1] // k.shape[1]
    kk, vv = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    at, loss = 0, 0.0
    for n in lens:
        m = slice(at, at + n)
        at += n
        s = torch.einsum("ihd,jhd->hij", q[m], kk[m]) * scale
        s = s.masked_fill(~torch.from_numpy(causal(n, window, sinks)), -torch.inf)
        loss = loss + (torch.einsum("hij,jhd->ihd", s.softmax(-1), vv[m]) * x["do"][m].double()).sum()
    loss.backward()
    return [t.grad.numpy() for t in (q, k, v)]


def weigh(q, k, lse, seen, scale):
    """(L,) f64: the attention that each key gets from the (T, H, D) query rows that see it."""
    q, k, lse = (torch.as_tensor(t).double() for t in (q, k, lse))
    k = k.repeat_interleave(q.shape[1] // k.shape[1], 1)
    p = (torch.einsum("thd,jhd->htj", q, k) * scale - lse[:, :, None]).exp()
    return p.masked_fill(~torch.as_tensor(seen)[None], 0.0).sum((0, 1)).numpy()


def kept(weights, n, budget, sinks, recent):
    """The tokens that a sequence of n keeps, in order; weights (layers, >= n) f32."""
    if n <= budget:
        return np.arange(n)
    w = weights[:, :n].astype(np.float64).sum(0).astype(np.float32)
    order = sorted(range(sinks, n - recent), key=lambda t: (bool(np.isnan(w[t])), -w[t] if w[t] == w[t] else 0.0, t))
    chosen = order[:budget - sinks - recent]
    return np.array(sorted([*range(sinks), *chosen, *range(n - recent, n)]), dtype=np.int64)


def evict(model, seqs, budgets, weights, sinks, recent):
    """The cache model and the weights (layers, sequences, tokens; changed) after an eviction."""
    for s, budget in zip(seqs, budgets):
        n = int(model.lens[s])
        if n <= budget:
            continue
        keep = kept(weights[:, s], n, budget, sinks, recent)
        for j, t in enumerate(keep):
            a, b = model.place(s, int(t)), model.place(s, j)
            model.k[(slice(None), *b)], model.v[(slice(None), *b)] = model.k[(slice(None), *a)], model.v[(slice(None), *a)]
            weights[:, s, j] = weights[:, s, t]
        model.lens[s] = budget
        model.release(s, model.pages(budget), model.pages(n))
