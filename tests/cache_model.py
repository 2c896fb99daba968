"""What the cache operations and attention over the cache mean, in plain Python
and f64: the reference of the GPU tests.  Also inputs and error bounds."""
from __future__ import annotations

import numpy as np
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


class Model:
    """A cache in numpy: the operations of ``attn_cache_*`` one entry at a time."""

    def __init__(self, k, v, table, lens, refs):
        self.k, self.v = np.array(k), np.array(v)
        self.table, self.lens, self.refs = (np.array(x) for x in (table, lens, refs))
        self.page = self.k.shape[2]

    def pages(self, n):
        return -(-int(n) // self.page)

    def alloc(self, n):
        return [int(p) for p in np.flatnonzero(self.refs == 0)[:n]]

    def extend(self, seqs, counts):
        cow = []
        free = iter(self.alloc(len(self.refs)))
        refs0 = self.refs.copy()
        for s, c in zip(seqs, counts):
            n, slot = int(self.lens[s]), self.pages(self.lens[s])
            if n % self.page and c and refs0[self.table[s, slot - 1]] > 1:
                old, new = self.table[s, slot - 1], next(free)
                cow.append((old, new, n % self.page))
                self.refs[old] -= 1
                self.refs[new] = 1
                self.table[s, slot - 1] = new
            for i in range(slot, self.pages(n + c)):
                self.table[s, i] = p = next(free)
                self.refs[p] = 1
            self.lens[s] += c
        for old, new, rows in cow:
            self.k[:, new, :rows], self.v[:, new, :rows] = self.k[:, old, :rows], self.v[:, old, :rows]

    def place(self, s, t):
        return int(self.table[s, t // self.page]), t % self.page

    def write(self, layer, seqs, cu, k, v):
        for i, s in enumerate(seqs):
            n = cu[i + 1] - cu[i]
            for x in range(n):
                p, r = self.place(s, int(self.lens[s]) - n + x)
                self.k[layer, p, r], self.v[layer, p, r] = k[cu[i] + x], v[cu[i] + x]

    def fork(self, parents, children):
        free = iter(self.alloc(len(self.refs)))
        for s, c in zip(parents, children):
            n = int(self.lens[s])
            full, tail = divmod(n, self.page)
            self.table[c, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.refs[p] += 1
            if tail:
                old, new = self.table[s, full], next(free)
                self.table[c, full] = new
                self.refs[new] = 1
                self.k[:, new, :tail], self.v[:, new, :tail] = self.k[:, old, :tail], self.v[:, old, :tail]
            self.lens[c] = n

    def release(self, s, first, last):
        for i in range(first, last):
            self.refs[self.table[s, i]] -= 1

    def keep(self, seqs, n_draft, keep, n_keep):
        for i, s in enumerate(seqs):
            old = int(self.lens[s])
            base = old - n_draft[i]
            for j in range(n_keep[i]):
                a, b = self.place(s, base + keep[i][j]), self.place(s, base + j)
                self.k[(slice(None), *b)], self.v[(slice(None), *b)] = self.k[(slice(None), *a)], self.v[(slice(None), *a)]
            self.lens[s] = base + n_keep[i]
            self.release(s, self.pages(self.lens[s]), self.pages(old))

    def free(self, seqs):
        for s in seqs:
            self.release(s, 0, self.pages(self.lens[s]))
            self.lens[s] = 0

    def compact(self):
        live = np.flatnonzero(self.refs > 0)
        movers = [p for p in live if p >= len(live)]
        holes = [p for p in range(len(live)) if self.refs[p] == 0]
        remap = np.arange(len(self.refs), dtype=np.int32)
        for a, b in zip(movers, holes):
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
            self.refs[b], self.refs[a], remap[a] = self.refs[a], 0, b
        for s in range(len(self.lens)):
            n = self.pages(self.lens[s])
            self.table[s, :n] = remap[self.table[s, :n]]
        return remap

    def rows(self, s, layer):
        """(k, v) rows of a sequence, (L, H, D)."""
        at = [self.place(s, t) for t in range(int(self.lens[s]))]
        p, r = [x[0] for x in at], [x[1] for x in at]
        return self.k[layer, p, r], self.v[layer, p, r]


def attention(q, k, v, seen, scale):
    """f64 attention of (T, H, D) queries over (L, Hkv, D) keys; seen (T, L) bool.
    Returns o, lse (H, T), and sum_j p_j |v_j|, by which rounding errors of p are bounded."""
    q, k, v = (torch.as_tensor(x).double() for x in (q, k, v))
    g = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("thd,jhd->htj", q, k) * scale
    s = s.masked_fill(~torch.as_tensor(seen)[None], -torch.inf)
    m = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full((*s.shape[:2], 1), -torch.inf, dtype=s.dtype)
    m = torch.where(torch.isinf(m), 0.0, m)
    e = (s - m).exp()
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    return (torch.einsum("htj,jhd->thd", p, v), (m + total.log())[..., 0],
            torch.einsum("htj,jhd->thd", p, v.abs()))


def check_output(o, lse, want, in_dtype, what=""):
    """O and lse against f64.  Per element, |o - ref| <= step_o |ref| + (step_p + c) sum p |v|:
    o is rounded once to its type; each p is rounded to the input type for the value
    contraction (f32 inputs: to the split's 2^-24 or not at all); c = 2^-12 covers the f32
    scores (their error times |p|: at most 128 products' f32 sums of N(0, 1) values, below
    1e-4 for the sizes here), 2^x to 2^-21 and the f32 sums.  For f32 inputs the library's
    1e-5 of absolute error holds.  lse: 1e-3, the library's."""
    ref, ref_lse, pv = want
    o, lse = o.double().cpu(), lse.double().cpu()
    step_p = 0.0 if in_dtype == torch.float32 else HALF_STEP[in_dtype]
    bound = HALF_STEP[torch.float32] * 4 + pv * (step_p + 2.0 ** -12)
    assert torch.isfinite(o).all(), f"{what}: O is not finite"
    return ref, ref_lse, o, lse, bound


def assert_output(o, lse, want, in_dtype, what=""):
    out_step = HALF_STEP[o.dtype]
    ref, ref_lse, o64, lse64, bound = check_output(o, lse, want, in_dtype, what)
    if in_dtype == torch.float32:
        bound = torch.full_like(bound, 1e-5)
    off = (o64 - ref).abs() - (bound + out_step * ref.abs())
    assert off.numel() == 0 or off.max() <= 0, f"{what}: O is {float(off.max()):.3e} over its bound"
    none = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse64), none), f"{what}: rows that see nothing differ"
    assert (lse64[none] == -torch.inf).all()
    assert none.all() or (lse64 - ref_lse)[~none].abs().max() <= 1e-3, f"{what}: lse"


def seen_tree(n, t, mask_rows=None):
    """(T, L) visibility: everything before the T last tokens; of those, mask bits or u <= t."""
    seen = np.zeros((t, n), bool)
    seen[:, :n - t] = True
    for i in range(t):
        for u in range(t):
            seen[i, n - t + u] = u <= i if mask_rows is None else bool(int(mask_rows[i][u >> 6]) >> (u & 63) & 1)
    return seen
