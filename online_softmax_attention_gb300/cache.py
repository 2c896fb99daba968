"""The paged key / value cache and attention over it (argument marshalling only;
every step runs in the CUDA library, see ``attn_cache`` in ``include/attn.h``).

A ``Cache`` is a view of the caller's tensors: the pools ``k`` and ``v``
(layers, pages, page_size, heads, D), the page ``table`` (sequences, pages a
sequence can hold), the sequences' ``lens`` and the pages' reference counts
``refs`` (0 = free), the last three int32.  The operations change those tensors
on the current stream without synchronising, so a captured loop can hold them
(it needs those tensors, not the ``Cache``); what a list gets wrong is reported by
``device_status()`` and changes nothing (``write`` and ``free`` do the other entries).

    cache = Cache.empty(layers, pages, page_size, heads, D, max_seqs=64, max_pages=256)
    o, lse = fwd(q, k, v, causal=True, cu_seqlens_q=cu)       # the prompts
    cache.extend(seqs, lengths)                               # their room
    cache.write(seqs, cu, k, v, layer=0)                      # their rows
    cache.extend(seqs, ones); cache.write(seqs, cu1, k1, v1)  # a new token each
    o1, lse1 = tree_fwd(q1, cache, seqs, cu1)                 # over the cache

A cache that stays within a budget: ``weights = cache.new_weights()``; after each
``tree_fwd``, ``cache.weigh(seqs, cu1, q1, lse1, weights)`` adds the attention that every cached
token got; ``cache.evict(seqs, budgets, weights)`` keeps the heaviest.  The weights are the
caller's: after ``fork`` copy the parents' rows to the children's, weigh drafted tokens
after ``keep``, and start a sequence anew with ``fresh``.
"""
from __future__ import annotations

import torch

from . import _abi, _host

_DT = {torch.float16: _abi.ATTN_F16, torch.bfloat16: _abi.ATTN_BF16, torch.float32: _abi.ATTN_F32}


def _ints(x, device: torch.device, name: str) -> torch.Tensor:
    """A list argument as a contiguous int32 vector on the cache's device."""
    if isinstance(x, torch.Tensor) and x.dtype == torch.int32 and x.device == device and x.dim() == 1 \
            and x.is_contiguous():
        return x
    x = torch.as_tensor(x, dtype=torch.int32 if isinstance(x, (list, tuple)) and not x else None)
    if x.dim() != 1 or x.is_floating_point() or x.dtype == torch.bool:
        raise ValueError(f"{name} must be a vector of whole numbers")
    return _host.int32(x, device, name)


def _rows(t: torch.Tensor, name: str, heads: int | None, D: int, dtype: torch.dtype, device) -> tuple[int, int, int]:
    """Address, token stride and head stride of a (tokens, heads, D) tensor."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != D or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be (tokens, {heads if heads is not None else 'heads'}, {D}), got {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on the cache's device {device}, got {t.device}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the D axis must be contiguous")
    # a size-1 axis is never stepped along, so any aligned stride describes it
    return t.data_ptr(), st if shape[0] > 1 else shape[1] * D, sh if shape[1] > 1 else D


class Cache:
    """A paged key / value cache over the caller's tensors."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor):
        if k.dim() != 5 or v.shape != k.shape or v.stride() != k.stride():
            raise ValueError("k and v must be (layers, pages, page_size, heads, D) with the same strides, got "
                             f"{tuple(k.shape)} and {tuple(v.shape)}")
        if k.dtype not in _DT or v.dtype != k.dtype:
            raise TypeError("k and v must share one of float16, bfloat16, float32")
        dev = k.device
        if not k.is_cuda or any(t.device != dev for t in (v, table, lens, refs)):
            raise ValueError("k, v, table, lens and refs must be on one CUDA device")
        if any(t.dtype != torch.int32 for t in (table, lens, refs)):
            raise TypeError("table, lens and refs must be int32")
        if table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1) or lens.shape != table.shape[:1] \
                or refs.shape != k.shape[1:2] or not lens.is_contiguous() or not refs.is_contiguous():
            raise ValueError("table must be (sequences, pages) with contiguous rows, lens (sequences,) and refs (pages,)")
        if k.stride(4) != 1:
            raise ValueError("k, v: the D axis must be contiguous")
        self.k, self.v, self.table, self.lens, self.refs = k, v, table, lens, refs
        self.device = dev
        self._index = dev.index
        self._native = _host.native()
        shape, self.dtype = k.shape, k.dtype
        self.n_layers, _, _, self.n_heads, self.head_dim = shape
        self.max_seqs = table.shape[0]
        # a size-1 axis is never stepped along: give it the stride of a contiguous layout
        dense = (shape[1] * shape[2] * shape[3] * shape[4], shape[2] * shape[3] * shape[4], shape[3] * shape[4], shape[4])
        self.args = _host.CACHE.pack(
            k.data_ptr(), v.data_ptr(), *(k.stride(i) if shape[i] > 1 else dense[i] for i in range(4)),
            table.data_ptr(), lens.data_ptr(), refs.data_ptr(),
            table.stride(0) if table.shape[0] > 1 else table.shape[1], shape[0], shape[1], shape[2], shape[3], shape[4],
            _DT[k.dtype], table.shape[0], table.shape[1])
        need = _host.entry("attn_cache_workspace_bytes")
        if need(self.args, 0) == 0:
            raise ValueError("unsupported cache: page_size a power of two up to 1024, D 64 or 128, "
                             "16-byte aligned rows")

    @classmethod
    def empty(cls, n_layers: int, n_pages: int, page_size: int, n_heads: int, head_dim: int, *, max_seqs: int,
              max_pages: int, dtype: torch.dtype = torch.bfloat16, device="cuda") -> "Cache":
        """A cache of its own memory, every page free and every sequence empty."""
        dev = torch.device(device)
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        k, v = (torch.zeros((n_layers, n_pages, page_size, n_heads, head_dim), dtype=dtype, device=dev) for _ in range(2))
        table = torch.zeros((max_seqs, max_pages), dtype=torch.int32, device=dev)
        return cls(k, v, table, torch.zeros(max_seqs, dtype=torch.int32, device=dev),
                   torch.zeros(n_pages, dtype=torch.int32, device=dev))

    def _workspace(self, n: int) -> torch.Tensor:
        """Scratch of one call with a list of n entries, from the stream that the call runs on (or
        the graph that captures it), so that it lives as long as the call needs it."""
        need = _host.entry("attn_cache_workspace_bytes")
        return torch.empty(need(self.args, n), dtype=torch.uint8, device=self.device)

    def _done(self, name: str, rc: int | None) -> bool:
        """Whether the compiled binding made the call; an error becomes an exception."""
        if rc:
            _abi.check(rc, name)
        return rc is not None

    def _call(self, name: str, *args) -> None:
        index = self.device.index
        _host.call(index, _host.entry(name), name, self.args, *args, _host.raw_stream(index))

    def _call_packed(self, name: str, args: bytes) -> None:
        index = self.device.index
        _host.call(index, _host.entry(name), name, args, _host.raw_stream(index))

    def _lists(self, n: int | None, **lists) -> list:
        out = [_ints(x, self.device, name) for name, x in lists.items()]
        n = out[0].numel() if n is None else n
        for name, x in zip(lists, out):
            if x.numel() != n:
                raise ValueError(f"{name} must have {n} entries, got {x.numel()}")
        return out

    def extend(self, seqs, counts) -> None:
        """Room for ``counts[i]`` more tokens of sequence ``seqs[i]``: pages and lengths."""
        if self._done("attn_cache_extend", self._native.extend(self.args, self._index, seqs, counts)):
            return
        seqs, counts = self._lists(None, seqs=seqs, counts=counts)
        ws = self._workspace(seqs.numel())
        self._call("attn_cache_extend", seqs.data_ptr(), counts.data_ptr(), seqs.numel(), ws.data_ptr(), ws.numel())

    def write(self, seqs, cu_seqlens, k: torch.Tensor, v: torch.Tensor, *, layer: int = 0) -> None:
        """New rows (tokens, heads, D) of one layer: rows ``cu[i]:cu[i + 1]`` become the
        last tokens of sequence ``seqs[i]`` (``extend`` made their room)."""
        if self._done("attn_cache_write", self._native.write(self.args, self._index, seqs, cu_seqlens, k, v, layer)):
            return
        seqs = _ints(seqs, self.device, "seqs")
        cu = _ints(cu_seqlens, self.device, "cu_seqlens")
        if cu.numel() != seqs.numel() + 1:
            raise ValueError(f"cu_seqlens must have {seqs.numel() + 1} entries, got {cu.numel()}")
        kt = _host.VIEW.pack(*_rows(k, "k", self.n_heads, self.head_dim, self.dtype, self.device))
        vt = _host.VIEW.pack(*_rows(v, "v", self.n_heads, self.head_dim, self.dtype, self.device))
        if k.shape[0] != v.shape[0]:
            raise ValueError("k and v must have as many tokens as each other")
        self._call("attn_cache_write", int(layer), seqs.data_ptr(), cu.data_ptr(), seqs.numel(), kt, vt, k.shape[0])

    def fork(self, parents, children) -> None:
        """The empty sequence ``children[i]`` becomes a copy of ``parents[i]`` that shares its full pages."""
        if self._done("attn_cache_fork", self._native.fork(self.args, self._index, parents, children)):
            return
        parents, children = self._lists(None, parents=parents, children=children)
        ws = self._workspace(parents.numel())
        self._call("attn_cache_fork", parents.data_ptr(), children.data_ptr(), parents.numel(), ws.data_ptr(), ws.numel())

    def keep(self, seqs, n_draft, keep: torch.Tensor, n_keep) -> None:
        """Of the last ``n_draft[i]`` tokens of ``seqs[i]`` keeps the ``n_keep[i]`` at the
        ascending offsets ``keep[i, :n_keep[i]]``; the others go."""
        if self._done("attn_cache_keep", self._native.keep(self.args, self._index, seqs, n_draft, keep, n_keep)):
            return
        seqs, n_draft, n_keep = self._lists(None, seqs=seqs, n_draft=n_draft, n_keep=n_keep)
        if not isinstance(keep, torch.Tensor):
            keep = torch.as_tensor(keep)
        if keep.dim() != 2 or keep.shape[0] != seqs.numel() or keep.is_floating_point() or keep.dtype == torch.bool:
            raise ValueError(f"keep must be ({seqs.numel()}, offsets) whole numbers, got {tuple(keep.shape)}")
        keep = _host.int32(keep, self.device, "keep")
        ws = self._workspace(seqs.numel())
        self._call("attn_cache_keep", seqs.data_ptr(), n_draft.data_ptr(), keep.data_ptr(), keep.shape[1],
                   n_keep.data_ptr(), seqs.numel(), ws.data_ptr(), ws.numel())

    def free(self, seqs) -> None:
        """Empties the sequences; pages that no other sequence holds are free again."""
        if self._done("attn_cache_free", self._native.free(self.args, self._index, seqs)):
            return
        seqs = _ints(seqs, self.device, "seqs")
        self._call("attn_cache_free", seqs.data_ptr(), seqs.numel())

    def compact(self, *, remap: torch.Tensor | None = None) -> None:
        """Moves the live pages to the front of the pool.  ``remap`` (pages,) int32 gets every page's new index."""
        if remap is not None and (remap.dtype != torch.int32 or remap.device != self.device or
                                  remap.shape != self.refs.shape or not remap.is_contiguous()):
            raise ValueError("remap must be a contiguous int32 vector of one entry per page on the cache's device")
        ws = self._workspace(0)
        self._call("attn_cache_compact", remap.data_ptr() if remap is not None else None, ws.data_ptr(),
                   ws.numel())

    def new_weights(self, n_layers: int | None = None) -> torch.Tensor:
        """Weights of 0 for ``weigh`` and ``evict``: (layers, sequences, tokens a sequence can hold) float32."""
        return torch.zeros((n_layers or self.n_layers, self.max_seqs, self.table.shape[1] * self.k.shape[2]),
                           dtype=torch.float32, device=self.device)

    def _weights(self, weights: torch.Tensor) -> torch.Tensor:
        if weights.dim() != 3 or weights.dtype != torch.float32 or weights.device != self.device \
                or weights.shape[0] < 1 or weights.shape[1] != self.max_seqs or (weights.shape[2] > 1 and weights.stride(2) != 1) \
                or weights.stride(0) < 0 or (self.max_seqs > 1 and weights.stride(1) < weights.shape[2]) \
                or (weights.shape[0] > 1 and weights.stride(0) < weights.stride(1) * (self.max_seqs - 1) + weights.shape[2]):
            raise ValueError(f"weights must be float32 (layers, {self.max_seqs}, tokens) with rows of their own on the "
                             f"cache's device {self.device}, got {weights.dtype} {tuple(weights.shape)}")
        return weights

    def weigh(self, seqs, cu_seqlens_q, q: torch.Tensor, lse: torch.Tensor, weights: torch.Tensor, *, layer: int = 0,
              scale: float | None = None, window: int | None = None, sinks: int = 0, fresh=None) -> None:
        """Adds to ``weights[layer, seqs[i], j]`` the attention that token j of sequence ``seqs[i]``
        gets from the query rows ``cu[i]:cu[i + 1]`` of q, summed over rows and heads.

        The arguments are those of ``tree_fwd`` (without a mask), ``lse`` what it returned.  The
        last ``fresh[i]`` tokens' weights start anew (None: the new tokens', ``cu[i + 1] - cu[i]``)."""
        if self._done("attn_cache_weigh", self._native.weigh(self.args, self._index, seqs, cu_seqlens_q, q, lse, weights, layer,
                                                             scale, window, sinks, fresh)):
            return
        dev, D = self.device, self.head_dim
        seqs, cu = _ints(seqs, dev, "seqs"), _ints(cu_seqlens_q, dev, "cu_seqlens_q")
        n = seqs.numel()
        if cu.numel() != n + 1:
            raise ValueError(f"cu_seqlens_q must have {n + 1} entries, got {cu.numel()}")
        if fresh is not None:
            fresh, = self._lists(n, fresh=fresh)
        w = self._weights(weights)
        if not 0 <= int(layer) < min(self.n_layers, w.shape[0]):
            raise ValueError(f"layer must be one of {min(self.n_layers, w.shape[0])}, got {layer}")
        q_fields = _rows(q, "q", None, D, self.dtype, dev)
        T, H, _ = q.shape
        if tuple(lse.shape) != (H, T) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != dev:
            raise ValueError(f"lse must be contiguous float32 {(H, T)} on the cache's device")
        head = (self.args, int(layer), H, *q_fields, lse.data_ptr(), w[int(layer)].data_ptr(),
                w.stride(1) if self.max_seqs > 1 else w.shape[2], w.shape[2], n, T,
                _host.f32(scale) if scale is not None else D ** -0.5, *_host.window(window, sinks), seqs.data_ptr(),
                cu.data_ptr(), fresh.data_ptr() if fresh is not None else 0)
        need = _host.call(dev.index, _host.entry("attn_weigh_workspace_bytes"), None, _host.WEIGH.pack(*head, 0, 0))
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        self._call_packed("attn_cache_weigh", _host.WEIGH.pack(*head, ws.data_ptr() if need else 0, need))

    def evict(self, seqs, budgets, weights: torch.Tensor, *, sinks: int = 0, recent: int = 0) -> None:
        """Cuts every sequence ``seqs[i]`` of more than ``budgets[i]`` tokens to that many: the first
        ``sinks``, the last ``recent`` and the heaviest others by ``weights`` summed over its
        layers (equal ones: the first).  Rows and weights move down; a whole list or nothing."""
        if self._done("attn_cache_evict", self._native.evict(self.args, self._index, seqs, budgets, weights, sinks, recent)):
            return
        seqs, budgets = self._lists(None, seqs=seqs, budgets=budgets)
        w = self._weights(weights)
        for x, name in ((sinks, "sinks"), (recent, "recent")):
            if not isinstance(x, int) or isinstance(x, bool) or not 0 <= x < 2 ** 31:
                raise ValueError(f"{name} must be a whole number, 0 or more, got {x!r}")
        packed = _host.WEIGHTS.pack(w.data_ptr(), w.stride(0) if w.shape[0] > 1 else w.shape[1] * w.shape[2],
                                    w.stride(1) if self.max_seqs > 1 else w.shape[2], w.shape[0], w.shape[2])
        n = seqs.numel()
        ws = torch.empty(_host.entry("attn_cache_evict_workspace_bytes")(self.args, n, w.shape[2]), dtype=torch.uint8,
                         device=self.device)
        self._call("attn_cache_evict", seqs.data_ptr(), budgets.data_ptr(), n, packed, sinks, recent, ws.data_ptr(),
                   ws.numel())


class TreeCall:
    """Prepared attention of new tokens over a cache: holds the argument struct,
    outputs and workspace.  Lengths and tables are read when it runs.  It has to live
    until its runs are done, and as long as a graph that captured one.

    ``mask`` (n_q, words) int64: bit u of row t (bit u % 64 of word u // 64) lets
    new token t see new token u; without it a new token sees those up to itself.
    ``window``: of what a new token would see so, it sees the first ``sinks`` tokens and the
    last ``window`` (None: all).
    """

    def __init__(self, q: torch.Tensor, cache: Cache, seqs, cu_seqlens_q, *, layer: int = 0,
                 mask: torch.Tensor | None = None, scale: float | None = None,
                 out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 window: int | None = None, sinks: int = 0):
        dev, D, dtype = cache.device, cache.head_dim, cache.dtype
        self.cache = cache
        self.seqs = seqs = _ints(seqs, dev, "seqs")
        self.cu = cu = _ints(cu_seqlens_q, dev, "cu_seqlens_q")
        n = seqs.numel()
        if cu.numel() != n + 1:
            raise ValueError(f"cu_seqlens_q must have {n + 1} entries, got {cu.numel()}")
        q_fields = _rows(q, "q", None, D, dtype, dev)
        T, H, _ = shape = q.shape
        if out is None:
            out_dtype = out_dtype or dtype
            out = torch.empty(shape, dtype=out_dtype, device=dev)
        else:
            out_dtype = out.dtype
            if out.shape != shape:
                raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
        if out_dtype != dtype and out_dtype != torch.float32:
            raise TypeError(f"the output is {dtype} or float32, not {out_dtype}")
        if lse is None:
            lse = torch.empty((H, T), dtype=torch.float32, device=dev)
        elif tuple(lse.shape) != (H, T) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != dev:
            raise ValueError(f"lse must be contiguous float32 {(H, T)} on the cache's device")
        words = 0
        if mask is not None:
            if mask.dtype != torch.int64 or mask.dim() != 2 or mask.shape[0] != T or mask.shape[1] < 1 \
                    or not mask.is_contiguous() or mask.device != dev:
                raise ValueError(f"mask must be contiguous int64 ({T}, words) on the cache's device")
            words = mask.shape[1]
        self.o, self.lse, self.inputs = out, lse, (q, mask)
        head = (cache.args, int(layer), H, *q_fields, *_rows(out, "out", H, D, out_dtype, dev), lse.data_ptr(),
                seqs.data_ptr(), cu.data_ptr(), mask.data_ptr() if mask is not None else 0, n, T, words,
                _host.f32(scale) if scale is not None else D ** -0.5, _DT[out_dtype])
        window = _host.window(window, sinks)
        if workspace is None:
            # (0 bytes: arguments that the call will refuse)
            workspace = torch.empty(_host.call(dev.index, _host.entry("attn_tree_workspace_bytes"), None, _host.TREE.pack(*head, 0, 0, *window)) or 256,
                                    dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on the cache's device {dev}")
        self.workspace = workspace
        self.args = _host.TREE.pack(*head, workspace.data_ptr(), workspace.numel() * workspace.element_size(), *window)

    def run(self, stream: torch.cuda.Stream | None = None):
        index = self.cache.device.index
        s = _host.raw_stream(index) if stream is None else stream.cuda_stream
        _host.call(index, _host.entry("attn_tree_fwd"), "attn_tree_fwd", self.args, s)
        return self.o, self.lse


def tree_fwd(q, cache: Cache, seqs, cu_seqlens_q, *, layer: int = 0, mask: torch.Tensor | None = None,
             scale: float | None = None, out_dtype: torch.dtype | None = None, window: int | None = None, sinks: int = 0):
    """Attention of new tokens over the cache.  Returns ``(o, lse)``; lse is (H, T) f32, natural log.

    Rows ``cu[i]:cu[i + 1]`` of q are the last tokens of sequence ``seqs[i]``: one token
    (decoding), a chunk, or with ``mask`` a tree of drafts; ``window`` and ``sinks`` bound what
    they see (see ``TreeCall``)."""
    r = _host.native().tree(cache.args, cache._index, q, seqs, cu_seqlens_q, mask, layer, scale,
                            -1 if out_dtype is None else _DT.get(out_dtype, 99), window, sinks)
    if r is None:
        return TreeCall(q, cache, seqs, cu_seqlens_q, layer=layer, mask=mask, scale=scale, out_dtype=out_dtype,
                        window=window, sinks=sinks).run()
    return r if type(r) is tuple else _abi.check(r, "attn_tree_fwd")
