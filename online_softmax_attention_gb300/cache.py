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


class TreeCall:
    """Prepared attention of new tokens over a cache: holds the argument struct,
    outputs and workspace.  Lengths and tables are read when it runs.  It has to live
    until its runs are done, and as long as a graph that captured one.

    ``mask`` (n_q, words) int64: bit u of row t (bit u % 64 of word u // 64) lets
    new token t see new token u; without it a new token sees those up to itself.
    """

    def __init__(self, q: torch.Tensor, cache: Cache, seqs, cu_seqlens_q, *, layer: int = 0,
                 mask: torch.Tensor | None = None, scale: float | None = None,
                 out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
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
        if workspace is None:
            # (0 bytes: arguments that the call will refuse)
            workspace = torch.empty(_host.call(dev.index, _host.entry("attn_tree_workspace_bytes"), None, _host.TREE.pack(*head, 0, 0)) or 256,
                                    dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on the cache's device {dev}")
        self.workspace = workspace
        self.args = _host.TREE.pack(*head, workspace.data_ptr(), workspace.numel() * workspace.element_size())

    def run(self, stream: torch.cuda.Stream | None = None):
        index = self.cache.device.index
        s = _host.raw_stream(index) if stream is None else stream.cuda_stream
        _host.call(index, _host.entry("attn_tree_fwd"), "attn_tree_fwd", self.args, s)
        return self.o, self.lse


def tree_fwd(q, cache: Cache, seqs, cu_seqlens_q, *, layer: int = 0, mask: torch.Tensor | None = None,
             scale: float | None = None, out_dtype: torch.dtype | None = None):
    """Attention of new tokens over the cache.  Returns ``(o, lse)``; lse is (H, T) f32, natural log.

    Rows ``cu[i]:cu[i + 1]`` of q are the last tokens of sequence ``seqs[i]``: one token
    (decoding), a chunk, or with ``mask`` a tree of drafts (see ``TreeCall``)."""
    r = _host.native().tree(cache.args, cache._index, q, seqs, cu_seqlens_q, mask, layer, scale,
                            -1 if out_dtype is None else _DT.get(out_dtype, 99))
    if r is None:
        return TreeCall(q, cache, seqs, cu_seqlens_q, layer=layer, mask=mask, scale=scale, out_dtype=out_dtype).run()
    return r if type(r) is tuple else _abi.check(r, "attn_tree_fwd")
