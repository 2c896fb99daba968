"""The paged key / value cache and attention over it (argument marshalling only;
every step runs in the CUDA library, see ``attn_cache`` in ``include/attn.h``).

A ``Cache`` is a view of the caller's tensors: the pools ``k`` and ``v``
(layers, pages, page_size, heads, D), the page ``table`` (sequences, pages a
sequence can hold), the sequences' ``lens`` and the pages' reference counts
``refs`` (0 = free), the last three int32.  The operations change those tensors
on the current stream without synchronising, so a captured loop can hold them;
what a list gets wrong is reported by ``device_status()`` and changes nothing.

    cache = Cache.empty(layers, pages, page_size, heads, D, max_seqs=64, max_pages=256)
    o, lse = fwd(q, k, v, causal=True, cu_seqlens_q=cu)       # the prompts
    cache.extend(seqs, lengths)                               # their room
    cache.write(seqs, cu, k, v, layer=0)                      # their rows
    cache.extend(seqs, ones); cache.write(seqs, cu1, k1, v1)  # a new token each
    o1, lse1 = tree_fwd(q1, cache, seqs, cu1)                 # over the cache
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi

_DT = {torch.float16: _abi.ATTN_F16, torch.bfloat16: _abi.ATTN_BF16, torch.float32: _abi.ATTN_F32}


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


class _on:
    """Makes `device` current for a call when another one is."""

    __slots__ = ("guard",)

    def __init__(self, device: torch.device):
        self.guard = torch.cuda.device(device) if device.index != torch.cuda.current_device() else None

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _ints(x, device: torch.device, name: str) -> torch.Tensor:
    """A list argument as a contiguous int32 vector on the cache's device."""
    if isinstance(x, torch.Tensor) and x.dtype == torch.int32 and x.device == device and x.dim() == 1 \
            and x.is_contiguous():
        return x
    x = torch.as_tensor(x, dtype=torch.int32 if isinstance(x, (list, tuple)) and not x else None)
    if x.dim() != 1 or x.is_floating_point() or x.dtype == torch.bool:
        raise ValueError(f"{name} must be a vector of whole numbers")
    if not x.is_cuda and x.numel() and not -2 ** 31 <= int(x.min()) <= int(x.max()) < 2 ** 31:
        raise ValueError(f"{name}: entries must fit 32 bits")
    return x.to(device=device, dtype=torch.int32).contiguous()


def _rows(t: torch.Tensor, name: str, heads: int | None, D: int, dtype: torch.dtype, device) -> _abi.AttnTensor:
    """A (tokens, heads, D) view for the library."""
    if t.dim() != 3 or t.shape[2] != D or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be (tokens, {heads if heads is not None else 'heads'}, {D}), got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on the cache's device {device}, got {t.device}")
    if t.stride(2) != 1:
        raise ValueError(f"{name}: the D axis must be contiguous")
    # a size-1 axis is never stepped along, so any aligned stride describes it
    return _abi.AttnTensor(t.data_ptr() if t.numel() else None, t.stride(0) if t.shape[0] > 1 else t.shape[1] * D,
                           t.stride(1) if t.shape[1] > 1 else D)


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
        c = _abi.Cache()
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.n_layers, c.n_pages, c.page_size, c.H_kv, c.D = k.shape
        # a size-1 axis is never stepped along: give it the stride of a contiguous layout
        dense = [c.n_pages * c.page_size * c.H_kv * c.D, c.page_size * c.H_kv * c.D, c.H_kv * c.D, c.D]
        st = [k.stride(i) if k.shape[i] > 1 else dense[i] for i in range(4)]
        c.stride_layer, c.stride_page, c.stride_tok, c.stride_head = st
        c.table, c.lens, c.refs = table.data_ptr(), lens.data_ptr(), refs.data_ptr()
        c.max_seqs, c.max_pages = table.shape
        c.table_stride = table.stride(0) if table.shape[0] > 1 else table.shape[1]
        c.dtype = _DT[k.dtype]
        self.args = c
        self._ref = ctypes.byref(c)
        self._lib = _abi.load()
        if self._lib.attn_cache_workspace_bytes(self._ref, 0) == 0:
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
        # torch's caching allocator returns 512-byte aligned blocks
        return torch.empty(self._lib.attn_cache_workspace_bytes(self._ref, n), dtype=torch.uint8, device=self.device)

    def _lists(self, n: int | None, **lists) -> list:
        out = [_ints(x, self.device, name) for name, x in lists.items()]
        n = out[0].numel() if n is None else n
        for name, x in zip(lists, out):
            if x.numel() != n:
                raise ValueError(f"{name} must have {n} entries, got {x.numel()}")
        return out

    def extend(self, seqs, counts) -> None:
        """Room for ``counts[i]`` more tokens of sequence ``seqs[i]``: pages and lengths."""
        seqs, counts = self._lists(None, seqs=seqs, counts=counts)
        ws = self._workspace(seqs.numel())
        with _on(self.device):
            _abi.check(self._lib.attn_cache_extend(self._ref, seqs.data_ptr(), counts.data_ptr(), seqs.numel(),
                                                   ws.data_ptr(), ws.numel(), _stream(self.device)), "attn_cache_extend")

    def write(self, seqs, cu_seqlens, k: torch.Tensor, v: torch.Tensor, *, layer: int = 0) -> None:
        """New rows (tokens, heads, D) of one layer: rows ``cu[i]:cu[i + 1]`` become the
        last tokens of sequence ``seqs[i]`` (``extend`` made their room)."""
        c = self.args
        seqs = _ints(seqs, self.device, "seqs")
        cu = _ints(cu_seqlens, self.device, "cu_seqlens")
        if cu.numel() != seqs.numel() + 1:
            raise ValueError(f"cu_seqlens must have {seqs.numel() + 1} entries, got {cu.numel()}")
        kt = _rows(k, "k", c.H_kv, c.D, self.k.dtype, self.device)
        vt = _rows(v, "v", c.H_kv, c.D, self.k.dtype, self.device)
        if k.shape[0] != v.shape[0]:
            raise ValueError("k and v must have as many tokens as each other")
        with _on(self.device):
            _abi.check(self._lib.attn_cache_write(self._ref, int(layer), seqs.data_ptr(), cu.data_ptr(), seqs.numel(),
                                                  ctypes.byref(kt), ctypes.byref(vt), k.shape[0],
                                                  _stream(self.device)), "attn_cache_write")

    def fork(self, parents, children) -> None:
        """The empty sequence ``children[i]`` becomes a copy of ``parents[i]`` that shares its full pages."""
        parents, children = self._lists(None, parents=parents, children=children)
        ws = self._workspace(parents.numel())
        with _on(self.device):
            _abi.check(self._lib.attn_cache_fork(self._ref, parents.data_ptr(), children.data_ptr(), parents.numel(),
                                                 ws.data_ptr(), ws.numel(), _stream(self.device)), "attn_cache_fork")

    def keep(self, seqs, n_draft, keep: torch.Tensor, n_keep) -> None:
        """Of the last ``n_draft[i]`` tokens of ``seqs[i]`` keeps the ``n_keep[i]`` at the
        ascending offsets ``keep[i, :n_keep[i]]``; the others go."""
        seqs, n_draft, n_keep = self._lists(None, seqs=seqs, n_draft=n_draft, n_keep=n_keep)
        keep = torch.as_tensor(keep)
        if keep.dim() != 2 or keep.shape[0] != seqs.numel() or keep.is_floating_point() or keep.dtype == torch.bool:
            raise ValueError(f"keep must be ({seqs.numel()}, offsets) whole numbers, got {tuple(keep.shape)}")
        keep = keep.to(device=self.device, dtype=torch.int32).contiguous()
        ws = self._workspace(seqs.numel())
        with _on(self.device):
            _abi.check(self._lib.attn_cache_keep(self._ref, seqs.data_ptr(), n_draft.data_ptr(),
                                                 keep.data_ptr() if keep.numel() else None, keep.shape[1],
                                                 n_keep.data_ptr(), seqs.numel(), ws.data_ptr(), ws.numel(),
                                                 _stream(self.device)), "attn_cache_keep")

    def free(self, seqs) -> None:
        """Empties the sequences; pages that no other sequence holds are free again."""
        seqs = _ints(seqs, self.device, "seqs")
        with _on(self.device):
            _abi.check(self._lib.attn_cache_free(self._ref, seqs.data_ptr(), seqs.numel(), _stream(self.device)),
                       "attn_cache_free")

    def compact(self, *, remap: torch.Tensor | None = None) -> None:
        """Moves the live pages to the front of the pool.  ``remap`` (pages,) int32 gets every page's new index."""
        if remap is not None and (remap.dtype != torch.int32 or remap.device != self.device or
                                  remap.shape != self.refs.shape or not remap.is_contiguous()):
            raise ValueError("remap must be a contiguous int32 vector of one entry per page on the cache's device")
        ws = self._workspace(0)
        with _on(self.device):
            _abi.check(self._lib.attn_cache_compact(self._ref, remap.data_ptr() if remap is not None else None,
                                                    ws.data_ptr(), ws.numel(), _stream(self.device)),
                       "attn_cache_compact")


class TreeCall:
    """Prepared attention of new tokens over a cache: holds the argument struct,
    outputs and workspace.  Lengths and tables are read when it runs.

    ``mask`` (n_q, words) int64: bit u of row t (bit u % 64 of word u // 64) lets
    new token t see new token u; without it a new token sees those up to itself.
    """

    def __init__(self, q: torch.Tensor, cache: Cache, seqs, cu_seqlens_q, *, layer: int = 0,
                 mask: torch.Tensor | None = None, scale: float | None = None,
                 out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
        c, dev = cache.args, cache.device
        self.cache = cache
        self.seqs = _ints(seqs, dev, "seqs")
        self.cu = _ints(cu_seqlens_q, dev, "cu_seqlens_q")
        if self.cu.numel() != self.seqs.numel() + 1:
            raise ValueError(f"cu_seqlens_q must have {self.seqs.numel() + 1} entries, got {self.cu.numel()}")
        a = _abi.TreeArgs()
        a.cache = c
        a.q = _rows(q, "q", None, c.D, cache.k.dtype, dev)
        T, H = q.shape[:2]
        out_dtype = out.dtype if out is not None else out_dtype or q.dtype
        if out_dtype not in _DT:
            raise TypeError(f"unsupported dtype {out_dtype}; use the cache's or float32")
        self.o = out if out is not None else torch.empty((T, H, c.D), dtype=out_dtype, device=dev)
        self.lse = lse if lse is not None else torch.empty((H, T), dtype=torch.float32, device=dev)
        if self.o.shape != q.shape:
            raise ValueError(f"out must be {tuple(q.shape)}, got {tuple(self.o.shape)}")
        if tuple(self.lse.shape) != (H, T) or self.lse.dtype != torch.float32 or not self.lse.is_contiguous() \
                or self.lse.device != dev:
            raise ValueError(f"lse must be contiguous float32 {(H, T)} on the cache's device")
        a.o = _rows(self.o, "out", H, c.D, out_dtype, dev)
        a.lse = self.lse.data_ptr() if self.lse.numel() else None
        if mask is not None:
            if mask.dtype != torch.int64 or mask.dim() != 2 or mask.shape[0] != T or mask.shape[1] < 1 \
                    or not mask.is_contiguous() or mask.device != dev:
                raise ValueError(f"mask must be contiguous int64 ({T}, words) on the cache's device")
            a.mask = mask.data_ptr() if T else None
            a.mask_words = mask.shape[1]
        self.inputs = (q, mask)
        a.seqs, a.cu = self.seqs.data_ptr(), self.cu.data_ptr()
        a.layer, a.H, a.n, a.n_q = int(layer), H, self.seqs.numel(), T
        a.scale = float(scale) if scale is not None else c.D ** -0.5
        a.o_dtype = _DT[out_dtype]
        self.args = a
        self._ref = ctypes.byref(a)
        lib = cache._lib
        if workspace is None:
            with _on(dev):
                need = lib.attn_tree_workspace_bytes(self._ref)
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        self.workspace = workspace
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
        self._fn = lib.attn_tree_fwd

    def run(self, stream: torch.cuda.Stream | None = None):
        dev = self.cache.device
        s = _stream(dev) if stream is None else ctypes.c_void_p(stream.cuda_stream)
        with _on(dev):
            _abi.check(self._fn(self._ref, s), "attn_tree_fwd")
        return self.o, self.lse


def tree_fwd(q, cache: Cache, seqs, cu_seqlens_q, *, layer: int = 0, mask: torch.Tensor | None = None,
             scale: float | None = None, out_dtype: torch.dtype | None = None):
    """Attention of new tokens over the cache.  Returns ``(o, lse)``; lse is (H, T) f32, natural log.

    Rows ``cu[i]:cu[i + 1]`` of q are the last tokens of sequence ``seqs[i]``: one token
    (decoding), a chunk, or with ``mask`` a tree of drafts (see ``TreeCall``)."""
    return TreeCall(q, cache, seqs, cu_seqlens_q, layer=layer, mask=mask, scale=scale, out_dtype=out_dtype).run()
