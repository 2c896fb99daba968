"""What a call costs on the host: current stream, device switch, argument structs and lists.

A short attention call takes a few microseconds on the GPU, so the binding's
own time decides how fast short calls follow one another.  The argument structs
are therefore packed by one ``struct.pack`` (a ctypes field assignment costs as
much as the whole pack), streams are passed as their raw handles, and the device
is switched only when another one is current.  Calls whose arguments need no
conversion skip the interpreter's share altogether (``native``).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import warnings

import torch

from . import _abi

raw_stream = torch._C._cuda_getCurrentRawStream  # device index -> cudaStream_t of torch's current stream
_current_device = torch._C._cuda_getDevice

# native layouts of the argument structs in include/attn.h, field by field
_TENSOR = "Pqq"
FWD = struct.Struct("@" + _TENSOR * 4 + "P" + "iiii" + "f" + "iiii" + "PP" + "PN" + "iii" + "f" + "P" + "ii" + "0P")
BWD = struct.Struct("@" + _TENSOR * 5 + "P" + _TENSOR * 3 + "iiii" + "f" + "iiiii" + "PP" + "PN" + "ii" + "f" + "ii" + "0P")
CACHE = struct.Struct("@" + "PP" + "qqqq" + "PPP" + "q" + "iiiiiiii" + "0P")
TREE = struct.Struct("@" + "%ds" % CACHE.size + "ii" + _TENSOR * 2 + "PPPP" + "iii" + "f" + "i" + "PN" + "0P")
VIEW = struct.Struct("@" + _TENSOR)
for _s, _c in ((FWD, _abi.FwdArgs), (BWD, _abi.BwdArgs), (CACHE, _abi.Cache), (TREE, _abi.TreeArgs),
               (VIEW, _abi.AttnTensor)):
    if _s.size != ctypes.sizeof(_c):
        raise ImportError(f"packed layout of {_c.__name__} does not match its fields")

_FLOAT_MAX = 3.4028234663852886e38


def f32(x: float) -> float:
    """`x` as a C float takes it (beyond its range: infinite, which the library refuses)."""
    x = float(x)
    return x if -_FLOAT_MAX <= x <= _FLOAT_MAX or x != x else ctypes.c_float(x).value


def int32(x: torch.Tensor, device: torch.device, name: str) -> torch.Tensor:
    """Whole numbers as int32 on the device, never cut to their low bits: host values that do
    not fit raise, device values become the nearest int32, which no operation accepts."""
    if x.dtype == torch.int64:
        if x.is_cuda:
            x = x.clamp(-2 ** 31, 2 ** 31 - 1)
        elif x.numel() and not -2 ** 31 <= int(x.min()) <= int(x.max()) < 2 ** 31:
            raise ValueError(f"{name}: entries must fit 32 bits")
    elif x.dtype not in (torch.int32, torch.int16, torch.int8, torch.uint8):
        raise ValueError(f"{name} must be whole numbers of at most 64 bits, signed, not {x.dtype}")
    return x.to(device=device, dtype=torch.int32).contiguous()


def call(index: int, fn, where: str | None, *args) -> int:
    """`fn(*args)` with device `index` current.  With `where`, the result is a status
    and an error becomes an exception."""
    if index == _current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc and where is not None:
        _abi.check(rc, where)
    return rc


_NATIVE = os.path.join(os.path.dirname(_abi.LIB_PATH), "_native.so")
# the entry points that csrc/binding.cpp calls, in its order
_NATIVE_CALLS = ("attn_fwd", "attn_fwd_workspace_bytes", "attn_bwd", "attn_bwd_workspace_bytes", "attn_tree_fwd",
                 "attn_tree_workspace_bytes", "attn_cache_workspace_bytes", "attn_cache_extend", "attn_cache_fork",
                 "attn_cache_keep", "attn_cache_free", "attn_cache_write")
_native = None


class _NoBinding:
    """In place of a compiled binding that was not built: every call is left to the Python path."""

    def __getattr__(self, name: str):
        return lambda *args: None


def native():
    """The compiled binding (csrc/binding.cpp).  Its functions return None for
    arguments that they leave to the Python path, or a status of the library."""
    global _native
    if _native is None:
        lib = _abi.load()
        if not os.path.exists(_NATIVE):
            warnings.warn(f"the compiled torch binding is not built ({_NATIVE} is missing): calls cost more host time",
                          RuntimeWarning, stacklevel=3)
            _native = _NoBinding()
            return _native
        loader = importlib.machinery.ExtensionFileLoader("_native", _NATIVE)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_native", loader))
        loader.exec_module(module)
        module.init(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _NATIVE_CALLS))
        _native = module
    return _native


_fast = {}


def entry(name: str):
    """An entry point whose struct arguments may also be given as packed bytes or addresses."""
    fn = _fast.get(name)
    if fn is None:
        lib = _abi.load()
        typed = getattr(lib, name)
        fn = lib[name]  # a handle of its own, with its own argument types
        fn.restype = typed.restype
        fn.argtypes = [ctypes.c_void_p if issubclass(t, ctypes._Pointer) else t for t in typed.argtypes]
        _fast[name] = fn
    return fn
