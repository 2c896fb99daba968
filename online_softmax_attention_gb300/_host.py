"""What a call costs on the host: current stream, device switch, tensor views.

A short attention call takes a few microseconds on the GPU, so the binding's
own time decides how fast short calls follow one another.  The argument structs
are therefore packed by one ``struct.pack`` (a ctypes field assignment costs as
much as the whole pack), streams are passed as their raw handles, and the device
is switched only when another one is current.
"""
from __future__ import annotations

import ctypes
import struct

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
