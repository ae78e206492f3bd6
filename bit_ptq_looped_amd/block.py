"""Python binding of a block's parts between its linears and the attention
(the C ABI in include/loopq_block.h).

As in :mod:`bit_ptq_looped_amd.loopq`: argument marshalling only.  Tensors live
on the current GPU, its current HIP stream is used unless one is given, and a
non-zero status raises :class:`~bit_ptq_looped_amd.loopq.LoopQError`.
"""

from __future__ import annotations

import ctypes

from . import kv, loopq
from .loopq import _check, _dtype_code, _ptr, _stream

_P, _I, _F, _Z, _L, _D = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64,
                          ctypes.c_double)
# every entry point of include/loopq_block.h with its ctypes signature
SIGNATURES = {
    "loopq_rms_norm": ([_P, _L, _I, _P, _L, _I, _I, _I, _P, _F, _P, _L, _P, _L, _I, _P, _P, _F, _I, _I, _P], _I),
}

_lib = None


def load():
    """The library of :func:`loopq.load`, with the signatures of this header."""
    global _lib
    if _lib is None:
        lib = kv.load()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _on(t, stream):
    """The stream of a call whose first tensor is t: the current device's, where t has to live."""
    if t.device.index != loopq._torch_mod().cuda.current_device():
        raise ValueError("the tensors' device must be the current one")
    return _stream(stream)


def _rows2(t, what: str, rows: int, width: int):
    """Pointer, row distance and dtype code of [rows][width] with dense rows."""
    if tuple(t.shape) != (rows, width) or (width > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: expected [{rows}][{width}] with dense rows")
    return _ptr(t), (t.stride(0) if rows > 1 else width), _dtype_code(t)


def _dense(t, what: str, dtype, n: int):
    if t.dtype is not dtype or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{what}: a contiguous {dtype} tensor of at least {n} values")
    return _ptr(t)


# ----------------------------------------------------------------- device calls

def loopq_rms_norm(x, weight, eps: float, y=None, residual=None, sum_out=None, codes=None, steps=None,
                   clip: float = 1.0, bits_a: int = 8, per_token: bool = False, stream=None):
    """x [rows][K] (+ residual) through the RMS norm into y and / or Eq.(4) codes and steps."""
    torch = loopq._torch_mod()
    rows, K = x.shape
    xp = _rows2(x, "x", rows, K)
    rp = _rows2(residual, "residual", rows, K) if residual is not None else (None, 0, 0)
    sp = _rows2(sum_out, "sum_out", rows, K) if sum_out is not None else (None, 0, rp[2])
    if sp[2] != rp[2]:
        raise ValueError("sum_out must have the residual's type")
    yp = _rows2(y, "y", rows, K) if y is not None else (None, 0, 0)
    wp = _dense(weight, "weight", torch.float32, K) if weight is not None else None
    cp = gp = None
    if codes is not None:
        if steps is None:
            raise ValueError("codes need steps")
        cp = _dense(codes, "codes", torch.int8, rows * K)
        gp = _dense(steps, "steps", torch.float32, rows * (K // 32))
    _check(load().loopq_rms_norm(*xp, *rp, rows, K, wp, eps, sp[0], sp[1], *yp, cp, gp, clip, bits_a, int(per_token),
                                 _on(x, stream)), "loopq_rms_norm")
