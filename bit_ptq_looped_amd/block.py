"""Python binding of a block's parts between its linears and the attention
(the C ABI in include/loopq_block.h).

As in :mod:`bit_ptq_looped_amd.loopq`: argument marshalling only.  Tensors live
on the current GPU, its current HIP stream is used unless one is given, and a
non-zero status raises :class:`~bit_ptq_looped_amd.loopq.LoopQError`.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import kv, loopq
from .kv import KVTable, _ints, _pool, _ref, _rows3, _table
from .loopq import _check, _dtype_code, _stream

LOOPQ_ROPE_HALF, LOOPQ_ROPE_PAIRS = 0, 1
LOOPQ_ROPE_PLAIN, LOOPQ_ROPE_LINEAR, LOOPQ_ROPE_BASE, LOOPQ_ROPE_PARTS = 0, 1, 2, 3


class Rope(NamedTuple):
    """Frequencies float64 [rot_dim / 2] on the device (radians a position),
    which elements form a pair, and the factor of the turned ones."""
    inv_freq: "torch.Tensor"  # noqa: F821
    layout: int = LOOPQ_ROPE_HALF
    magnitude: float = 1.0


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("magnitude", ctypes.c_float)]


_P, _I, _F, _Z, _L, _D = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64,
                          ctypes.c_double)
_RP = ctypes.POINTER(_Rope)
# every entry point of include/loopq_block.h with its ctypes signature
SIGNATURES = {
    "loopq_rms_norm": ([_P, _L, _I, _P, _L, _I, _I, _I, _P, _F, _P, _L, _P, _L, _I, _P, _P, _F, _I, _I, _P], _I),
    "loopq_rope_frequencies": ([_I, _I, _D, _D, _D, _D, _D, ctypes.POINTER(_D)], _I),
    "loopq_rope": ([_P, _L, _I, _I, _I, _I, _P, _RP, _P, _L, _P], _I),
    "loopq_kv_write_rope": ([kv._PP, _I, kv._TP, _P, _RP, _P, _L, _P, _L, _I, _I, _P, _L, _I, _P, _L, _I, _P], _I),
    "loopq_adapter_workspace_bytes": ([_I, _I, kv._ZP], _I),
    "loopq_adapter_apply": ([_P, _L, _I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _I, _P, _L, _P, _Z, _P], _I),
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


_torch = None
_codes = None  # dtype code of each type of activations


def _types():
    global _torch, _codes
    if _torch is None:
        torch = loopq._torch_mod()
        _codes = {torch.float32: loopq.LOOPQ_F32, torch.bfloat16: loopq.LOOPQ_BF16}
        _torch = torch
    return _torch


def _on(t, stream):
    """The stream of a call whose first tensor is t: the current device's, where t has to live."""
    index = t.get_device()
    if index != _torch._C._cuda_getDevice():
        raise ValueError("the tensors' device must be the current one")
    if stream is None and loopq._raw_stream is not None:
        return loopq._raw_stream(index)
    return _stream(stream)


def _rows2(t, what: str, rows: int, width: int):
    """Pointer, row distance and dtype code of [rows][width] with dense rows."""
    code = _codes.get(t.dtype)
    if t.shape != (rows, width) or (width > 1 and t.stride(1) != 1) or code is None or not t.is_cuda:
        raise ValueError(f"{what}: expected [{rows}][{width}] of float32 or bfloat16 with dense rows on the GPU")
    return t.data_ptr(), (t.stride(0) if rows > 1 else width), code


def _dense(t, what: str, dtype, n: int):
    if t.dtype is not dtype or not t.is_contiguous() or t.numel() < n or not t.is_cuda:
        raise ValueError(f"{what}: a contiguous {dtype} tensor of at least {n} values on the GPU")
    return t.data_ptr()


def _rope(r: Rope) -> _Rope:
    f = r.inv_freq
    return _Rope(_dense(f, "inv_freq", _types().float64, 1), 2 * f.numel(), r.layout, r.magnitude)


# ----------------------------------------------------------------- host-only calls

def loopq_rope_frequencies(scaling: int, rot_dim: int, base: float = 10000.0, factor: float = 1.0,
                           length: float = 0.0, low: float = 0.0, high: float = 0.0):
    """The frequencies of a scaling as a list of rot_dim / 2 floats."""
    f = (ctypes.c_double * max(rot_dim // 2, 1))()
    _check(load().loopq_rope_frequencies(scaling, rot_dim, base, factor, length, low, high, f),
           "loopq_rope_frequencies")
    return list(f)


def loopq_adapter_workspace_bytes(rows: int, max_rank: int) -> int:
    b = ctypes.c_size_t()
    _check(load().loopq_adapter_workspace_bytes(rows, max_rank, _ref(b)), "loopq_adapter_workspace_bytes")
    return b.value


# ----------------------------------------------------------------- device calls

def loopq_rms_norm(x, weight, eps: float, y=None, residual=None, sum_out=None, codes=None, steps=None,
                   clip: float = 1.0, bits_a: int = 8, per_token: bool = False, stream=None):
    """x [rows][K] (+ residual) through the RMS norm into y and / or Eq.(4) codes and steps."""
    torch = _types()
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


def loopq_rope(x, positions, rope: Rope, out, stream=None):
    """x, out [tokens][heads][head_dim], positions int32 [tokens]; out may be x itself."""
    _types()
    tokens, heads, dim = x.shape
    xp, ldx = _rows3(x, None, dim, "x")
    op, ldo = _rows3(out, heads, dim, "out")
    if out.dtype != x.dtype or out.shape != x.shape:
        raise ValueError("out must have x's type and shape")
    _check(load().loopq_rope(xp, ldx, _dtype_code(x), tokens, heads, dim, _ints(positions, "positions", tokens),
                             _ref(_rope(rope)), op, ldo, _on(x, stream)), "loopq_rope")


def loopq_kv_write_rope(pool, slab: int, table: KVTable, cu, rope: Rope, k, v, q=None, q_out=None, stream=None):
    """k turned and v into a slab as the last tokens of each row, q turned into q_out
    (bfloat16 or float32; q itself if it has that type)."""
    _types()
    p = _pool(pool)
    heads, dim = p.heads, p.head_dim
    kp, ldk = _rows3(k, heads, dim, "k")
    vp, ldv = _rows3(v, heads, dim, "v")
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have one type and shape")
    qp = op = None
    ldq = ldo = heads_q = q_dtype = 0
    if q is not None:
        if q.dtype != k.dtype or q.shape[0] != k.shape[0] or q_out is None or q_out.shape != q.shape:
            raise ValueError("q must have k's type and tokens, q_out its shape")
        qp, ldq = _rows3(q, None, dim, "q")
        op, ldo = _rows3(q_out, None, dim, "q_out")
        heads_q, q_dtype = q.shape[1], _dtype_code(q_out)
    _check(load().loopq_kv_write_rope(_ref(p), slab, _ref(_table(table)), _ints(cu, "cu", table.lens.numel() + 1),
                                      _ref(_rope(rope)), kp, ldk, vp, ldv, _dtype_code(k), k.shape[0], qp, ldq,
                                      heads_q, op, ldo, q_dtype, _on(k, stream)), "loopq_kv_write_rope")


def loopq_adapter_apply(x, ids, A, B, scales, y, workspace, ranks=None, stream=None):
    """y [rows][N] float32 += scales[a] B[a] (A[a] x) for the adapter a = ids[row] of each row.

    x [rows][K], A bfloat16 [adapters][max_rank][K], B bfloat16 [adapters][N][max_rank]."""
    torch = _types()
    rows, K = x.shape
    n, rank, width = A.shape
    if width != K or B.shape[0] != n or B.shape[2] != rank:
        raise ValueError("A is [adapters][max_rank][K], B [adapters][N][max_rank]")
    N = B.shape[1]
    xp, ldx, dtype = _rows2(x, "x", rows, K)
    yp, ldy, y_dtype = _rows2(y, "y", rows, N)
    if y_dtype != loopq.LOOPQ_F32:
        raise ValueError("y must be float32")
    _check(load().loopq_adapter_apply(xp, ldx, dtype, rows, K, N, _ints(ids, "ids", rows),
                                      _dense(A, "A", torch.bfloat16, 1), _dense(B, "B", torch.bfloat16, 1),
                                      _dense(scales, "scales", torch.float32, n),
                                      _ints(ranks, "ranks", n) if ranks is not None else None, n, rank, yp, ldy,
                                      *kv._ws(workspace), _on(x, stream)), "loopq_adapter_apply")


# ----------------------------------------------------------------- buffer helpers

def empty_adapter_workspace(rows: int, max_rank: int, device="cuda"):
    import torch
    return torch.empty(max(loopq_adapter_workspace_bytes(rows, max_rank), 256), dtype=torch.uint8, device=device)
