"""Python binding of the paged key-value cache and the attention over it
(the C ABI in include/loopq_kv.h).

As in :mod:`bit_ptq_looped_amd.loopq`: argument marshalling only.  Tensors live
on the GPU, the current HIP stream is used unless one is given, and a non-zero
status raises :class:`~bit_ptq_looped_amd.loopq.LoopQError`.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import loopq
from .loopq import _check, _dtype_code, _ptr, _stream

LOOPQ_KV_DONE, LOOPQ_KV_NO_PAGES, LOOPQ_KV_ROW_FULL = 0, 1, 2


class KVTable(NamedTuple):
    """Page table int32 [rows][max_pages], lengths int32 [rows] and reference
    counts int32 [num_pages], all on the device."""
    table: "torch.Tensor"  # noqa: F821
    lens: "torch.Tensor"   # noqa: F821
    refs: "torch.Tensor"   # noqa: F821


class _Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_int32) for n in
                                              ("num_pages", "slabs", "heads", "page_size", "head_dim")]


class _Table(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("table", "lens", "refs")] + \
               [(n, ctypes.c_int32) for n in ("rows", "max_pages", "num_pages")]


_ref = ctypes.byref
_P, _I, _F, _Z, _L = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
_ZP, _PP, _TP = ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(_Pool), ctypes.POINTER(_Table)
# every entry point of include/loopq_kv.h with its ctypes signature
SIGNATURES = {
    "loopq_kv_pool_bytes": ([_I, _I, _I, _I, _I, _ZP], _I),
    "loopq_kv_workspace_bytes": ([_I, _I, _ZP], _I),
    "loopq_kv_reserve": ([_TP, _I, _P, _TP, _P, _P, _Z, _P], _I),
    "loopq_kv_write": ([_PP, _I, _TP, _P, _P, _L, _P, _L, _I, _I, _P], _I),
    "loopq_kv_fork": ([_PP, _TP, _P, _TP, _P, _P, _Z, _P], _I),
    "loopq_kv_trim": ([_TP, _I, _I, _I, _TP, _P], _I),
    "loopq_kv_compact": ([_PP, _TP, _TP, _P, _P, _P, _Z, _P], _I),
    "loopq_kv_copy_pages": ([_PP, _P, _PP, _P, _I, _P], _I),
    "loopq_attn_workspace_bytes": ([_I, _I, _I, _I, _ZP], _I),
    "loopq_attn_decode": ([_PP, _I, _TP, _P, _L, _I, _I, _F, _I, _I, _P, _L, _P, _Z, _P], _I),
    "loopq_attn_prefill": ([_PP, _I, _TP, _P, _P, _L, _I, _I, _I, _F, _I, _I, _P, _L, _P, _Z, _P], _I),
}

_lib = None


def load():
    """The library of :func:`loopq.load`, with the signatures of this header."""
    global _lib
    if _lib is None:
        lib = loopq.load()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _pool(t) -> _Pool:
    """pool tensor bf16 [num_pages][slabs][2][heads][page_size][head_dim]"""
    shape = t.shape
    if len(shape) != 6 or shape[2] != 2 or t.dtype is not _types().bfloat16 or not t.is_contiguous():
        raise ValueError("a pool is a contiguous bfloat16 tensor [pages][slabs][2][heads][page_size][head_dim]")
    P, S, _, H, n, D = shape
    return _Pool(_ptr(t), P, S, H, n, D)


_torch = None


def _types():
    global _torch
    if _torch is None:
        _torch = loopq._torch_mod()
    return _torch


def _ints(t, what: str, n: int = 0) -> int:
    if t.dtype is not (_torch or _types()).int32 or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{what}: a contiguous int32 tensor of at least {n} values")
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    return t.data_ptr()


def _table(t: KVTable) -> _Table:
    table, lens, refs = t
    shape = table.shape
    if len(shape) != 2 or lens.numel() != shape[0]:
        raise ValueError("a table is [rows][max_pages] with one length per row")
    return _Table(_ints(table, "table"), _ints(lens, "lens"), _ints(refs, "refs"), shape[0], shape[1], refs.numel())


def _rows3(x, heads, dim: int, what: str):
    """Pointer and row distance of [tokens][heads][dim] with dense heads."""
    shape = x.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{what}: expected [tokens][{heads if heads is not None else 'heads'}][{dim}], got {tuple(shape)}")
    row, head, one = x.stride()
    if (one != 1 or (head != dim and shape[1] > 1)) and x.numel():
        raise ValueError(f"{what}: heads and elements of a token must be dense")
    if not x.is_cuda:
        raise ValueError("tensor must live on the GPU")
    return x.data_ptr(), (row if shape[0] > 1 else shape[1] * dim)


def _ws(workspace):
    return _ptr(workspace), workspace.numel() * workspace.element_size()


# ----------------------------------------------------------------- host-only calls

def loopq_kv_pool_bytes(num_pages: int, slabs: int, heads: int, page_size: int, head_dim: int) -> int:
    b = ctypes.c_size_t()
    _check(load().loopq_kv_pool_bytes(num_pages, slabs, heads, page_size, head_dim, _ref(b)),
           "loopq_kv_pool_bytes")
    return b.value


def loopq_kv_workspace_bytes(rows: int, num_pages: int) -> int:
    b = ctypes.c_size_t()
    _check(load().loopq_kv_workspace_bytes(rows, num_pages, _ref(b)), "loopq_kv_workspace_bytes")
    return b.value


def loopq_attn_workspace_bytes(queries: int, heads_q: int, rows: int, head_dim: int) -> int:
    b = ctypes.c_size_t()
    _check(load().loopq_attn_workspace_bytes(queries, heads_q, rows, head_dim, _ref(b)),
           "loopq_attn_workspace_bytes")
    return b.value


# ----------------------------------------------------------------- device calls

def loopq_kv_reserve(table: KVTable, page_size: int, grow, out: KVTable, info, workspace, stream=None):
    """Room for grow[b] more tokens in each row; out may be table itself."""
    _check(load().loopq_kv_reserve(_ref(_table(table)), page_size, _ints(grow, "grow", table.lens.numel()),
                                   _ref(_table(out)), _ints(info, "info", 2), *_ws(workspace),
                                   _stream(stream)), "loopq_kv_reserve")


def loopq_kv_write(pool, slab: int, table: KVTable, cu, k, v, stream=None):
    """k, v [tokens][heads][head_dim]: the last tokens of each row into a slab."""
    p = _pool(pool)
    kp, ldk = _rows3(k, p.heads, p.head_dim, "k")
    vp, ldv = _rows3(v, p.heads, p.head_dim, "v")
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have one type and shape")
    _check(load().loopq_kv_write(_ref(p), slab, _ref(_table(table)),
                                 _ints(cu, "cu", table.lens.numel() + 1), kp, ldk, vp, ldv, _dtype_code(k),
                                 k.shape[0], _stream(stream)), "loopq_kv_write")


def loopq_kv_fork(pool, table: KVTable, parent, out: KVTable, info, workspace, stream=None):
    """Row i of out takes the tokens of row parent[i] of table."""
    _check(load().loopq_kv_fork(_ref(_pool(pool)), _ref(_table(table)),
                                _ints(parent, "parent", out.lens.numel()), _ref(_table(out)),
                                _ints(info, "info", 2), *_ws(workspace), _stream(stream)), "loopq_kv_fork")


def loopq_kv_trim(table: KVTable, page_size: int, window: int, sinks: int, out: KVTable, stream=None):
    """Drop the pages that a sliding window has left behind; out may be table."""
    _check(load().loopq_kv_trim(_ref(_table(table)), page_size, window, sinks, _ref(_table(out)),
                                _stream(stream)), "loopq_kv_trim")


def loopq_kv_compact(pool, table: KVTable, out: KVTable, page_map, info, workspace, stream=None):
    """Move the used pages to the front of the pool; out may be table itself."""
    _check(load().loopq_kv_compact(_ref(_pool(pool)), _ref(_table(table)), _ref(_table(out)),
                                   _ints(page_map, "page_map", table.refs.numel()), _ints(info, "info", 2),
                                   *_ws(workspace), _stream(stream)), "loopq_kv_compact")


def loopq_kv_copy_pages(src_pool, src, dst_pool, dst, stream=None):
    """Page dst[i] of dst_pool = page src[i] of src_pool."""
    if src.numel() != dst.numel():
        raise ValueError("src and dst must have one length")
    _check(load().loopq_kv_copy_pages(_ref(_pool(src_pool)), _ints(src, "src"), _ref(_pool(dst_pool)),
                                      _ints(dst, "dst"), src.numel(), _stream(stream)), "loopq_kv_copy_pages")


def _out_like(q, out):
    if out.dtype != q.dtype or out.shape != q.shape:
        raise ValueError("out must have q's type and shape")


def loopq_attn_decode(pool, slab: int, table: KVTable, q, out, workspace, scale: float, window: int = 0,
                      sinks: int = 0, stream=None):
    """q, out [rows][heads_q][head_dim]: one new token per row."""
    p = _pool(pool)
    qp, ldq = _rows3(q, None, p.head_dim, "q")
    op, ldo = _rows3(out, None, p.head_dim, "out")
    _out_like(q, out)
    if q.shape[0] != table.lens.numel():
        raise ValueError("one query per row")
    _check(load().loopq_attn_decode(_ref(p), slab, _ref(_table(table)), qp, ldq, _dtype_code(q),
                                    q.shape[1], scale, window, sinks, op, ldo, *_ws(workspace), _stream(stream)),
           "loopq_attn_decode")


def loopq_attn_prefill(pool, slab: int, table: KVTable, cu, q, out, workspace, scale: float, window: int = 0,
                       sinks: int = 0, stream=None):
    """q, out [queries][heads_q][head_dim]: cu[b] .. cu[b+1]-1 are row b's last tokens."""
    p = _pool(pool)
    qp, ldq = _rows3(q, None, p.head_dim, "q")
    op, ldo = _rows3(out, None, p.head_dim, "out")
    _out_like(q, out)
    _check(load().loopq_attn_prefill(_ref(p), slab, _ref(_table(table)),
                                     _ints(cu, "cu", table.lens.numel() + 1), qp, ldq, _dtype_code(q), q.shape[0],
                                     q.shape[1], scale, window, sinks, op, ldo, *_ws(workspace), _stream(stream)),
           "loopq_attn_prefill")


# ----------------------------------------------------------------- buffer helpers

def empty_pool(num_pages: int, slabs: int, heads: int, page_size: int, head_dim: int, device="cuda"):
    """Uninitialized pool."""
    import torch
    loopq_kv_pool_bytes(num_pages, slabs, heads, page_size, head_dim)  # checks the shape
    return torch.empty((num_pages, slabs, 2, heads, page_size, head_dim), dtype=torch.bfloat16, device=device)


def new_table(rows: int, max_pages: int, num_pages: int, device="cuda") -> KVTable:
    """Empty rows and free pages."""
    import torch
    return KVTable(torch.full((rows, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(rows, dtype=torch.int32, device=device),
                   torch.zeros(num_pages, dtype=torch.int32, device=device))


def empty_table(rows: int, max_pages: int, num_pages: int, device="cuda") -> KVTable:
    """Uninitialized buffers of a table, for a call's out."""
    import torch
    return KVTable(torch.empty((rows, max_pages), dtype=torch.int32, device=device),
                   torch.empty(rows, dtype=torch.int32, device=device),
                   torch.empty(num_pages, dtype=torch.int32, device=device))


def empty_pages_workspace(rows: int, num_pages: int, device="cuda"):
    import torch
    return torch.empty(max(loopq_kv_workspace_bytes(rows, num_pages), 256), dtype=torch.uint8, device=device)


def empty_attn_workspace(pool, queries: int, heads_q: int, rows: int):
    import torch
    return torch.empty(max(loopq_attn_workspace_bytes(queries, heads_q, rows, pool.shape[5]), 256),
                       dtype=torch.uint8, device=pool.device)
