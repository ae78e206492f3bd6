"""The cache's and the attention's entry points reject bad arguments on the
host, before any HIP call, and size their buffers without a GPU."""

import ctypes
import os
import re

import pytest

from bit_ptq_looped_amd import kv, loopq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # a non-null, aligned address; never dereferenced because validation fails first
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = -1, -2, -3, -6


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(loopq.LIB_PATH):
        from bit_ptq_looped_amd import build
        build.build(verbose=False)
    return kv.load()


def pool(**kw):
    f = dict(data=FAKE, num_pages=8, slabs=2, heads=2, page_size=16, head_dim=64)
    f.update(kw)
    return kv._Pool(*f.values())


def table(at=0, **kw):
    f = dict(table=FAKE + at, lens=FAKE + 4096 + at, refs=FAKE + 8192 + at, rows=4, max_pages=3, num_pages=8)
    f.update(kw)
    return kv._Table(*f.values())


R = ctypes.byref
OTHER = 1 << 16


def test_every_declared_symbol_is_bound(lib):
    text = open(os.path.join(ROOT, "include", "loopq_kv.h")).read()
    names = re.findall(r"^int32_t\s+(loopq_\w+)\(", text, flags=re.M)
    assert sorted(names) == sorted(kv.SIGNATURES)


def test_sizes(lib):
    assert kv.loopq_kv_pool_bytes(10, 4, 16, 16, 128) == 10 * 4 * 2 * 16 * 16 * 128 * 2
    assert kv.loopq_kv_pool_bytes(1 << 22, 96, 64, 256, 128) > 2 ** 40
    assert kv.loopq_kv_workspace_bytes(0, 1) % 256 == 0
    assert kv.loopq_kv_workspace_bytes(100, 5000) >= 5000 * 4 + 4 * 400
    assert kv.loopq_attn_workspace_bytes(4, 16, 4, 128) % 256 == 0


@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=0), INVALID), (dict(page_size=12), UNSUPPORTED), (dict(page_size=4), UNSUPPORTED),
    (dict(page_size=512), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=(1 << 22) + 1), UNSUPPORTED),
    (dict(slabs=1 << 14, heads=64, page_size=256, head_dim=128), UNSUPPORTED), (dict(slabs=1, heads=1 << 15), UNSUPPORTED),
    (dict(slabs=(1 << 16) + 1, heads=1), UNSUPPORTED), (dict(slabs=0), INVALID), (dict(heads=-1), INVALID), (dict(data=None), INVALID), (dict(data=FAKE + 8), ALIGNMENT)])
def test_pools_are_checked(lib, kw, want):
    p, t, u = pool(**kw), table(), table(OTHER)
    n = p.num_pages if 0 < p.num_pages <= 1 << 22 else 8
    t.num_pages = u.num_pages = n
    assert lib.loopq_attn_decode(R(p), 0, R(t), FAKE, 128, 1, 2, 1.0, 0, 0, FAKE + OTHER, 128, FAKE, 1 << 30, None) == want
    assert lib.loopq_attn_prefill(R(p), 0, R(t), FAKE, FAKE, 128, 1, 5, 2, 1.0, 0, 0, FAKE + OTHER, 128, FAKE, 1 << 30, None) == want
    assert lib.loopq_kv_write(R(p), 0, R(t), FAKE, FAKE, 128, FAKE, 128, 1, 5, None) == want
    assert lib.loopq_kv_fork(R(p), R(t), FAKE, R(u), FAKE, FAKE, 1 << 30, None) == want
    assert lib.loopq_kv_compact(R(p), R(t), R(u), FAKE, FAKE, FAKE, 1 << 30, None) == want
    assert lib.loopq_kv_copy_pages(R(p), FAKE, R(pool()), FAKE, 3, None) == want
    if "data" not in kw:
        b = ctypes.c_size_t()
        assert lib.loopq_kv_pool_bytes(p.num_pages, p.slabs, p.heads, p.page_size, p.head_dim, R(b)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(refs=None), INVALID), (dict(table=FAKE + 2), ALIGNMENT),
    (dict(rows=-1), INVALID), (dict(rows=8193), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(rows=1024, max_pages=1 << 22), UNSUPPORTED),
    (dict(rows=1, max_pages=(1 << 22) + 1), UNSUPPORTED), (dict(num_pages=0), INVALID)])
def test_tables_are_checked(lib, kw, want):
    p, t = pool(), table(**kw)
    u = table(1 << 40)
    u.rows, u.max_pages, u.num_pages = t.rows, t.max_pages, t.num_pages
    assert lib.loopq_attn_decode(R(p), 0, R(t), FAKE, 128, 1, 2, 1.0, 0, 0, FAKE + OTHER, 128, FAKE, 1 << 30, None) == want
    assert lib.loopq_kv_write(R(p), 0, R(t), FAKE, FAKE, 128, FAKE, 128, 1, 5, None) == want
    assert lib.loopq_kv_fork(R(p), R(t), FAKE, R(u), FAKE, FAKE, 1 << 30, None) == want
    assert lib.loopq_kv_trim(R(t), 16, 8, 0, R(u), None) == want
    assert lib.loopq_kv_reserve(R(t), 16, FAKE, R(u), FAKE, FAKE, 1 << 30, None) == want
    assert lib.loopq_kv_compact(R(p), R(t), R(u), FAKE, FAKE, FAKE, 1 << 30, None) == want


def test_pairs_of_tables(lib):
    p, t = pool(), table()
    ws = (FAKE, 1 << 30, None)
    assert lib.loopq_kv_fork(R(p), R(t), FAKE, R(t), FAKE, *ws) == INVALID  # fork is not in place
    assert lib.loopq_kv_fork(R(p), R(t), FAKE, R(table(OTHER, refs=FAKE + 8192 + 4)), FAKE, *ws) == INVALID  # overlap
    assert lib.loopq_kv_reserve(R(t), 16, FAKE, R(table(OTHER, refs=t.refs)), FAKE, *ws) == INVALID  # one buffer shared
    for kw in (dict(max_pages=4), dict(num_pages=9), dict(rows=5)):
        assert lib.loopq_kv_reserve(R(t), 16, FAKE, R(table(OTHER, **kw)), FAKE, *ws) == INVALID
        assert lib.loopq_kv_trim(R(t), 16, 8, 0, R(table(OTHER, **kw)), None) == INVALID
    assert lib.loopq_kv_compact(R(pool(num_pages=9)), R(t), R(t), FAKE, FAKE, *ws) == INVALID


def test_reserve_trim_fork_compact_arguments(lib):
    p, t, u = pool(), table(), table(OTHER)
    need = kv.loopq_kv_workspace_bytes(4, 8)
    ws = (FAKE, need, None)
    assert lib.loopq_kv_reserve(R(t), 24, FAKE, R(u), FAKE, *ws) == UNSUPPORTED
    assert lib.loopq_kv_reserve(R(t), 16, None, R(u), FAKE, *ws) == INVALID
    assert lib.loopq_kv_reserve(R(t), 16, FAKE + 1, R(u), FAKE, *ws) == ALIGNMENT
    assert lib.loopq_kv_reserve(R(t), 16, FAKE, R(u), None, *ws) == INVALID
    assert lib.loopq_kv_reserve(R(t), 16, FAKE, R(u), FAKE, None, need, None) == WORKSPACE
    assert lib.loopq_kv_reserve(R(t), 16, FAKE, R(u), FAKE, FAKE, need - 1, None) == WORKSPACE
    assert lib.loopq_kv_reserve(R(t), 16, FAKE, R(u), FAKE, FAKE + 4, need, None) == ALIGNMENT
    assert lib.loopq_kv_reserve(R(table(rows=0)), 16, None, R(table(OTHER, rows=0)), None, None, 0, None) == 0
    assert lib.loopq_kv_trim(R(t), 16, 0, 0, R(u), None) == INVALID
    assert lib.loopq_kv_trim(R(t), 16, 1, -1, R(u), None) == INVALID
    assert lib.loopq_kv_fork(R(p), R(t), None, R(u), FAKE, *ws) == INVALID
    assert lib.loopq_kv_fork(R(p), R(t), FAKE, R(u), FAKE, FAKE, need - 1, None) == WORKSPACE
    assert lib.loopq_kv_compact(R(p), R(t), R(u), None, FAKE, *ws) == INVALID
    assert lib.loopq_kv_compact(R(p), R(t), R(u), FAKE, FAKE, FAKE, need - 1, None) == WORKSPACE
    assert lib.loopq_kv_copy_pages(R(p), None, R(p), FAKE, 1, None) == INVALID
    assert lib.loopq_kv_copy_pages(R(p), FAKE, R(pool(heads=3)), FAKE, 1, None) == INVALID
    assert lib.loopq_kv_copy_pages(R(p), FAKE, R(p), FAKE, -1, None) == INVALID
    assert lib.loopq_kv_copy_pages(R(p), None, R(p), None, 0, None) == 0


def test_write_arguments(lib):
    p, t = pool(), table()
    call = lambda slab=0, cu=FAKE, k=FAKE, ldk=128, v=FAKE, ldv=128, dt=1, n=5: \
        lib.loopq_kv_write(R(p), slab, R(t), cu, k, ldk, v, ldv, dt, n, None)
    assert call(slab=2) == INVALID and call(slab=-1) == INVALID and call(n=-1) == INVALID and call(cu=None) == INVALID
    assert call(k=None) == INVALID and call(v=None) == INVALID and call(ldk=120) == INVALID
    assert call(dt=2) == UNSUPPORTED
    assert call(k=FAKE + 8) == ALIGNMENT and call(ldv=132) == ALIGNMENT and call(cu=FAKE + 2) == ALIGNMENT
    assert call(ldk=130, dt=0) == ALIGNMENT
    assert call(n=0, cu=None) == 0


@pytest.mark.parametrize("prefill", [False, True])
def test_attention_arguments(lib, prefill):
    p, t = pool(), table()
    need = kv.loopq_attn_workspace_bytes(5, 4, 4, 64)

    def call(slab=0, cu=FAKE, q=FAKE, ldq=256, dt=1, n=5, hq=4, scale=1.0, window=0, sinks=0, out=FAKE + OTHER, ldo=256,
             ws=FAKE, size=need):
        tail = (hq, scale, window, sinks, out, ldo, ws, size, None)
        if prefill:
            return lib.loopq_attn_prefill(R(p), slab, R(t), cu, q, ldq, dt, n, *tail)
        return lib.loopq_attn_decode(R(p), slab, R(t), q, ldq, dt, *tail)

    assert call(slab=2) == INVALID and call(slab=-1) == INVALID
    assert call(q=None) == INVALID and call(out=None) == INVALID
    assert call(window=-1) == INVALID and call(sinks=-1) == INVALID
    assert call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    assert call(hq=3) == UNSUPPORTED and call(hq=0) == INVALID
    assert call(dt=2) == UNSUPPORTED
    assert call(q=FAKE + 8) == ALIGNMENT and call(ldo=260) == ALIGNMENT and call(ldq=248) == INVALID
    assert call(out=FAKE + 64) == INVALID  # overlaps q
    assert call(ws=None) == WORKSPACE and call(size=0) == WORKSPACE and call(ws=FAKE + 128) == ALIGNMENT
    if prefill:
        assert call(cu=None) == INVALID and call(cu=FAKE + 2) == ALIGNMENT and call(n=-1) == INVALID
        assert call(n=0, q=None, out=None) == 0
        assert call(n=(1 << 31) - 1, hq=4096, ldq=1 << 18, ldo=1 << 18) == UNSUPPORTED  # query tiles are counted in 32 bits
    assert call(hq=1 << 15) == UNSUPPORTED
    t.rows = 0
    assert call(q=None, out=None) == 0


def test_a_write_larger_than_a_launch_is_refused(lib):
    """A launch has fewer than 2^32 work-items, eight elements each, 256 of them a work-group."""
    call = lambda heads, dim, n: lib.loopq_kv_write(R(pool(heads=heads, head_dim=dim)), 0, R(table()), FAKE, FAKE, heads * dim, FAKE,
                                                    heads * dim, 1, n, None)  # noqa: E731
    assert call(2048, 128, 1 << 17) == UNSUPPORTED  # 2^32
    assert call(2, 64, (1 << 28) - 15) == UNSUPPORTED  # 2^32 - 240: its last work-group ends at 2^32
    assert call(2, 64, (1 << 31) - 1) == UNSUPPORTED


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("dt", [0, 1])
def test_columns_of_the_same_rows_do_not_overlap(lib, prefill, dt):
    """q and out in one wider row of 600 elements; a call that gets past the check lacks a workspace."""
    p, t, item = pool(), table(), 2 if dt else 4

    def call(q, out, ldq=600, ldo=600, n=4):
        tail = (4, 1.0, 0, 0, FAKE + OTHER + out * item, ldo, None, 0, None)
        if prefill:
            return lib.loopq_attn_prefill(R(p), 0, R(t), FAKE, FAKE + OTHER + q * item, ldq, dt, n, *tail)
        return lib.loopq_attn_decode(R(p), 0, R(t), FAKE + OTHER + q * item, ldq, dt, *tail)

    for q, out in ((0, 256), (256, 0), (8, 344), (344, 8), (0, 4 * 600), (0, 256 + 600), (256 + 1200, 0)):
        assert call(q, out) == WORKSPACE
    for q, out in ((0, 0), (0, 248), (248, 0), (0, 352), (352, 0), (0, 600), (0, 592), (1200, 8), (8, 1200)):
        assert call(q, out) == INVALID
    assert call(0, 256, ldo=608) == INVALID  # rows that drift apart
    if prefill:
        assert call(0, 256, n=1) == WORKSPACE and call(0, 248, n=1) == INVALID
