"""The entry points of include/loopq_block.h reject bad arguments on the host,
before any HIP call, and size their buffers without a GPU."""

import ctypes
import math
import os
import re

import pytest

from bit_ptq_looped_amd import block, kv, loopq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # a non-null, aligned address; never dereferenced because validation fails first
MB = 1 << 24    # room between the fake buffers of a call
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = -1, -2, -3, -6
F32, BF16 = loopq.LOOPQ_F32, loopq.LOOPQ_BF16
NAN, INF = float("nan"), float("inf")
R = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(loopq.LIB_PATH):
        from bit_ptq_looped_amd import build
        build.build(verbose=False)
    return block.load()


def test_every_declared_symbol_is_bound(lib):
    text = open(os.path.join(ROOT, "include", "loopq_block.h")).read()
    names = re.findall(r"^int32_t\s+(loopq_\w+)\(", text, flags=re.M)
    assert sorted(names) == sorted(block.SIGNATURES)


# --------------------------------------------------------------------- norm

def norm(lib, **kw):
    f = dict(x=FAKE, ldx=64, xt=F32, res=FAKE + MB, ldr=64, rt=F32, rows=5, K=64, w=FAKE + 2 * MB, eps=1e-6,
             sum=FAKE + 3 * MB, lds=64, y=FAKE + 4 * MB, ldy=64, yt=F32, codes=FAKE + 5 * MB, steps=FAKE + 6 * MB,
             clip=1.0, bits=4, per_token=0, stream=None)
    assert set(kw) <= set(f)
    f.update(kw)
    return lib.loopq_rms_norm(*f.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(K=-8), INVALID), (dict(K=60), UNSUPPORTED), (dict(K=72, ldx=72), UNSUPPORTED),
    (dict(K=32800), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(xt=2), UNSUPPORTED), (dict(rt=2), UNSUPPORTED), (dict(yt=-1), UNSUPPORTED), (dict(bits=6), UNSUPPORTED),
    (dict(clip=0.0), INVALID), (dict(clip=-1.0), INVALID), (dict(clip=NAN), INVALID), (dict(clip=INF), INVALID),
    (dict(x=None), INVALID), (dict(y=None, codes=None), INVALID), (dict(res=None), INVALID), (dict(steps=None), INVALID),
    (dict(ldx=56), INVALID), (dict(ldr=32), INVALID), (dict(lds=0), INVALID), (dict(ldy=-64), INVALID),
    (dict(x=FAKE + 8), ALIGNMENT), (dict(ldx=66), ALIGNMENT), (dict(rt=BF16, ldr=68), ALIGNMENT), (dict(y=FAKE + 4 * MB + 4), ALIGNMENT),
    (dict(sum=FAKE + 3 * MB + 4), ALIGNMENT), (dict(w=FAKE + 2 * MB + 4), ALIGNMENT), (dict(codes=FAKE + 5 * MB + 4), ALIGNMENT),
    (dict(steps=FAKE + 6 * MB + 2), ALIGNMENT),
    # buffers that share memory and are not the same rows
    (dict(y=FAKE + 64), INVALID), (dict(y=FAKE, yt=BF16), INVALID), (dict(y=FAKE, ldy=68), INVALID), (dict(sum=FAKE + MB + 16), INVALID),
    (dict(sum=FAKE + 4 * MB), INVALID), (dict(codes=FAKE + 256), INVALID), (dict(codes=FAKE + 6 * MB), INVALID), (dict(steps=FAKE + MB), INVALID),
    (dict(y=FAKE + 2 * MB), INVALID), (dict(sum=FAKE + 2 * MB), INVALID), (dict(codes=FAKE + 2 * MB), INVALID), (dict(steps=FAKE + 2 * MB), INVALID)])
def test_norm_arguments(lib, kw, want):
    assert norm(lib, **kw) == want


def test_norm_of_no_rows(lib):
    assert norm(lib, rows=0, x=None, y=None, codes=None) == 0


# ------------------------------------------------------------------ binding

def test_binding_refuses_other_shapes():
    import torch
    x = torch.zeros((3, 64))
    for kw in (dict(y=torch.zeros((3, 32))), dict(y=torch.zeros((64, 3)).T), dict(y=x, residual=x, sum_out=x.bfloat16())):
        with pytest.raises(ValueError):
            block.loopq_rms_norm(x, None, 1e-6, **kw)


# ------------------------------------------------------------------- rotary

def rope_spec(**kw):
    f = dict(inv_freq=FAKE + 9 * MB, rot_dim=64, layout=0, magnitude=1.0)
    f.update(kw)
    return block._Rope(*f.values())


def rope(lib, spec=None, **kw):
    f = dict(x=FAKE, ldx=128, dt=F32, tokens=5, heads=2, dim=64, pos=FAKE + MB, spec=R(spec or rope_spec()), out=FAKE + 2 * MB, ldo=128, stream=None)
    f.update(kw)
    return lib.loopq_rope(*f.values())


def pool(**kw):
    f = dict(data=FAKE, num_pages=8, slabs=2, heads=2, page_size=16, head_dim=64)
    f.update(kw)
    return kv._Pool(*f.values())


def table(**kw):
    f = dict(table=FAKE + MB, lens=FAKE + 2 * MB, refs=FAKE + 3 * MB, rows=4, max_pages=3, num_pages=8)
    f.update(kw)
    return kv._Table(*f.values())


def write(lib, spec=None, p=None, t=None, **kw):
    f = dict(pool=R(p or pool()), slab=1, table=R(t or table()), cu=FAKE + 4 * MB, spec=R(spec or rope_spec()), k=FAKE + 5 * MB, ldk=128,
             v=FAKE + 6 * MB, ldv=128, dt=F32, tokens=5, q=FAKE + 7 * MB, ldq=256, hq=4, qo=FAKE + 8 * MB, ldqo=256, qt=F32, stream=None)
    f.update(kw)
    return lib.loopq_kv_write_rope(*f.values())


SPECS = [(dict(inv_freq=None), INVALID), (dict(inv_freq=FAKE + 4), ALIGNMENT), (dict(rot_dim=0), UNSUPPORTED), (dict(rot_dim=-2), UNSUPPORTED),
         (dict(rot_dim=33), UNSUPPORTED), (dict(rot_dim=66), UNSUPPORTED), (dict(layout=2), INVALID), (dict(layout=-1), INVALID),
         (dict(magnitude=NAN), INVALID), (dict(magnitude=INF), INVALID)]


@pytest.mark.parametrize("kw,want", SPECS)
def test_rope_specs(lib, kw, want):
    assert rope(lib, rope_spec(**kw)) == want and write(lib, rope_spec(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(spec=None), INVALID), (dict(heads=0), INVALID), (dict(dim=0), INVALID), (dict(dim=80, ldx=160, ldo=160), UNSUPPORTED),
    (dict(heads=1 << 15, ldx=1 << 21, ldo=1 << 21), UNSUPPORTED), (dict(dt=2), UNSUPPORTED), (dict(tokens=-1), INVALID),
    (dict(tokens=(1 << 26) - 3, out=FAKE + (1 << 40)), UNSUPPORTED), (dict(pos=None), INVALID), (dict(pos=FAKE + 2), ALIGNMENT), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(x=FAKE + 8), ALIGNMENT), (dict(ldx=130), ALIGNMENT), (dict(ldx=120), INVALID), (dict(ldo=64), INVALID),
    (dict(out=FAKE + 128), INVALID), (dict(out=FAKE, ldo=132), INVALID)])
def test_rope_arguments(lib, kw, want):
    if "spec" in kw:
        assert lib.loopq_rope(FAKE, 128, F32, 5, 2, 64, FAKE, None, FAKE + MB, 128, None) == want
    else:
        assert rope(lib, **kw) == want


def test_rope_of_no_tokens(lib):
    assert rope(lib, tokens=0, x=None, out=None, pos=None) == 0
    assert write(lib, tokens=0, k=None, q=None, qo=None) == 0
    assert write(lib, t=table(rows=0), k=None) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(slab=2), INVALID), (dict(slab=-1), INVALID), (dict(cu=None), INVALID), (dict(cu=FAKE + 2), ALIGNMENT), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(k=FAKE + 5 * MB + 8), ALIGNMENT), (dict(ldk=64), INVALID), (dict(ldv=130), ALIGNMENT), (dict(dt=2), UNSUPPORTED),
    (dict(qt=2), UNSUPPORTED), (dict(tokens=-1), INVALID), (dict(tokens=(1 << 26) - 3), UNSUPPORTED), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(hq=0), INVALID), (dict(hq=1 << 15), UNSUPPORTED), (dict(q=FAKE + 7 * MB + 4), ALIGNMENT), (dict(ldq=128), INVALID), (dict(ldqo=258), ALIGNMENT),
    (dict(qo=FAKE + 5 * MB), INVALID), (dict(qo=FAKE + 6 * MB), INVALID), (dict(qo=FAKE + 7 * MB, qt=BF16), INVALID), (dict(qo=FAKE + 7 * MB + 64), INVALID)])
def test_write_rope_arguments(lib, kw, want):
    assert write(lib, **kw) == want


def test_write_rope_checks_pool_and_table(lib):
    assert write(lib, p=pool(head_dim=80)) == UNSUPPORTED and write(lib, p=pool(data=None)) == INVALID
    assert write(lib, p=pool(num_pages=9)) == INVALID and write(lib, t=table(lens=None)) == INVALID
    assert write(lib, t=table(table=FAKE + 2)) == ALIGNMENT


@pytest.mark.parametrize("args,want", [
    ((4, 64, 1e4, 1, 0, 0, 0), INVALID), ((-1, 64, 1e4, 1, 0, 0, 0), INVALID), ((0, 63, 1e4, 1, 0, 0, 0), UNSUPPORTED), ((0, 0, 1e4, 1, 0, 0, 0), UNSUPPORTED),
    ((0, 130, 1e4, 1, 0, 0, 0), UNSUPPORTED), ((2, 2, 1e4, 2, 0, 0, 0), UNSUPPORTED), ((0, 64, 1.0, 1, 0, 0, 0), INVALID), ((0, 64, NAN, 1, 0, 0, 0), INVALID),
    ((1, 64, 1e4, 0.5, 0, 0, 0), INVALID), ((1, 64, 1e4, NAN, 0, 0, 0), INVALID), ((3, 64, 1e4, 2, 0, 1, 32), INVALID), ((3, 64, 1e4, 2, 8192, 4, 4), INVALID),
    ((3, 64, 1e4, 2, 8192, -1, 4), INVALID), ((3, 64, 1e4, INF, 8192, 1, 4), INVALID)])
def test_frequency_arguments(lib, args, want):
    with pytest.raises(loopq.LoopQError) as e:
        block.loopq_rope_frequencies(*args)
    assert e.value.status == want
    assert lib.loopq_rope_frequencies(0, 64, 1e4, 1, 0, 0, 0, None) == INVALID


def test_frequencies():
    """Against the formulas, and by what each scaling promises."""
    plain = block.loopq_rope_frequencies(block.LOOPQ_ROPE_PLAIN, 8, 10000.0)
    assert plain == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)
    assert block.loopq_rope_frequencies(block.LOOPQ_ROPE_LINEAR, 8, 10000.0, 4.0) == pytest.approx([f / 4 for f in plain], rel=1e-14)
    wide = block.loopq_rope_frequencies(block.LOOPQ_ROPE_BASE, 128, 10000.0, 8.0)
    old = block.loopq_rope_frequencies(block.LOOPQ_ROPE_PLAIN, 128, 10000.0)
    assert wide[0] == 1.0 and wide[-1] == pytest.approx(old[-1] / 8, rel=1e-13)
    assert all(a <= b * (1 + 1e-13) for a, b in zip(wide, old))
    parts = block.loopq_rope_frequencies(block.LOOPQ_ROPE_PARTS, 128, 10000.0, 16.0, 8192.0, 1.0, 32.0)
    for f, p in zip(old, parts):
        turns = 8192.0 * f / (2 * math.pi)
        g = min(max((turns - 1.0) / 31.0, 0.0), 1.0)
        assert p == pytest.approx(g * f + (1 - g) * f / 16.0, rel=1e-13)
        assert p == f if turns >= 32 else p < f
    assert block.loopq_rope_frequencies(block.LOOPQ_ROPE_PARTS, 64, 500000.0, 1.0, 8192.0, 1.0, 4.0) == \
        pytest.approx(block.loopq_rope_frequencies(block.LOOPQ_ROPE_PLAIN, 64, 500000.0), rel=1e-14)


def test_a_base_that_overflows_is_refused(lib):
    with pytest.raises(loopq.LoopQError):
        block.loopq_rope_frequencies(block.LOOPQ_ROPE_BASE, 4, 1e300, 1e10)
    assert block.loopq_rope_frequencies(block.LOOPQ_ROPE_LINEAR, 4, 1e300, 1e10)[0] == 1e-10


# ----------------------------------------------------------------- adapters

def adapter(lib, **kw):
    f = dict(x=FAKE, ldx=64, dt=F32, rows=5, K=64, N=48, ids=FAKE + MB, A=FAKE + 2 * MB, B=FAKE + 3 * MB, scales=FAKE + 4 * MB,
             ranks=FAKE + 5 * MB, adapters=3, max_rank=16, y=FAKE + 6 * MB, ldy=48, ws=FAKE + 7 * MB, size=MB, stream=None)
    f.update(kw)
    return lib.loopq_adapter_apply(*f.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=60), UNSUPPORTED), (dict(K=65544), UNSUPPORTED),
    (dict(N=0), INVALID), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(adapters=0), INVALID), (dict(adapters=(1 << 16) + 1), UNSUPPORTED),
    (dict(max_rank=0), INVALID), (dict(max_rank=12), UNSUPPORTED), (dict(max_rank=136), UNSUPPORTED), (dict(dt=2), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(ids=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(scales=None), INVALID),
    (dict(y=None), INVALID), (dict(ldx=56), INVALID), (dict(ldy=47), INVALID), (dict(x=FAKE + 8), ALIGNMENT), (dict(ldx=66), ALIGNMENT),
    (dict(ids=FAKE + MB + 2), ALIGNMENT), (dict(A=FAKE + 2 * MB + 8), ALIGNMENT), (dict(B=FAKE + 3 * MB + 8), ALIGNMENT),
    (dict(scales=FAKE + 4 * MB + 1), ALIGNMENT), (dict(ranks=FAKE + 5 * MB + 2), ALIGNMENT), (dict(y=FAKE + 6 * MB + 2), ALIGNMENT),
    (dict(ldx=1 << 23), UNSUPPORTED), (dict(dt=BF16, ldx=1 << 24), UNSUPPORTED), (dict(ldy=1 << 24), UNSUPPORTED), (dict(y=FAKE), INVALID), (dict(y=FAKE + 256), INVALID), (dict(ws=None), WORKSPACE), (dict(size=0), WORKSPACE), (dict(ws=FAKE + 7 * MB + 64), ALIGNMENT)])
def test_adapter_arguments(lib, kw, want):
    assert adapter(lib, **kw) == want


def test_adapter_workspace(lib):
    need = block.loopq_adapter_workspace_bytes(5, 16)
    assert need % 256 == 0 and need >= 5 * 16 * 4
    assert adapter(lib, size=need - 1) == WORKSPACE
    assert adapter(lib, rows=0, x=None, y=None, ws=None) == 0
    for args, want in (((-1, 16), INVALID), ((5, 0), INVALID), ((5, 12), UNSUPPORTED), ((5, 136), UNSUPPORTED)):
        with pytest.raises(loopq.LoopQError) as e:
            block.loopq_adapter_workspace_bytes(*args)
        assert e.value.status == want


def test_an_adapter_workspace_serves_smaller_calls(lib):
    """A server allocates once, for its largest batch and rank: no call of fewer rows or of a smaller rank needs more."""
    counts = list(range(0, 2600)) + [n + d for n in range(2624, 70000, 64) for d in (-1, 0, 1)] + [131072, 1 << 20]
    for rank in (8, 64, 128):
        need = [block.loopq_adapter_workspace_bytes(n, rank) for n in counts]
        assert need == sorted(need)
    for n in (1, 65, 2048, 2112, 40000):
        need = [block.loopq_adapter_workspace_bytes(n, r) for r in range(8, 129, 8)]
        assert need == sorted(need)
    # the call asks for no more than that: a workspace of enough bytes is only refused for its alignment
    for most, rows in ((17000, 8192), (17000, 16384), (2112, 2048), (8256, 8192), (1 << 20, 32768)):
        size = block.loopq_adapter_workspace_bytes(most, 64)
        assert adapter(lib, rows=rows, K=8, ldx=8, N=1, ldy=1, max_rank=64, ws=FAKE + 7 * MB + 64, size=size) == ALIGNMENT
