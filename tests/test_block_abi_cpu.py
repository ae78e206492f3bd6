"""The entry points of include/loopq_block.h reject bad arguments on the host,
before any HIP call, and size their buffers without a GPU."""

import os
import re

import pytest

from bit_ptq_looped_amd import block, loopq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # a non-null, aligned address; never dereferenced because validation fails first
MB = 1 << 24    # room between the fake buffers of a call
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = -1, -2, -3, -6
F32, BF16 = loopq.LOOPQ_F32, loopq.LOOPQ_BF16
NAN, INF = float("nan"), float("inf")


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
