"""Low-rank adapters of many requests (include/loopq_block.h) on the GPU.

Small whole numbers make every product and sum exact in fp32, so results have
to be equal to numpy's bit for bit whatever the order; real numbers are compared
with 64 bits within the bound of their roundings."""

import numpy as np
import pytest
import torch

from bit_ptq_looped_amd import block, loopq

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def i32(v):
    return torch.tensor(np.asarray(v).tolist(), dtype=torch.int32, device="cuda")


def used(ranks, n, R):
    return np.full(n, R) if ranks is None else np.clip(ranks, 0, R)


def reference(x, ids, A, B, scales, ranks, y):
    """(y in 64 bits, bound) of numpy arrays.  n terms are added in fp32 (each step at most one
    ulp off, a truncating adder among them): 2 (n + 16) U of their magnitudes; the scale,
    the product with it and the last sum round once each."""
    n, R, K = A.shape
    out, err = y.astype(np.float64), np.zeros(y.shape)
    for m, a in enumerate(ids):
        if not 0 <= a < n:
            continue
        r = int(used(ranks, n, R)[a])
        ax, s = x[m].astype(np.float64), float(scales[a])
        z = s * (A[a, :r] @ ax)
        ez = abs(s) * (np.abs(A[a, :r]) @ np.abs(ax)) * 2 * (K + 18) * U
        b = B[a, :, :r]
        out[m] += b @ z
        err[m] = np.abs(b) @ ez + 2 * (r + 16) * U * (np.abs(b) @ (np.abs(z) + ez)) + 2 * U * (np.abs(out[m]) + np.abs(y[m]))
    return out, err


def apply(x, ids, A, B, scales, y, ranks=None):
    ws = block.empty_adapter_workspace(x.shape[0], A.shape[1])
    ws.view(torch.float32).fill_(float("nan"))  # nothing of it is taken for a result
    block.loopq_adapter_apply(x, i32(ids), A, B, scales, y, ws, ranks=None if ranks is None else i32(ranks))
    torch.cuda.synchronize()


def whole(rng, rows, K, N, n, R):
    """Numbers whose products and sums stay below 2^24."""
    top = max(1, min(4, int(2 ** 24 / (K * 2 * 2 * R * 2))))
    return (rng.integers(-top, top + 1, (rows, K)), rng.integers(-1, 2, (n, R, K)), rng.integers(-1, 2, (n, N, R)),
            rng.choice([0.5, 1.0, 2.0], n), rng.integers(-1000, 1001, (rows, N)))


SIZES = [  # rows, K, N, adapters, max_rank
    (1, 8, 1, 1, 8), (1, 2048, 6144, 4, 16), (3, 520, 70, 2, 24), (16, 1024, 333, 5, 8), (17, 2560, 260, 3, 40),
    (48, 2560, 512, 32, 16), (64, 136, 129, 7, 128), (65, 384, 192, 4, 64), (100, 6912, 256, 8, 32), (129, 640, 68, 2, 72),
    (500, 2048, 1000, 6, 16), (700, 5632, 130, 3, 48), (1031, 264, 260, 40, 8), (2100, 512, 515, 5, 128), (5000, 96, 64, 3, 16),
    (257, 8, 1, 3, 8), (300, 136, 77, 2, 24), (400, 520, 200, 20, 64), (320, 1032, 130, 9, 128), (600, 2048, 65, 70, 32), (1200, 304, 260, 30, 48),
    # few rows in one launch (rank up to 32, few outputs) and in two
    (1, 2560, 1100, 2, 8), (5, 2056, 2050, 3, 32), (70, 1544, 1025, 9, 16), (3, 512, 1024, 2, 24), (9, 6912, 3100, 4, 32), (600, 1032, 1030, 5, 32),
    # in tiles: rows (K + N) of 5 2^19 and more
    (257, 8, 10400, 3, 8), (300, 136, 8800, 2, 24), (400, 6520, 200, 20, 64), (320, 8200, 130, 9, 128), (600, 4360, 65, 70, 32),
    (1200, 304, 1999, 30, 48), (5000, 456, 77, 3, 16), (2100, 1024, 515, 5, 128), (40000, 8, 64, 200, 8), (3000, 640, 257, 1500, 8),
    (200, 13200, 33, 3, 72), (20, 64, 140000, 2, 16), (1031, 2560, 260, 40, 8)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("order", ["requests", "mixed", "one"])
@pytest.mark.parametrize("rows,K,N,n,R", SIZES)
def test_whole_numbers(lq, rows, K, N, n, R, order, dtype):
    rng = np.random.default_rng(rows * 7 + K + N)
    x, A, B, s, y = whole(rng, rows, K, N, n, R)
    ranks = rng.integers(-1, R + 3, n)
    ranks[rng.integers(n)] = R
    ids = rng.integers(-1, n + 1, rows)
    ids[rng.integers(rows)] = -2 ** 31
    if order == "requests":
        ids = np.sort(ids)
    if order == "one":
        ids[:] = n - 1
    want, _ = reference(x, ids, A, B, s, ranks, y)
    got = dev(y)
    # what lies past an adapter's rank is not used, whatever it holds
    fa, fb = A.astype(np.float32), B.astype(np.float32)
    for a, r in enumerate(used(ranks, n, R)):
        fa[a, r:], fb[a, :, r:] = np.nan, np.inf
    apply(dev(x, dtype), ids, dev(fa, BF16), dev(fb, BF16), dev(s, F32), got, ranks)
    assert torch.equal(got.double().cpu(), torch.from_numpy(want))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,K,N,n,R", SIZES)
def test_real_numbers(lq, rows, K, N, n, R, dtype):
    rng = np.random.default_rng(rows + 3 * K + N)
    x = dev(rng.standard_normal((rows, K)) * np.exp(2 * rng.standard_normal((rows, 1))), dtype)
    A, B = dev(rng.standard_normal((n, R, K)) / np.sqrt(K), BF16), dev(rng.standard_normal((n, N, R)), BF16)
    s, y = dev(rng.uniform(-2, 2, n), F32), dev(rng.standard_normal((rows, N)), F32)
    ids = np.sort(rng.integers(-1, n, rows))
    host = [t.double().cpu().numpy() for t in (x, A, B, s, y)]
    want, err = reference(host[0], ids, host[1], host[2], host[3], None, host[4])
    apply(x, ids, A, B, s, y)
    off = np.abs(y.double().cpu().numpy() - want)
    assert np.all(off <= err)
    if (ids >= 0).any():  # worst cases do not add up: far below the bound in norm, as sums of independent roundings are
        assert np.linalg.norm(off) <= 8 * U * np.sqrt(K) * np.linalg.norm(err / (2 * (K + 18) * U))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,K,N,n,R", [(20, 512, 300, 4, 16), (200, 512, 320, 4, 64), (900, 768, 130, 4, 24), (900, 2904, 130, 4, 24),
                                             (300, 512, 8400, 4, 64), (2700, 968, 64, 30, 16)])
def test_what_is_not_finite_stays_with_its_rows(lq, rows, K, N, n, R, dtype):
    rng = np.random.default_rng(rows)
    x, A, B, s, y = whole(rng, rows, K, N, n, R)
    ids = rng.integers(-1, n, rows)
    ids[:4] = [0, 1, 2, 3]
    want, _ = reference(x, ids, A, B, s, None, y)
    x, A, B, s, y = dev(x, dtype), dev(A, BF16), dev(B, BF16), dev(s, F32), dev(y)
    A[1, 3, 5], B[2, 7, 1] = float("nan"), float("inf")
    x[0, 9] = float("inf")
    y[3, 11] = float("nan")
    none = int(np.flatnonzero(ids == -1)[0])
    y[none, 1] = float("nan")
    want[none, 1] = want[3, 11] = np.nan
    apply(x, ids, A, B, s, y)
    got = y.double().cpu().numpy()
    fine = np.ones(rows, dtype=bool)
    fine[0] = False
    fine[ids == 1] = False
    one = np.flatnonzero(ids == 2)
    assert not np.isfinite(got[ids == 1]).all(axis=1).any() and not np.isfinite(got[0]).all()
    cols = np.arange(N) != 7
    assert np.array_equal(got[one][:, cols], want[one][:, cols])  # B's infinity: that output of its own rows
    fine[one] = False
    assert np.array_equal(got[fine], want[fine], equal_nan=True)


@pytest.mark.parametrize("rows,K,N,n,R", [(7, 264, 131, 3, 16), (300, 512, 515, 3, 32), (1500, 520, 66, 3, 8), (300, 512, 8515, 3, 32), (1500, 1720, 66, 3, 8)])
def test_strides_and_rows_without_an_adapter(lq, rows, K, N, n, R):
    """Columns of wider rows, odd distances of y, and nothing written but rows with an adapter."""
    rng = np.random.default_rng(rows)
    x, A, B, s, y = whole(rng, rows, K, N, n, R)
    ids = np.sort(rng.integers(-1, n + 1, rows))
    want, _ = reference(x, ids, A, B, s, None, y)
    xw = torch.full((rows, K + 40), float("nan"), device="cuda")
    xw[:, 8:8 + K] = dev(x)
    none = (ids < 0) | (ids >= n)
    xw[torch.from_numpy(none).cuda()] = float("nan")
    yw = torch.full((rows + 2, N + 5), 3.5, device="cuda")
    yw[1:-1, 3:3 + N] = dev(y)
    yw[1:-1, 3:3 + N][torch.from_numpy(none).cuda()] = float("nan")
    want[none] = np.nan
    apply(xw[:, 8:8 + K], ids, dev(A, BF16), dev(B, BF16), dev(s, F32), yw[1:-1, 3:3 + N])
    got = yw.double().cpu().numpy()
    assert np.array_equal(got[1:-1, 3:3 + N], want, equal_nan=True)
    got[1:-1, 3:3 + N] = 3.5
    assert (got == 3.5).all()


@pytest.mark.parametrize("rows,K,N,n,R", [(9, 1024, 300, 4, 16), (12, 2560, 2300, 4, 24), (400, 2048, 1500, 4, 16), (260, 1024, 300, 4, 64), (1300, 640, 100, 8, 16), (700, 2048, 300, 12, 64),
                                             (300, 640, 130, 9, 128), (1000, 1024, 68, 40, 24), (1300, 1960, 100, 8, 16), (700, 2048, 1800, 12, 64),
                                             (300, 640, 8130, 9, 128), (1100, 2408, 68, 40, 24)])
def test_a_row_does_not_depend_on_other_rows(lq, rows, K, N, n, R):
    rng = np.random.default_rng(rows)
    x, A, B = dev(rng.standard_normal((rows, K))), dev(rng.standard_normal((n, R, K)), BF16), dev(rng.standard_normal((n, N, R)), BF16)
    s, y = dev(rng.uniform(-2, 2, n), F32), dev(rng.standard_normal((rows, N)))
    ids = rng.integers(0, n, rows)
    mixed, again = y.clone(), y.clone()
    apply(x, ids, A, B, s, mixed)
    apply(x, ids, A, B, s, again)
    assert torch.equal(mixed, again)
    for a in range(min(n, 3)):
        one = y.clone()
        apply(x, np.full(rows, a), A, B, s, one)
        mine = torch.from_numpy(ids == a).cuda()
        assert torch.equal(one[mine], mixed[mine])


@pytest.mark.parametrize("rows, dtype, N, n", [(40, BF16, 68, 3), (300, BF16, 8600, 3), (300, BF16, 8600, 9), (300, F32, 8600, 9)])
def test_rows_far_apart(lq, rows, dtype, N, n):
    """Row distances at the limit: a tile spans almost 2^31 bytes, the matrix much more."""
    rng = np.random.default_rng(rows)
    K, R, ld = 264, 16, (1 << 24) - 8
    ldx = ld if dtype is BF16 else (1 << 23) - 8
    x, A, B, s, y = whole(rng, rows, K, N, n, R)
    ids = rng.integers(-1, n, rows)
    want, _ = reference(x, ids, A, B, s, None, y)
    xw = torch.empty((rows - 1) * ldx + K, dtype=dtype, device="cuda").as_strided((rows, K), (ldx, 1))
    yw = torch.empty((rows - 1) * ld + N, device="cuda").as_strided((rows, N), (ld, 1))
    xw.copy_(dev(x, dtype))
    yw.copy_(dev(y))
    apply(xw, ids, dev(A, BF16), dev(B, BF16), dev(s, F32), yw)
    assert torch.equal(yw.double().cpu(), torch.from_numpy(want))


def test_no_rows_and_no_adapters(lq):
    A, B, s = dev(np.ones((2, 8, 16)), BF16), dev(np.ones((2, 5, 8)), BF16), dev(np.ones(2), F32)
    y = torch.zeros((0, 5), device="cuda")
    apply(torch.zeros((0, 16), device="cuda"), [], A, B, s, y)
    for rows in (3, 400, 130000):
        y = torch.full((rows, 5), float("nan"), device="cuda")
        apply(torch.zeros((rows, 16), device="cuda"), [-1] * rows, A, B, s, y)
        assert y.isnan().all()


@pytest.mark.parametrize("rows", [6, 400, 2700])
def test_on_a_stream_and_in_a_graph(lq, rows):
    rng = np.random.default_rng(rows)
    K, N, n, R = 768, 260, 4, 16
    x, A, B = dev(rng.standard_normal((rows, K))), dev(rng.standard_normal((n, R, K)), BF16), dev(rng.standard_normal((n, N, R)), BF16)
    s, first, ids = dev(rng.uniform(-2, 2, n), F32), dev(rng.standard_normal((rows, N))), i32(rng.integers(-1, n, rows))
    ws, y = block.empty_adapter_workspace(rows, R), first.clone()
    step = lambda: block.loopq_adapter_apply(x, ids, A, B, s, y, ws)  # noqa: E731
    loopq.loopq_timing_reset()
    loopq.loopq_timing_enable(True)
    step()
    loopq.loopq_timing_enable(False)
    assert loopq.loopq_timing_read()[loopq.LOOPQ_KERNEL_ADAPTER][1] == 1
    want = y.clone()
    side = torch.cuda.Stream()
    y.copy_(first)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        y.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        step()


def test_one_workspace_serves_every_call(lq):
    """The workspace of a program's largest batch and rank, with what other calls left in it."""
    rng = np.random.default_rng(5)
    K, N, n = 512, 320, 4
    ws = block.empty_adapter_workspace(8256, 64)
    ws.view(torch.float32).fill_(float("nan"))
    for rows, R in ((8256, 64), (8192, 64), (5, 16), (2048, 64), (300, 32), (8192, 8)):
        x, A, B = dev(rng.standard_normal((rows, K))), dev(rng.standard_normal((n, R, K)), BF16), dev(rng.standard_normal((n, N, R)), BF16)
        s, y, ids = dev(rng.uniform(-2, 2, n), F32), dev(rng.standard_normal((rows, N))), np.sort(rng.integers(-1, n, rows))
        want = y.clone()
        apply(x, ids, A, B, s, want)
        block.loopq_adapter_apply(x, i32(ids), A, B, s, y, ws)
        assert torch.equal(y, want)


def by_adapter(x, ids, A, B, s, y):
    """As reference, an adapter's rows at a time (whole numbers: exact whatever the order)."""
    out = y.astype(np.float64)
    order = np.argsort(ids, kind="stable")
    for part in np.split(order, np.flatnonzero(np.diff(ids[order])) + 1):
        a = int(ids[part[0]])
        if 0 <= a < A.shape[0]:
            out[part] += s[a] * ((x[part].astype(np.float64) @ A[a].T.astype(np.float64)) @ B[a].T.astype(np.float64))
    return out


@pytest.mark.parametrize("rows,K,N,n,R,dtype", [
    (1 << 20, 8, 3, 5, 8, F32), ((1 << 20) - 1, 8, 2, 5, 8, BF16),  # the most rows
    (40000, 8, 64, 1 << 16, 8, F32), (300, 8, 64, 1 << 16, 8, BF16),  # the most adapters
    (3, 8, 1 << 20, 2, 8, F32), (2, 8, 1 << 20, 2, 24, F32),  # the most outputs
    (45, 65536, 40, 2, 128, F32), (45, 65536, 40, 2, 128, BF16), (30, 65536, 40, 2, 128, F32), (2, 65536, 40, 2, 32, F32)])  # the longest rows
def test_the_largest_sizes(lq, rows, K, N, n, R, dtype):
    rng = np.random.default_rng(rows + K + N + n)
    x, A, B = (rng.integers(-1, 2, size).astype(np.int8) for size in ((rows, K), (n, R, K), (n, N, R)))
    s, y, ids = rng.choice([0.5, 1.0, 2.0], n), rng.integers(-1000, 1001, (rows, N)), rng.integers(-1, n + 1, rows)
    ids[:2] = [n - 1, 0]
    got = dev(y)
    apply(dev(x, dtype), ids, dev(A, BF16), dev(B, BF16), dev(s, F32), got)
    assert torch.equal(got.double().cpu(), torch.from_numpy(by_adapter(x, ids, A, B, s, y)))


@pytest.mark.parametrize("rows,N,R", [(40, 260, 16), (40, 260, 64), (300, 8600, 16), (2700, 260, 32)])
def test_replays_follow_the_ids(lq, rows, N, R):
    """A captured call, replayed with other ids, ranks and scales in place: in requests, in any order, none at all."""
    rng = np.random.default_rng(rows + R)
    K, n = 768, 9
    x, A, B = dev(rng.standard_normal((rows, K))), dev(rng.standard_normal((n, R, K)), BF16), dev(rng.standard_normal((n, N, R)), BF16)
    s, ids, ranks, first = dev(np.ones(n)), i32([-1] * rows), i32([0] * n), dev(rng.standard_normal((rows, N)))
    y, want, ws, other = first.clone(), first.clone(), block.empty_adapter_workspace(rows, R), block.empty_adapter_workspace(rows, R)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.loopq_adapter_apply(x, ids, A, B, s, y, ws, ranks=ranks)
    for turn in range(5):
        now = rng.integers(-1, n + 1, rows)
        ids.copy_(i32(now if turn % 2 else np.sort(now) if turn < 4 else np.full(rows, -1)))
        ranks.copy_(i32(rng.integers(-1, R + 2, n)))
        s.copy_(dev(rng.uniform(-2, 2, n)))
        y.copy_(first)
        want.copy_(first)
        other.view(torch.float32).fill_(float("nan"))
        block.loopq_adapter_apply(x, ids, A, B, s, want, other, ranks=ranks)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and (turn == 4) == torch.equal(y, first)
