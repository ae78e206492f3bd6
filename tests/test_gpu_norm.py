"""Residual and RMS norm (include/loopq_block.h) on the GPU.

With r one fp32 number by definition, everything after it is a chain of single
fp32 operations: y, codes and steps are compared bit for bit with numpy (and the
oracle's quantizer) on that chain, and y with the formula in 64 bits within its
roundings."""

import numpy as np
import pytest
import torch

import oracle
from bit_ptq_looped_amd import block

pytestmark = pytest.mark.gpu

EPS = np.float32(1e-6)
U = 2.0 ** -24
FORMS = [32, 40, 64, 96, 128, 200, 256, 480, 512, 520, 1024, 1056, 2048, 2560, 2592, 4096, 5280, 6912, 8192, 10560, 16384, 17920, 32768]


def f32(t):
    return t.float().cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16()


def make(rows, K, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed * 1000003 + rows * 131 + K)
    x = torch.randn((rows, K), generator=g) * scale
    x[:, :: max(1, K // 3)] *= 20
    return x.to(dtype).cuda()


def reference(x, res, w, clip=1.0, bits=8, per_token=False):
    """(h, z, codes, steps, z in 64 bits, r) as numpy."""
    h = f32(x)
    if res is not None:
        h = h + f32(res)
        if res.dtype is torch.bfloat16:
            h = bf16(h).float().numpy()
    with np.errstate(all="ignore"):
        ms = np.mean(h.astype(np.float64) ** 2, axis=1, keepdims=True)
        r = (1.0 / np.sqrt(ms + np.float64(EPS))).astype(np.float32)
        z = h * r
        exact = h.astype(np.float64) / np.sqrt(ms + np.float64(EPS))
        if w is not None:
            z = z * f32(w)
            exact = exact * f32(w).astype(np.float64)
    if h.shape[1] % 32 or not np.isfinite(z).all():
        return h, z, None, None, exact, r
    if per_token:
        codes, steps = oracle.quant_act(z, clip, bits, h.shape[1])
        steps = np.repeat(steps, h.shape[1] // 32, axis=1)
    else:
        codes, steps = oracle.quant_act(z, clip, bits)
    return h, z, codes, steps, exact, r


def run(x, res, w, y_dtype=None, codes=False, sum_out=True, **kw):
    rows, K = x.shape
    out = dict(y=torch.empty((rows, K), dtype=y_dtype, device="cuda") if y_dtype else None,
               sum_out=torch.empty_like(res) if res is not None and sum_out else None,
               codes=torch.empty((rows, K), dtype=torch.int8, device="cuda") if codes else None,
               steps=torch.empty((rows, K // 32), dtype=torch.float32, device="cuda") if codes else None)
    block.loopq_rms_norm(x, w, float(EPS), residual=res, **out, **kw)
    torch.cuda.synchronize()
    return out


def check(x, res, w, out, **kw):
    h, z, codes, steps, exact, r = reference(x, res, w, **kw)
    if out["sum_out"] is not None:
        assert np.array_equal(f32(out["sum_out"]), h)
    if out["y"] is not None:
        got = out["y"].cpu()
        want = torch.from_numpy(z).to(got.dtype)
        assert torch.equal(got, want)
        # r (below 2^-126 to a multiple of 2^-149), h r and (h r) w are rounded to 24 bits each, the result to its type
        half = torch.finfo(got.dtype).eps / 2 if got.dtype is torch.bfloat16 else 0
        assert np.all(np.abs(got.double().numpy() - exact) <= np.abs(exact) * (3.1 * U + 2.0 ** -150 / r.astype(np.float64) + 1.01 * half) + 1e-38)
    if out["codes"] is not None:
        assert np.array_equal(out["steps"].cpu().numpy(), steps)
        assert np.array_equal(out["codes"].cpu().numpy(), codes)


@pytest.mark.parametrize("rows", [1, 5, 1100])
@pytest.mark.parametrize("K", FORMS)
def test_sizes(lq, K, rows):
    if rows * K > 8_000_000:
        rows = 1030
        if K > 8192:
            rows = 67
    w = make(1, K, torch.float32, 3)[0]
    x, res = make(rows, K, torch.float32, 1), make(rows, K, torch.bfloat16, 2, 3.0)
    quant = K % 32 == 0
    check(x, res, w, run(x, res, w, torch.bfloat16, codes=quant, bits_a=4, clip=0.75), bits=4, clip=0.75)
    check(x, None, w, run(x, None, w, torch.float32, codes=quant, bits_a=8, per_token=True), bits=8, per_token=True)


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rt", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(3, 96), (70, 2560), (1500, 2048)])
def test_types(lq, rows, K, xt, rt, bits, per_token):
    x, res = make(rows, K, xt, 4), None if rt is None else make(rows, K, rt, 5)
    w = None if bits == 4 else make(1, K, torch.float32, 6)[0]
    kw = dict(bits=bits, clip=0.9, per_token=per_token)
    for yt in (None, torch.float32, torch.bfloat16):
        out = run(x, res, w, yt, codes=True, sum_out=yt is not None, bits_a=bits, clip=0.9, per_token=per_token)
        check(x, res, w, out, **kw)


def test_codes_are_those_of_the_quantizer(lq):
    """The same bits as loopq_quant_act and loopq_quant_act_per_token on y."""
    x, res, w = make(300, 2048, torch.float32, 7), make(300, 2048, torch.float32, 8), make(1, 2048, torch.float32, 9)[0]
    for bits in (4, 8):
        for token, call in ((False, lq.loopq_quant_act), (True, lq.loopq_quant_act_per_token)):
            out = run(x, res, w, torch.float32, codes=True, bits_a=bits, clip=0.5, per_token=token)
            codes, steps = torch.empty_like(out["codes"]), torch.empty_like(out["steps"])
            call(out["y"], None, None, 0.5, bits, codes, steps)
            assert torch.equal(codes, out["codes"]) and torch.equal(steps, out["steps"])


@pytest.mark.parametrize("rows,K", [(4, 64), (4, 2048), (1200, 2560), (3, 6912), (2, 10560)])
def test_rows_of_zeros_and_extremes(lq, rows, K):
    x = make(rows, K, torch.float32, 10)
    x[0] = 0
    x[1] = 3.0e38  # squares pass fp32's range
    if rows > 2:
        x[2] = 1e-30  # the mean lies far below eps
    out = run(x, None, None, torch.float32, codes=True, bits_a=8)
    check(x, None, None, out, bits=8)
    assert not out["y"][0].any() and not out["codes"][0].any() and not out["steps"][0].any()


@pytest.mark.parametrize("rows,K", [(5, 64), (5, 2048), (700, 2560)])
def test_codes_of_weights_that_are_not_finite(lq, rows, K):
    """Finite rows, weights that make z infinite, NaN or overflow: codes and steps as loopq_quant_act has them from z."""
    x, w = make(rows, K, torch.float32, 27), torch.ones(K, device="cuda")
    w[3], w[35], w[36] = float("inf"), float("nan"), 3.4e38
    y, codes, steps = torch.empty_like(x), torch.empty((rows, K), dtype=torch.int8, device="cuda"), torch.empty((rows, K // 32), device="cuda")
    block.loopq_rms_norm(x, w, float(EPS), y=y, codes=codes, steps=steps, bits_a=8)
    c2, s2 = torch.empty_like(codes), torch.empty_like(steps)
    lq.loopq_quant_act(y, None, None, 1.0, 8, c2, s2)
    assert torch.equal(codes, c2) and np.array_equal(f32(steps), f32(s2), equal_nan=True)


@pytest.mark.parametrize("rows,K", [(6, 64), (6, 2048), (1200, 2560), (6, 6912), (6, 10560)])
@pytest.mark.parametrize("rt", [torch.float32, torch.bfloat16])
def test_rows_that_are_not_finite(lq, rows, K, rt):
    x, res = make(rows, K, torch.float32, 11), make(rows, K, rt, 12)
    bad = {1: float("nan"), 3: float("inf"), 5: float("-inf")}
    for row, v in bad.items():
        x[row, (7 * row) % K] = v
    if rt is torch.bfloat16:
        x[4, 3], res[4, 3] = 3.4e38, 0  # rounds to infinity in the residual's type
        bad[4] = 0
    out = run(x, res, None, torch.float32, codes=True, bits_a=4)
    h, z, *_ = reference(x, res, None)
    assert np.array_equal(f32(out["sum_out"]), h, equal_nan=True) and np.array_equal(f32(out["y"]), z, equal_nan=True)
    for row in range(min(rows, 8)):
        if row in bad:
            assert out["steps"][row].isnan().all() and not out["codes"][row].any()
        else:
            codes, steps = oracle.quant_act(z[row:row + 1], 1.0, 4)
            assert np.array_equal(out["codes"][row].cpu().numpy(), codes[0]) and np.array_equal(out["steps"][row].cpu().numpy(), steps[0])


@pytest.mark.parametrize("rows,K", [(5, 128), (1100, 2048), (3, 6912)])
def test_strides_and_rows_behind(lq, rows, K):
    """Columns of wider rows, and nothing written outside a row."""
    def wide(dtype, seed):
        t = make(rows + 2, K + 24, dtype, seed)
        return t, t[1:-1, 8:8 + K]
    (_, x), (_, res), w = wide(torch.float32, 13), wide(torch.bfloat16, 14), make(1, K, torch.float32, 15)[0]
    yw, y = wide(torch.bfloat16, 16)
    sw, s = wide(torch.bfloat16, 17)
    y0, s0 = yw.clone(), sw.clone()
    codes = torch.full((rows + 2, K), 99, dtype=torch.int8, device="cuda")
    steps = torch.full((rows + 2, K // 32), -1.0, device="cuda")
    block.loopq_rms_norm(x, w, float(EPS), y=y, residual=res, sum_out=s, codes=codes[1:-1], steps=steps[1:-1], bits_a=8)
    check(x, res, w, dict(y=y, sum_out=s, codes=codes[1:-1], steps=steps[1:-1]), bits=8)
    y0[1:-1, 8:8 + K], s0[1:-1, 8:8 + K] = y, s
    assert torch.equal(yw, y0) and torch.equal(sw, s0)
    assert (codes[[0, -1]] == 99).all() and (steps[[0, -1]] == -1).all()


@pytest.mark.parametrize("rows,K", [(3, 64), (1100, 2560), (9, 2048), (2, 10560)])
def test_in_place(lq, rows, K):
    w = make(1, K, torch.float32, 18)[0]
    for dt in (torch.float32, torch.bfloat16):
        x, res = make(rows, K, dt, 19), make(rows, K, dt, 20)
        want = run(x, res, w, dt)
        for y_is_x in (True, False):  # y over x and the sum over the residual, or the other way round
            a, b = x.clone(), res.clone()
            y, s = (a, b) if y_is_x else (b, a)
            block.loopq_rms_norm(a, w, float(EPS), y=y, residual=b, sum_out=s)
            assert torch.equal(y, want["y"]) and torch.equal(s, want["sum_out"])


def test_many_short_rows(lq):
    """More rows than work-groups of one launch dimension's 16 bits."""
    x = make(600_000, 64, torch.bfloat16, 21)
    out = run(x, None, None, torch.float32)
    check(x, None, None, out)


def test_offsets_past_32_bits(lq):
    rows, K = 66_000, 32768
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    y, codes = torch.empty_like(x), torch.empty((rows, K), dtype=torch.int8, device="cuda")
    steps = torch.empty((rows, K // 32), device="cuda")
    x[-3:] = make(3, K, torch.bfloat16, 25)
    block.loopq_rms_norm(x, None, float(EPS), y=y, codes=codes, steps=steps, bits_a=8)
    check(x[-3:], None, None, dict(y=y[-3:], sum_out=None, codes=codes[-3:], steps=steps[-3:]), bits=8)
    assert not y[:-3].any() and not codes[:-3].any()


def test_calls_are_recorded(lq):
    x = make(3, 64, torch.float32, 26)
    lq.loopq_timing_reset()
    lq.loopq_timing_enable(True)
    run(x, None, None, torch.float32)
    lq.loopq_timing_enable(False)
    assert lq.loopq_timing_read()[lq.LOOPQ_KERNEL_NORM][1] == 1


def test_on_a_stream_and_in_a_graph(lq):
    x, res, w = make(37, 2560, torch.float32, 22), make(37, 2560, torch.bfloat16, 23), make(1, 2560, torch.float32, 24)[0]
    want = run(x, res, w, torch.bfloat16, codes=True, bits_a=4)
    got = {k: torch.zeros_like(v) for k, v in want.items()}
    step = lambda: block.loopq_rms_norm(x, w, float(EPS), residual=res, bits_a=4, **got)  # noqa: E731
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        step()
    other.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in got.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
        run(x, res, w, torch.bfloat16)


def far_from_a_border(n, seed, lo, hi):
    """x [n][8] whose r lies 2^-hi .. 2^-lo of itself above or below the border between two fp32 numbers; the nearer one of each.

    Four elements are chosen one after the other, each the largest fp32 number whose square does not exceed what is
    left of the sum; the last is 2^-20, so that y there is r 2^-20, exactly."""
    from decimal import Decimal, getcontext
    getcontext().prec = 70
    rng = np.random.default_rng(seed)
    x, r = np.zeros((n, 8), dtype=np.float32), np.zeros(n, dtype=np.float32)
    eps = Decimal(float(EPS))
    for m in range(n):
        below = np.float32(rng.uniform(0.25, 4.0))
        above = np.nextafter(below, np.float32(8))
        border = (Decimal(float(below)) + Decimal(float(above))) / 2
        off = Decimal(float(rng.choice([-1, 1]) * 2.0 ** -rng.uniform(lo, hi)))
        left = (1 / (border * (1 + off)) ** 2 - eps) * 8 - Decimal(2) ** -40
        x[m, 7] = 2.0 ** -20
        for i in range(4):
            h = np.float32(float(left.sqrt()))
            while Decimal(float(h)) ** 2 > left:
                h = np.nextafter(h, np.float32(0))
            x[m, i] = h
            left -= Decimal(float(h)) ** 2
        mean = sum(Decimal(float(v)) ** 2 for v in x[m]) / 8
        true = 1 / (mean + eps).sqrt()
        assert Decimal(2) ** Decimal(-hi - 0.1) < abs(true / border - 1) < Decimal(2) ** Decimal(-lo + 0.1)
        r[m] = above if true > border else below
    return x, r


def test_the_root_has_its_64_bits(lq):
    """Rows whose r lies close to a border between two fp32 numbers, farther from it than the roundings of 64 bits reach.

    Of eight elements five are not zero: the sum is rounded four times, the mean (an eighth of it) never, eps is added
    with one rounding, and a root takes half of an error on: 2.5 2^-53 before the root, which adds less than 2^-52.
    Together below 2^-51; the rows stay 2^-50 away."""
    x, want = far_from_a_border(3000, 31, 46.0, 49.8)
    y = torch.empty((3000, 8), device="cuda")
    block.loopq_rms_norm(torch.from_numpy(x).cuda(), None, float(EPS), y=y)
    got = y[:, 7].cpu().numpy() * np.float32(2.0 ** 20)
    wrong = got != want
    assert not wrong.any(), f"{int(wrong.sum())} of {len(want)} rows"


# ---------------------------------------------- work-groups that take several rows

# widths, and the threads that a row of them gets where there are many rows
TURNS = [(96, 32), (480, 64), (1024, 128), (1056, 256), (2560, 256), (4096, 256), (6912, 256), (8192, 512)]


def turns(T):
    """Rows of one turn of the launch (8192 threads a CU), and so many that every work-group takes two and some a third."""
    once = torch.cuda.get_device_properties(0).multi_processor_count * 8192 // T
    return once, 2 * once + once // 3 + 5


def same(a, b):
    return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)


def turned(once, call, out):
    """The same call a turn's rows at a time, into other buffers."""
    other = {k: torch.zeros_like(v) for k, v in out.items()}
    rows = next(iter(out.values())).shape[0]
    for at in range(0, rows, once):
        part = slice(max(0, min(at, rows - once)), at + once)
        call(part, {k: v[part] for k, v in other.items()})
    return other


def pick(rows, once, bad):
    """Rows to compare with the host: both sides of each turn's end, and some between."""
    some = set(np.random.default_rng(rows).integers(0, rows, 24).tolist())
    for at in (0, once, 2 * once, rows):
        some |= {at + d for d in (-2, -1, 0, 1)}
    return sorted(r for r in some if 0 <= r < rows and r not in bad)


@pytest.mark.parametrize("K,T", TURNS)
def test_rows_of_several_turns(lq, K, T):
    """Codes and numbers, the sum over the residual: as with one row a work-group, and as on the host."""
    once, rows = turns(T)
    g = torch.Generator(device="cuda").manual_seed(K)
    x, res = torch.randn((rows, K), generator=g, device="cuda"), (3 * torch.randn((rows, K), generator=g, device="cuda")).bfloat16()
    w = 1 + 0.2 * torch.randn(K, generator=g, device="cuda")
    bad = {1: float("nan"), once + 1: float("inf"), 2 * once + 1: float("-inf"), rows - 3: float("nan")}
    for r, v in bad.items():
        x[r, (7 * r) % K] = v
    out = dict(y=torch.empty((rows, K), dtype=torch.bfloat16, device="cuda"), sum_out=torch.empty_like(res),
               codes=torch.empty((rows, K), dtype=torch.int8, device="cuda"), steps=torch.empty((rows, K // 32), device="cuda"))
    block.loopq_rms_norm(x, w, float(EPS), residual=res, bits_a=4, clip=0.75, **out)
    assert same(out, turned(once, lambda p, o: block.loopq_rms_norm(x[p], w, float(EPS), residual=res[p], bits_a=4, clip=0.75, **o), out))
    at = pick(rows, once, bad)
    check(x[at], res[at], w, {k: v[at] for k, v in out.items()}, bits=4, clip=0.75)
    for r in bad:
        assert out["steps"][r].isnan().all() and not out["codes"][r].any()
    # in place: the sum over the residual, the codes as before
    again = dict(out, y=None, sum_out=res, codes=torch.zeros_like(out["codes"]), steps=torch.zeros_like(out["steps"]))
    block.loopq_rms_norm(x, w, float(EPS), residual=res, bits_a=4, clip=0.75, **again)
    assert same({k: out[k] for k in ("sum_out", "codes", "steps")}, {k: again[k] for k in ("sum_out", "codes", "steps")})


@pytest.mark.parametrize("K,T", TURNS)
def test_rows_of_several_turns_with_one_step_a_token(lq, K, T):
    """bf16 rows over themselves, one step a row: the maximum's exchange between waves as well."""
    once, rows = turns(T)
    g = torch.Generator(device="cuda").manual_seed(K + 1)
    x = torch.randn((rows, K), generator=g, device="cuda").bfloat16()
    x *= torch.exp(torch.randn((rows, 1), generator=g, device="cuda")).bfloat16()
    x[torch.arange(rows, device="cuda"), torch.randint(0, K, (rows,), generator=g, device="cuda")] *= 8  # the maximum lies anywhere
    w = 1 + 0.2 * torch.randn(K, generator=g, device="cuda")
    bad = {0: float("inf"), once + 2: float("nan"), rows - 1: float("nan")}
    for r, v in bad.items():
        x[r, (11 * r) % K] = v
    out = dict(y=x.clone(), codes=torch.empty((rows, K), dtype=torch.int8, device="cuda"), steps=torch.empty((rows, K // 32), device="cuda"))
    block.loopq_rms_norm(out["y"], w, float(EPS), bits_a=8, per_token=True, **out)
    assert same(out, turned(once, lambda p, o: block.loopq_rms_norm(x[p], w, float(EPS), bits_a=8, per_token=True, **o), out))
    at = pick(rows, once, bad)
    check(x[at], None, w, dict({k: v[at] for k, v in out.items()}, sum_out=None), bits=8, per_token=True)
    for r in bad:
        assert out["steps"][r].isnan().all() and not out["codes"][r].any()


@pytest.mark.parametrize("rows,K", [(5, 64), (5, 2048), (700, 2560), (3, 6912), (2, 10560), (2, 32768)])
def test_token_codes_of_weights_that_are_not_finite(lq, rows, K):
    """One step a token from z with infinities and NaN: as loopq_quant_act_per_token has it from z."""
    x = make(rows, K, torch.float32, 28)
    for bad in ((3.0e38,), (float("nan"),), (float("inf"), float("nan")), (float("-inf"), 3.4e38)):
        w = torch.ones(K, device="cuda")
        for i, v in enumerate(bad):
            w[(13 * i + 3) % K] = v
        out = run(x, None, w, torch.float32, codes=True, bits_a=8, per_token=True)
        codes, steps = torch.empty_like(out["codes"]), torch.empty_like(out["steps"])
        lq.loopq_quant_act_per_token(out["y"], None, None, 1.0, 8, codes, steps)
        assert torch.equal(codes, out["codes"]) and np.array_equal(f32(steps), f32(out["steps"]), equal_nan=True)
