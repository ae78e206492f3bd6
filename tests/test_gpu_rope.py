"""Rotary positions (include/loopq_block.h) on the GPU, alone and with the cache
write, against numpy with angles in extended precision."""

import numpy as np
import pytest
import torch

from bit_ptq_looped_amd import block, kv, loopq

pytestmark = pytest.mark.gpu

HALF, PAIRS = block.LOOPQ_ROPE_HALF, block.LOOPQ_ROPE_PAIRS
F32, BF16 = torch.float32, torch.bfloat16


def bound(x, pair, m, far=2 ** 24):
    """What fp32 may be off for elements x turned with their partners: sine and cosine 3e-7
    (rounding of the angle to 24 bits and two ulp), three roundings of the factor, the product
    and the sum; the angle's 64 bits add up to 2 pi 2^-52 of the turns."""
    angle = 2.0 ** -52 * far
    return abs(m) * (np.abs(x) + np.abs(pair)) * (3e-7 + 3.1 * 2.0 ** -24 + angle) + 1e-37


def turn(x, pos, freq, layout, m, far=2 ** 24):
    """x [tokens][heads][dim] in 64 bits at pos -> (result, bound)."""
    rot = 2 * len(freq)
    t = np.asarray(pos, dtype=np.longdouble)[:, None] * np.asarray(freq, dtype=np.longdouble)
    c, s = (f(t).astype(np.float64)[:, None, :] for f in (np.cos, np.sin))
    ia, ib = (np.arange(rot // 2), np.arange(rot // 2) + rot // 2) if layout == HALF else (np.arange(0, rot, 2), np.arange(1, rot, 2))
    x = x.astype(np.float64)
    out, err = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = m * (a * c - b * s), m * (b * c + a * s)
    err[..., ia] = err[..., ib] = bound(a, b, m, far)
    return out, err


def close(got, want, err):
    half = torch.finfo(got.dtype).eps / 2 if got.dtype is BF16 else 0.0
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= err + half * (np.abs(want) + err))


def make(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def freqs(rot, base=10000.0):
    return block.loopq_rope_frequencies(block.LOOPQ_ROPE_PLAIN, rot, base)


def spec(freq, layout=HALF, m=1.0):
    return block.Rope(torch.tensor(freq, dtype=torch.float64, device="cuda"), layout, m)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (64, 2), (64, 38), (96, 96), (96, 48), (96, 94), (96, 16), (128, 128), (128, 64),
                                     (128, 126), (128, 80), (128, 20)])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 60), (37, 5), (4200, 3)])
def test_rotation(lq, tokens, heads, dim, rot, layout, dtype):
    x, f = make((tokens, heads, dim), dtype, tokens + rot), freqs(rot)
    rng = np.random.default_rng(tokens * rot)
    pos = rng.integers(0, 1 << 20, tokens)
    pos[0] = 0 if tokens > 1 else 77777
    out = torch.full_like(x, 7.0)
    block.loopq_rope(x, i32(pos), spec(f, layout, 1.25), out)
    want, err = turn(x.double().cpu().numpy(), pos, f, layout, 1.25)
    close(out, want, err)
    block.loopq_rope(x, i32(pos), spec(f, layout, 1.25), x)  # in place: the same bits
    assert torch.equal(x, out)


@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("rot", [128, 60])
def test_far_and_negative_positions(lq, layout, rot):
    pos = [2 ** 31 - 1, -2 ** 31, -1, 1, 2 ** 30 + 12345, -(2 ** 24) - 1]
    x, f = make((len(pos), 4, 128), F32, rot), freqs(rot)
    out = torch.empty_like(x)
    block.loopq_rope(x, i32(pos), spec(f, layout), out)
    want, err = turn(x.double().cpu().numpy(), pos, f, layout, 1.0, far=2 ** 31)
    close(out, want, err)


@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("dim,rot", [(96, 96), (128, 90)])
def test_the_negative_turn_is_the_transposed_one(lq, dim, rot, layout):
    """R(-p) R(p) = 1, and for a loss <g, R x> the gradient R(-p) g agrees with differences of the loss."""
    x, g, f = make((9, 4, dim), F32, 1), make((9, 4, dim), F32, 2), freqs(rot)
    pos = torch.arange(100, 109, dtype=torch.int32, device="cuda") * 977
    there, back, grad = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    block.loopq_rope(x, pos, spec(f, layout), there)
    block.loopq_rope(there, -pos, spec(f, layout), back)
    assert float((back - x).abs().max()) <= 4 * 5e-7 * float(x.abs().max())  # two turns, two elements each
    block.loopq_rope(g, -pos, spec(f, layout), grad)
    for t, h, e in ((0, 0, 0), (3, 1, rot // 2), (8, 3, dim - 1), (5, 2, 17)):
        d = torch.zeros_like(x)
        d[t, h, e] = 1.0
        moved = torch.empty_like(x)
        block.loopq_rope(d, pos, spec(f, layout), moved)
        slope = float((moved.double() * g.double()).sum())  # the loss is linear: its difference along d
        assert abs(slope - float(grad[t, h, e])) <= 4 * 5e-7 * float(g.abs().max())


@pytest.mark.parametrize("rot", [128, 100])
def test_offsets_past_32_bits(lq, rot):
    tokens, heads = 2100, 8192
    x, f = torch.zeros((tokens, heads, 128), dtype=BF16, device="cuda"), freqs(rot)
    x[-1] = make((heads, 128), BF16, rot)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    want, err = turn(x[-1:].double().cpu().numpy(), [tokens - 1], f, HALF, 1.0)
    block.loopq_rope(x, pos, spec(f), x)
    close(x[-1:], want, err)
    assert not x[:-1].any()


def test_columns_of_wider_rows(lq):
    wide = make((50, 3 * 256 + 64), BF16, 5)
    before = wide.clone()
    x, out = (wide[:, i:i + 256].unflatten(1, (2, 128)) for i in (0, 512))
    pos, f = torch.arange(50, dtype=torch.int32, device="cuda"), freqs(128)
    block.loopq_rope(x, pos, spec(f), out)
    want, err = turn(before[:, :256].double().cpu().numpy().reshape(50, 2, 128), range(50), f, HALF, 1.0)
    close(out, want, err)
    assert torch.equal(wide[:, :512], before[:, :512]) and torch.equal(wide[:, 768:], before[:, 768:])


@pytest.mark.parametrize("layout,rot", [(HALF, 64), (PAIRS, 64), (HALF, 50), (PAIRS, 50)])
def test_infinities_stay_with_their_pair(lq, layout, rot):
    x, f = make((3, 2, 64), F32, 6), freqs(rot)
    clean = torch.empty_like(x)
    pos = i32([5, 6, 7])
    block.loopq_rope(x, pos, spec(f, layout), clean)
    ia, ib = (3, 3 + rot // 2) if layout == HALF else (6, 7)
    x[1, 1, ia] = float("inf")
    x[1, 0, 63] = float("nan")
    out = torch.empty_like(x)
    block.loopq_rope(x, pos, spec(f, layout), out)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[1, 1, ia] = hit[1, 1, ib] = hit[1, 0, 63] = True
    if rot == 64:
        hit[1, 0, 31 if layout == HALF else 62] = True
    assert torch.equal(out[~hit], clean[~hit]) and not out[hit].isfinite().any()


# ------------------------------------------------------------- cache write

def world(rng, rows, heads, dim, page, slabs=2, news=None, width=9):
    """A pool of any bits, a table with holes, rows of many lengths, ragged new tokens."""
    news = [int(v) for v in (rng.choice([0, 1, 2, page, 3 * page + 1], rows) if news is None else news)]
    lens = [int(rng.integers(0, width * page - n + 1)) + n for n in news]
    pages = rows * width + 3
    order = rng.permutation(pages)
    table = np.full((rows, width), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = order[b * width:b * width + k]
    bits = torch.from_numpy(rng.integers(-32768, 32768, (pages, slabs, 2, heads, page, dim), dtype=np.int16)).cuda()
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return bits.view(BF16), table, lens, news, cu


def expect(pool, slab, table, lens, cu, k, v, page):
    """(page, place) of each token that is written, in order, and its position."""
    width, cap = table.shape[1], table.shape[1] * page
    where, pos = [], []
    for b, n in enumerate(lens):
        n = min(max(n, 0), cap)
        for t in range(cu[b], cu[b + 1]):
            p = n - int(cu[b + 1]) + t
            pos.append(p)
            ok = 0 <= p < cap and 0 <= table[b, p // page] < pool.shape[0]
            where.append((int(table[b, p // page]), p % page) if ok else None)
    return where, pos


def written(before, after, slab, where):
    """Keys and values of the written tokens; everything else has its old bits."""
    keep = torch.ones(before.shape, dtype=torch.bool, device="cuda")
    some = [w for w in where if w]
    pg, at = (torch.tensor([w[i] for w in some], device="cuda", dtype=torch.long) for i in (0, 1))
    keep[pg, slab, :, :, at] = False
    assert torch.equal(before.view(torch.int16)[keep], after.view(torch.int16)[keep])
    return after[pg, slab, 0, :, at], after[pg, slab, 1, :, at]


def check_write(rng, rows, heads, group, dim, rot, page, dtype, layout=HALF, q_dtype=None, slab=1, edit=None, **kw):
    pool, table, lens, news, cu = world(rng, rows, heads, dim, page, **kw)
    if edit:
        edit(table, lens)
    tokens, hq = int(cu[-1]) + 3, heads * group
    qkv = make((tokens, (hq + 2 * heads) * dim), dtype, int(rng.integers(1 << 30)))
    q, k, v = (qkv[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, hq), (hq, hq + heads), (hq + heads, hq + 2 * heads)))
    f = freqs(rot)
    out = torch.full((tokens, hq, dim), 5.0, dtype=q_dtype or dtype, device="cuda")
    before = pool.clone()
    t = kv.KVTable(torch.from_numpy(table).cuda(), i32(lens), torch.ones(pool.shape[0], dtype=torch.int32, device="cuda"))
    args = (pool, slab, t, torch.from_numpy(cu).cuda(), spec(f, layout, 0.75), k, v)
    block.loopq_kv_write_rope(*args, q, out)
    where, pos = expect(pool, slab, table, lens, cu, k, v, page)
    got_k, got_v = written(before, pool, slab, where)
    n = int(cu[-1])
    some = [i for i, w in enumerate(where) if w]
    want, err = turn(k[:n].double().cpu().numpy(), pos, f, layout, 0.75)
    close(got_k, want[some], err[some])
    assert torch.equal(got_v, v[some].to(BF16))
    want, err = turn(q[:n].double().cpu().numpy(), pos, f, layout, 0.75)
    close(out[:n], want, err)
    assert (out[n:] == 5.0).all()
    # without queries: the same cache
    other = before.clone()
    block.loopq_kv_write_rope(other, *args[1:])
    assert torch.equal(other.view(torch.int16), pool.view(torch.int16))
    # queries turned where they are: the same bits
    if out.dtype is dtype:
        block.loopq_kv_write_rope(*args, q, q)
        assert torch.equal(q[:n], out[:n])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,rot,layout", [(64, 64, HALF), (96, 64, PAIRS), (128, 128, HALF), (128, 32, HALF), (96, 90, HALF), (128, 34, PAIRS)])
@pytest.mark.parametrize("rows,heads,group,page", [(1, 1, 1, 8), (5, 3, 4, 16), (70, 2, 1, 32)])
def test_write(lq, rows, heads, group, page, dim, rot, layout, dtype):
    rng = np.random.default_rng(rows * dim + rot)
    check_write(rng, rows, heads, group, dim, rot, page, dtype, layout)
    check_write(rng, rows, heads, group, dim, rot, page, dtype, layout, q_dtype=BF16 if dtype is F32 else F32, slab=0)


@pytest.mark.parametrize("rows", [64, 65, 4097, 8192])
def test_write_finds_rows(lq, rows):
    rng = np.random.default_rng(rows)
    check_write(rng, rows, 1, 1, 64, 64, 8, BF16, news=rng.choice([0, 1, 1, 2], rows), width=2)


def test_write_of_bad_entries_and_lengths(lq):
    """Entries outside the pool, negative and overlong lengths, more new tokens than the row has."""
    def edit(table, lens):
        table[0, :] = [-1, 10 ** 9, -5, -2 ** 31] + [-1] * (table.shape[1] - 4)
        lens[1] = -7
        lens[2] = 2 ** 31 - 1
        lens[3] = 2
    rng = np.random.default_rng(3)
    check_write(rng, 6, 2, 2, 128, 128, 16, F32, news=[5, 4, 6, 9, 0, 2], edit=edit)
    check_write(rng, 6, 2, 2, 128, 50, 16, F32, news=[5, 4, 6, 9, 0, 2], edit=edit)


@pytest.mark.parametrize("rot", [64, 46])
def test_write_without_a_turn_is_the_plain_write(lq, rot):
    rng = np.random.default_rng(4)
    pool, table, lens, _, cu = world(rng, 9, 3, 64, 16)
    k, v = make((int(cu[-1]), 3, 64), F32, 8), make((int(cu[-1]), 3, 64), F32, 9)
    t = kv.KVTable(torch.from_numpy(table).cuda(), i32(lens), torch.ones(pool.shape[0], dtype=torch.int32, device="cuda"))
    other, cu = pool.clone(), torch.from_numpy(cu).cuda()
    block.loopq_kv_write_rope(pool, 1, t, cu, spec([0.0] * (rot // 2)), k, v)
    kv.loopq_kv_write(other, 1, t, cu, k, v)
    assert torch.equal(other.view(torch.int16), pool.view(torch.int16))


def test_empty_calls(lq):
    x, f = make((0, 2, 64), F32, 1), spec(freqs(64))
    block.loopq_rope(x, i32([]), f, x)
    pool = torch.zeros((4, 1, 2, 2, 16, 64), dtype=BF16, device="cuda")
    t = kv.new_table(0, 3, 4)
    block.loopq_kv_write_rope(pool, 0, t, i32([0]), f, make((3, 2, 64), F32, 1), make((3, 2, 64), F32, 2))
    torch.cuda.synchronize()
    assert not pool.any()


def test_on_a_stream_and_in_a_graph(lq):
    rng = np.random.default_rng(7)
    pool, table, lens, _, cu = world(rng, 12, 4, 128, 16, news=[1] * 12)
    q, k, v = make((12, 8, 128), F32, 1), make((12, 4, 128), F32, 2), make((12, 4, 128), F32, 3)
    t = kv.KVTable(torch.from_numpy(table).cuda(), i32(lens), torch.ones(pool.shape[0], dtype=torch.int32, device="cuda"))
    cu, f, first = torch.from_numpy(cu).cuda(), spec(freqs(128)), pool.clone()
    out = torch.zeros((12, 8, 128), dtype=BF16, device="cuda")
    step = lambda: block.loopq_kv_write_rope(pool, 1, t, cu, f, k, v, q, out)  # noqa: E731
    loopq.loopq_timing_reset()
    loopq.loopq_timing_enable(True)
    step()
    loopq.loopq_timing_enable(False)
    assert loopq.loopq_timing_read()[loopq.LOOPQ_KERNEL_ROPE][1] == 1
    want, want_pool = out.clone(), pool.clone()
    side = torch.cuda.Stream()
    pool.copy_(first)
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(pool.view(torch.int16), want_pool.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        pool.copy_(first)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool.view(torch.int16), want_pool.view(torch.int16))
        step()


# ------------------------------------------------ waves that take their heads in several passes

MANY = [(64, 64), (64, 38), (96, 96), (96, 94), (128, 128), (128, 126)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("dim,rot", MANY)
def test_many_heads_of_many_tokens(lq, dim, rot, layout, dtype):
    """From 4096 tokens on a wave has all 23 heads of its token: two passes and more, the last not full."""
    tokens, heads = 4100, 23
    x, f = make((tokens, heads, dim), dtype, dim + rot), freqs(rot)
    pos = np.random.default_rng(rot).integers(0, 1 << 20, tokens)
    out = torch.full_like(x, 7.0)
    block.loopq_rope(x, i32(pos), spec(f, layout, 1.25), out)
    few = torch.full_like(x, 7.0)  # a hundred tokens at a time: a wave has one pass
    for at in range(0, tokens, 100):
        block.loopq_rope(x[at:at + 100], i32(pos[at:at + 100]), spec(f, layout, 1.25), few[at:at + 100])
    assert torch.equal(out, few)
    some = np.r_[0:40, 2000:2040, tokens - 40:tokens]
    want, err = turn(x[some].double().cpu().numpy(), pos[some], f, layout, 1.25)
    close(out[some], want, err)
    block.loopq_rope(x, i32(pos), spec(f, layout, 1.25), x)
    assert torch.equal(x, out)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("dim,rot", MANY)
def test_write_of_many_tokens(lq, dim, rot, layout, dtype):
    """A wave goes from queries to keys to values, in the middle of a pass as well: 20 + 5 + 5 heads."""
    rng = np.random.default_rng(dim + rot)
    check_write(rng, 4, 5, 4, dim, rot, 32, dtype, layout, news=[1500, 0, 1300, 1400], width=80)
    check_write(rng, 3, 3, 1, dim, rot, 16, dtype, layout, q_dtype=BF16, news=[4100, 1, 7], width=300)


@pytest.mark.parametrize("rot", [128, 70])
def test_write_past_32_bits(lq, rot):
    """Pages whose elements lie more than 2^32 from the pool's start: the same as in a small pool."""
    heads, dim, page, slabs, rows = 8, 128, 256, 4, 3
    pages = (1 << 32) // (slabs * 2 * heads * page * dim) + 40
    news = [700, 1, 300]
    cu = i32(np.concatenate([[0], np.cumsum(news)]).tolist())
    k, v, q = (make((sum(news), h, dim), F32, rot + h) for h in (heads, heads, 2 * heads))
    pools, outs = [], []
    for n, first in ((12, 0), (pages, pages - 12)):
        pool = torch.zeros((n, slabs, 2, heads, page, dim), dtype=BF16, device="cuda")
        table = torch.arange(first, first + 12, dtype=torch.int32, device="cuda").view(3, 4)
        t = kv.KVTable(table, i32([900, 260, 300]), torch.ones(n, dtype=torch.int32, device="cuda"))
        out = torch.zeros((sum(news), 2 * heads, dim), dtype=BF16, device="cuda")
        block.loopq_kv_write_rope(pool, 3, t, cu, spec(freqs(rot)), k, v, q, out)
        pools.append(pool)
        outs.append(out)
    assert torch.equal(pools[0], pools[1][-12:]) and torch.equal(outs[0], outs[1])
    assert pools[0].any() and not any(pools[1][at:at + 64].any() for at in range(0, pages - 12 - 64, 64))
    assert not pools[1][-76:-12].any()


@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("rot", [64, 54])
def test_what_is_not_turned_keeps_every_bit(lq, rot, layout):
    """Every bf16 there is as a value and in the part of a head that is not turned: the same bits (a NaN: a NaN), subnormal numbers among them."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16)
    tokens, heads, dim, page = 256, 4, 128, 32
    t = kv.KVTable(torch.arange(8, dtype=torch.int32, device="cuda")[None], i32([tokens]), torch.ones(8, dtype=torch.int32, device="cuda"))
    v = bits.repeat(2).view(BF16).view(tokens, heads, dim)  # 131072 places, 65536 patterns
    k = v.clone()
    k[..., :rot] = make((tokens, heads, rot), BF16, rot)
    pool = torch.zeros((8, 1, 2, heads, page, dim), dtype=BF16, device="cuda")
    q = torch.zeros_like(k)
    block.loopq_kv_write_rope(pool, 0, t, i32([0, tokens]), spec(freqs(rot), layout), k, v, k, q)
    alone = torch.zeros_like(k)
    block.loopq_rope(k, torch.arange(tokens, dtype=torch.int32, device="cuda"), spec(freqs(rot), layout), alone)

    def kept(got, want):
        nan = want.isnan()
        assert torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan]) and got[nan].isnan().all()

    def rows(at):  # [tokens][heads][dim] of the slab's keys or values
        return pool[:, 0, at].transpose(1, 2).reshape(tokens, heads, dim)
    kept(rows(1).contiguous(), v)
    for got in (rows(0), q, alone):
        kept(got[..., rot:].contiguous(), k[..., rot:].contiguous())


def test_replays_follow_what_the_table_holds(lq):
    """A captured write of a batch's next tokens, replayed as the rows grow."""
    rng = np.random.default_rng(11)
    rows, heads, dim, page = 5, 2, 64, 16
    pool = torch.zeros((60, 1, 2, heads, page, dim), dtype=BF16, device="cuda")
    table = torch.from_numpy(rng.permutation(60).astype(np.int32)[:50].reshape(5, 10)).cuda()
    t, cu, f = kv.KVTable(table, i32([0] * 5), torch.ones(60, dtype=torch.int32, device="cuda")), i32(range(6)), spec(freqs(64))
    q, k, v = (make((rows, h, dim), F32, 40 + i) for i, h in enumerate((4, heads, heads)))
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.loopq_kv_write_rope(pool, 0, t, cu, f, k, v, q, out)
    for n in ([1, 16, 17, 2, 160], [2, 17, 18, 100, 33], [3, 18, 161, 0, 34]):
        t.lens.copy_(i32(n))
        before = pool.clone()
        block.loopq_kv_write_rope(before, 0, t, cu, f, k, v, q, want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.view(torch.int16), before.view(torch.int16)) and torch.equal(out, want)
