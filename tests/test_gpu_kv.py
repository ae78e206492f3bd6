"""The paged cache's bookkeeping on the GPU against the plain references of
kv_reference.py: page indices, lengths and reference counts are whole numbers
and have to be equal; page contents move as they are, bit for bit."""

import random

import numpy as np
import pytest
import torch

import kv_reference as ref
from bit_ptq_looped_amd import kv

pytestmark = pytest.mark.gpu


def i32(v, shape=None):
    t = torch.tensor(v, dtype=torch.int32, device="cuda")
    return t if shape is None else t.reshape(shape)


def dev_table(table, lens, refs, width):
    return kv.KVTable(i32(table, (len(table), width)), i32(lens, (len(lens),)), i32(refs))


def host(t):
    torch.cuda.synchronize()
    return t.table.tolist(), t.lens.tolist(), t.refs.tolist()


def make_pool(pages, slabs, heads, page, dim, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bits = torch.randint(-32768, 32768, (pages, slabs, 2, heads, page, dim), dtype=torch.int16, device="cuda", generator=g)
    return bits.view(torch.bfloat16)  # any bits, NaN among them: contents move as they are


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def state(rng, rows, width, pages, page, shared=False):
    """Random rows over random pages; every page of a row held once (some twice if shared)."""
    order = list(range(pages))
    rng.shuffle(order)
    table, lens, refs = [], [], [0] * pages
    for _ in range(rows):
        n = rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, width * page)])
        n = min(n, width * page, len(order) * page)
        mine = [order.pop() for _ in range(-(-n // page))]
        for p in mine:
            refs[p] = 1
        table.append(mine + [-1] * (width - len(mine)))
        lens.append(n)
    if shared and rows > 1 and lens[0] >= page:  # a shared full page
        table[1][0] = table[0][0]
        lens[1] = page
        for p in table[1][1:]:
            if p >= 0:
                refs[p] -= 1
        table[1][1:] = [-1] * (width - 1)
        refs = [0] * pages
        for row in table:
            for p in row:
                if p >= 0:
                    refs[p] += 1
    return table, lens, refs


@pytest.mark.parametrize("rows,width,pages,page,inplace", [
    (1, 1, 1, 8, False), (3, 4, 40, 16, False), (3, 4, 40, 16, True), (64, 9, 1000, 32, False),
    (1500, 5, 9000, 16, True), (7, 700, 70000, 16, False), (2, 3, 4_000_000, 256, False)])
def test_reserve(lq, rows, width, pages, page, inplace):
    rng = random.Random(rows * 7 + pages)
    table, lens, refs = state(rng, rows, width, pages, page)
    refs[pages // 2] += 1  # a pinned page is not free
    grow = [min(rng.choice([0, 1, 1, page, rng.randint(0, width * page)]), width * page - n) for n in lens]
    grow[rng.randrange(rows)] = -3
    want = ref.reserve(table, lens, refs, page, grow)
    t = dev_table(table, lens, refs, width)
    out = t if inplace else kv.empty_table(rows, width, pages)
    info = torch.empty(2, dtype=torch.int32, device="cuda")
    kv.loopq_kv_reserve(t, page, i32(grow), out, info, kv.empty_pages_workspace(rows, pages))
    assert (*host(out), info.tolist()) == (want[0], want[1], want[2], want[3])


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kind", ["pages", "row"])
def test_reserve_is_all_or_nothing(lq, kind, inplace):
    page, width, pages = 16, 4, 12
    table = [[3, 5, -1, -1], [7, -1, -1, -1], [-1] * 4]
    refs = [1 if p in (0, 3, 5, 7) else 0 for p in range(pages)]  # page 0 is pinned: 8 are free, 9 needed
    lens = [20, 16, 0]
    grow = [40, 48, 64] if kind == "pages" else [1, 49, 0]
    want = ref.reserve(table, lens, refs, page, grow)
    assert want[3][0] == (1 if kind == "pages" else 2)
    t = dev_table(table, lens, refs, width)
    out = t if inplace else kv.empty_table(3, width, pages)
    info = torch.empty(2, dtype=torch.int32, device="cuda")
    kv.loopq_kv_reserve(t, page, i32(grow), out, info, kv.empty_pages_workspace(3, pages))
    assert (*host(out), info.tolist()[0]) == (table, lens, refs, want[3][0])
    if kind == "pages":
        assert info.tolist()[1] == want[3][1]


@pytest.mark.parametrize("rows,out_rows,width,pages,page,slabs,heads,dim", [
    (1, 1, 1, 3, 8, 1, 1, 64), (1, 5, 3, 20, 16, 2, 3, 96), (4, 8, 6, 64, 32, 3, 2, 128), (40, 25, 7, 400, 16, 1, 5, 64),
    (8, 8, 5, 64, 128, 4, 2, 128), (30, 1100, 3, 1300, 8, 1, 1, 64), (3, 2, 900, 70000, 8, 1, 1, 64)])
def test_fork(lq, rows, out_rows, width, pages, page, slabs, heads, dim):
    rng = random.Random(rows + 31 * out_rows)
    table, lens, refs = state(rng, rows, width, pages, page, shared=True)
    pinned = next((table[b][n // page] for b, n in enumerate(lens) if n % page), None)
    if pinned is not None:
        refs[pinned] += 1  # somebody else holds a partial page: every child gets a copy
    parent = [rng.choice([-1, rng.randrange(rows), rng.randrange(rows), rows + 5]) for _ in range(out_rows)]
    want = ref.fork(table, lens, refs, page, parent)
    pool = make_pool(pages, slabs, heads, page, dim)
    expect = pool.clone()
    for src, dst in want[4]:
        expect[dst] = pool[src]
    t, out = dev_table(table, lens, refs, width), kv.empty_table(out_rows, width, pages)
    info = torch.empty(2, dtype=torch.int32, device="cuda")
    kv.loopq_kv_fork(pool, t, i32(parent), out, info, kv.empty_pages_workspace(max(rows, out_rows), pages))
    assert (*host(out), info.tolist()) == (want[0], want[1], want[2], want[3])
    assert same_bits(pool, expect)
    assert host(t) == (table, lens, refs)  # the old table stays as it was


def test_fork_without_free_pages_changes_nothing(lq):
    page, pages = 16, 3
    table, lens, refs = [[0, 1], [2, -1]], [20, 5], [1, 1, 1]
    pool = make_pool(pages, 1, 1, page, 64)
    before = pool.clone()
    t, out = dev_table(table, lens, refs, 2), kv.empty_table(3, 2, pages)
    info = torch.empty(2, dtype=torch.int32, device="cuda")
    kv.loopq_kv_fork(pool, t, i32([0, 0, 1]), out, info, kv.empty_pages_workspace(3, pages))
    assert (*host(out), info.tolist()) == ([[-1, -1]] * 3, [0, 0, 0], refs, [1, 1])
    assert same_bits(pool, before)


def test_fork_to_no_rows_frees_everything(lq):
    t = dev_table([[0, 2]], [20], [1, 0, 1], 2)
    out = kv.KVTable(torch.empty((0, 2), dtype=torch.int32, device="cuda"), i32([], (0,)), i32([9, 9, 9]))
    info = torch.empty(2, dtype=torch.int32, device="cuda")
    kv.loopq_kv_fork(make_pool(3, 1, 1, 16, 64), t, i32([], (0,)), out, info, kv.empty_pages_workspace(1, 3))
    assert out.refs.tolist() == [0, 0, 0] and info.tolist() == [0, 0]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("rows,width,pages,page,window,sinks", [
    (1, 1, 1, 8, 1, 0), (5, 12, 80, 16, 1, 0), (5, 12, 80, 16, 33, 17), (40, 30, 1400, 32, 100, 4), (6, 9, 99, 8, 1000, 5),
    (9, 40, 400, 16, 16, 16), (100, 200, 3000, 16, 300, 40)])
def test_trim(lq, rows, width, pages, page, window, sinks, inplace):
    rng = random.Random(rows + window)
    table, lens, refs = state(rng, rows, width, pages, page, shared=True)
    want = ref.trim(table, lens, refs, page, window, sinks)
    t = dev_table(table, lens, refs, width)
    out = t if inplace else kv.empty_table(rows, width, pages)
    kv.loopq_kv_trim(t, page, window, sinks, out)
    assert host(out) == want


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("rows,width,pages,page,slabs,heads,dim,keep", [
    (1, 1, 1, 8, 1, 1, 64, 0.5), (3, 5, 64, 16, 2, 3, 96, 0.4), (20, 6, 300, 16, 3, 2, 128, 0.7),
    (5, 5, 65, 32, 1, 1, 64, 1.0), (4, 4, 128, 8, 1, 2, 64, 0.0), (9, 100, 70000, 8, 1, 1, 64, 0.9)])
def test_compact(lq, rows, width, pages, page, slabs, heads, dim, keep, inplace):
    rng = random.Random(rows + pages)
    table, lens, refs = state(rng, rows, width, pages, page)
    for row in table:  # freed in the middle
        for k, p in enumerate(row):
            if p >= 0 and rng.random() > keep:
                row[k] = -1
                refs[p] = 0
    free = [p for p in range(pages) if refs[p] == 0]
    for p in free[-2:]:
        refs[p] = 1 + p % 3  # pinned outside the table
    want = ref.compact(table, lens, refs)
    pool = make_pool(pages, slabs, heads, page, dim)
    expect = pool.clone()
    for src, dst in want[5]:
        expect[dst] = pool[src]
    t = dev_table(table, lens, refs, width)
    out = t if inplace else kv.empty_table(rows, width, pages)
    page_map, info = torch.empty(pages, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    kv.loopq_kv_compact(pool, t, out, page_map, info, kv.empty_pages_workspace(rows, pages))
    assert host(out) == (want[0], want[1], want[2])
    assert page_map.tolist() == want[3] and info.tolist() == want[4]
    assert same_bits(pool, expect)


def test_compact_of_an_empty_and_of_a_full_pool(lq):
    for refs, table in (([0] * 64, [[-1, -1]]), ([1] * 64, [[63, 0]])):
        t = dev_table(table, [16], refs, 2)
        pool = make_pool(64, 1, 1, 8, 64)
        before = pool.clone()
        page_map, info = torch.empty(64, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
        kv.loopq_kv_compact(pool, t, t, page_map, info, kv.empty_pages_workspace(1, 64))
        assert host(t) == (table, [16], refs) and info.tolist() == [sum(refs), 0] and same_bits(pool, before)


@pytest.mark.parametrize("dim,heads,page,slabs", [(64, 1, 8, 1), (96, 5, 64, 3), (128, 2, 256, 2)])
def test_copy_pages(lq, dim, heads, page, slabs):
    a, b = make_pool(9, slabs, heads, page, dim, 1), make_pool(5, slabs, heads, page, dim, 2)
    want = b.clone()
    want[4], want[0] = a[8], a[2]
    kv.loopq_kv_copy_pages(a, i32([8, -1, 2, 9, 3]), b, i32([4, 1, 0, 2, 5]))  # pairs outside a pool are skipped
    assert same_bits(b, want)
    want = a.clone()
    want[1] = a[7]
    kv.loopq_kv_copy_pages(a, i32([7]), a, i32([1]))
    assert same_bits(a, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim,heads,page,slabs,slab,extra", [(64, 1, 8, 1, 0, 0), (96, 5, 32, 3, 2, 16), (128, 3, 16, 2, 0, 8)])
def test_write(lq, dtype, dim, heads, page, slabs, slab, extra):
    g = torch.Generator(device="cuda").manual_seed(dim)
    width, pages = 4, 30
    lens, news = [3 * page + 1, 5, 0, page, 2], [2 * page, 5, 0, 1, 4]  # row 4 has fewer tokens than are given
    table = [[20, 3, 9, 11], [5, -1, -1, -1], [-1] * 4, [7, -1, -1, -1], [8, -1, -1, -1]]
    table[0][2] = -1  # tokens without a page are dropped
    total = sum(news)
    rows = torch.randn((total + 3, 2 * heads * dim + extra), generator=g, device="cuda").to(dtype)  # 3 more than cu covers
    k = rows[:, :heads * dim].unflatten(1, (heads, dim))
    v = rows[:, heads * dim:2 * heads * dim].unflatten(1, (heads, dim))
    pool = make_pool(pages, slabs, heads, page, dim)
    want = pool.clone()
    cu = [sum(news[:b]) for b in range(len(news) + 1)]
    for b, (n, m) in enumerate(zip(lens, news)):
        for i in range(m):
            pos = n - m + i
            if pos < 0 or table[b][pos // page] < 0:
                continue
            for a, x in ((0, k), (1, v)):
                want[table[b][pos // page], slab, a, :, pos % page] = x[cu[b] + i].to(torch.bfloat16)
    t = dev_table(table, lens, [0] * pages, width)
    kv.loopq_kv_write(pool, slab, t, i32(cu), k, v)
    assert same_bits(pool, want)


def test_a_long_run_keeps_every_token(lq):
    """Reserve, write, fork, trim and compact in turn: each row's visible tokens stay what was written."""
    rng = random.Random(5)
    page, pages, width, dim, window, sinks = 8, 60, 12, 64, 20, 3
    pool = make_pool(pages, 1, 1, page, dim)
    cur, nxt = kv.new_table(3, width, pages), kv.empty_table(3, width, pages)
    ws, info = kv.empty_pages_workspace(3, pages), torch.empty(2, dtype=torch.int32, device="cuda")
    page_map = torch.empty(pages, dtype=torch.int32, device="cuda")
    tokens, stamp = [[], [], []], 0
    for step in range(40):
        grow = [rng.choice([0, 1, 1, 2, 9]) for _ in range(3)]
        grow = [g if len(r) + g <= width * page else 0 for g, r in zip(grow, tokens)]
        kv.loopq_kv_reserve(cur, page, i32(grow), cur, info, ws)
        assert info.tolist()[0] == 0
        new = []
        for r, g in zip(tokens, grow):
            for _ in range(g):
                stamp += 1
                r.append(stamp)
                new.append(stamp)
        if new:
            x = i32(new).to(torch.float32)[:, None, None].expand(-1, 1, dim).contiguous()
            kv.loopq_kv_write(pool, 0, cur, i32([sum(grow[:b]) for b in range(4)]), x, -x)
        if step % 3 == 1:
            parent = [rng.randrange(3) for _ in range(3)] if step % 2 else [rng.choice([-1, 0]), 1, 2]
            kv.loopq_kv_fork(pool, cur, i32(parent), nxt, info, ws)
            assert info.tolist()[0] == 0
            cur, nxt = nxt, cur
            tokens = [list(tokens[p]) if p >= 0 else [] for p in parent]
        if step % 4 == 2:
            kv.loopq_kv_trim(cur, page, window, sinks, cur)
        if step % 5 == 3:
            kv.loopq_kv_compact(pool, cur, cur, page_map, info, ws)
        table, lens, refs = host(cur)
        assert lens == [len(r) for r in tokens]
        held = [0] * pages
        for row in table:
            for p in row:
                if p >= 0:
                    held[p] += 1
        assert held == refs
        if step % 5 == 3:
            assert all(p < info.tolist()[0] for row in table for p in row)
        for row, r in zip(table, tokens):
            for j, want in enumerate(r):
                if j < sinks or j >= len(r) - window + 1:
                    got = pool[row[j // page], 0, :, 0, j % page, 0].float().tolist()
                    exact = float(torch.tensor(float(want)).to(torch.bfloat16))
                    assert row[j // page] >= 0 and got == [exact, -exact]


def test_bookkeeping_in_a_graph(lq):
    """The whole sequence captured once; each replay equals the eager run."""
    page, pages, width = 16, 50, 6
    pool = make_pool(pages, 2, 1, page, 64)
    first = pool.clone()
    table, lens, refs = [[4, 9, -1, -1, -1, -1], [6, 2, 30, 41, -1, -1]], [20, 55], [0] * pages
    for p in (4, 9, 6, 2, 30, 41):
        refs[p] = 1
    t = dev_table(table, lens, refs, width)
    a, b = kv.empty_table(2, width, pages), kv.empty_table(3, width, pages)
    grow, parent, cu = i32([1, 30]), i32([1, 0, 1]), i32([0, 1, 31])
    k = torch.randn((31, 1, 64), device="cuda")
    info, ws = torch.empty(2, dtype=torch.int32, device="cuda"), kv.empty_pages_workspace(3, pages)
    page_map = torch.empty(pages, dtype=torch.int32, device="cuda")

    def step():
        kv.loopq_kv_reserve(t, page, grow, a, info, ws)
        kv.loopq_kv_write(pool, 1, a, cu, k, k)
        kv.loopq_kv_fork(pool, a, parent, b, info, ws)
        kv.loopq_kv_trim(b, page, 17, 4, b)
        kv.loopq_kv_compact(pool, b, b, page_map, info, ws)

    step()
    want, eager = host(b), pool.clone()
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        with torch.cuda.graph(graph, stream=cap):
            step()
    torch.cuda.current_stream().wait_stream(cap)
    for _ in range(3):
        pool.copy_(first)
        b.table.fill_(7)
        b.refs.fill_(7)
        graph.replay()
        assert host(b) == want and same_bits(pool, eager)
        pool.copy_(first)
        step()
        assert host(b) == want and same_bits(pool, eager)


def test_timing_hooks_count_calls(lq):
    from bit_ptq_looped_amd import loopq
    pool = make_pool(8, 1, 1, 16, 64)
    pool.zero_()
    t = dev_table([[3, -1], [5, -1]], [9, 16], [0, 0, 0, 1, 0, 1, 0, 0], 2)
    info, q = torch.empty(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 2, 64), device="cuda")
    loopq.loopq_timing_reset()
    loopq.loopq_timing_enable(True)
    kv.loopq_kv_reserve(t, 16, i32([1, 1]), t, info, kv.empty_pages_workspace(2, 8))
    kv.loopq_kv_trim(t, 16, 8, 0, t)
    kv.loopq_attn_decode(pool, 0, t, q, torch.empty_like(q), kv.empty_attn_workspace(pool, 2, 2, 2), 1.0)
    loopq.loopq_timing_enable(False)
    times = loopq.loopq_timing_read()
    assert times[loopq.LOOPQ_KERNEL_KV][1] == 2 and times[loopq.LOOPQ_KERNEL_ATTN][1] == 1
    assert times[loopq.LOOPQ_KERNEL_KV][0] > 0 and times[loopq.LOOPQ_KERNEL_ATTN][0] > 0
