"""Attention over the paged cache on the GPU against kv_reference.attend (64
bits).  Every place that no query may see holds NaN: pages outside the tables,
tokens past the rows' lengths, tokens outside every window."""

import math
import random

import numpy as np
import pytest
import torch

import kv_reference as ref
from bit_ptq_looped_amd import kv

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, lens, heads=2, group=1, dim=128, page=16, window=0, sinks=0, dtype="bf16", slabs=2, slab=1,
                 news=None, width=None, seed=0, qmul=1.5, holes=(), trash=True):
        self.lens, self.news, self.page, self.window, self.sinks = lens, news, page, window, sinks
        self.dtype, self.slab, self.dim, self.hq = dtype, slab, dim, heads * group
        rng = random.Random(seed + sum(lens))
        self.width = width or max(1, max(-(-n // page) for n in lens)) + rng.randint(0, 2)
        count = [min(-(-max(n, 0) // page), self.width) for n in lens]
        pages = sum(count) + 3
        order = list(range(pages))
        rng.shuffle(order)
        self.table = []
        for c in count:
            mine = [order.pop() for _ in range(c)]
            self.table.append(mine + [-1] * (self.width - c))
        for b, k in holes:
            self.table[b][k] = rng.choice([-1, pages, pages + 1000, -2 ** 31, 2 ** 31 - 1])
        g = torch.Generator().manual_seed(seed + 17)
        pool = torch.full((pages, slabs, 2, heads, page, dim), math.nan)
        self.q_tokens = sum(news) if news is not None else len(lens)
        for b, n in enumerate(lens):
            top = min(n, self.width * page)
            first = top - (news[b] if news is not None else 1)
            for k in range(self.width):
                p = self.table[b][k]
                if not 0 <= p < pages or k * page >= top:
                    continue
                m = min(page, top - k * page)
                x = torch.randn((slabs, 2, heads, m, dim), generator=g)
                if trash and window:
                    for i in range(m):  # what no query sees
                        if k * page + i <= first - window and k * page + i >= sinks:
                            x[:, :, :, i] = math.nan
                pool[p, :, :, :, :m] = x
        self.pool = pool.to(torch.bfloat16).cuda()
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        self.q = (qmul * torch.randn((self.q_tokens, self.hq, dim), generator=g)).to(dt).cuda()
        self.scale = 1.0 / math.sqrt(dim)
        self.t = kv.KVTable(i32(self.table).reshape(len(lens), self.width), i32(lens), torch.zeros(pages, dtype=torch.int32, device="cuda"))
        if news is not None:
            self.cu = [sum(news[:b]) for b in range(len(news) + 1)]

    def run(self, q=None, out=None, scale=None):
        q = self.q if q is None else q
        out = torch.full_like(q, 7.0) if out is None else out
        ws = kv.empty_attn_workspace(self.pool, q.shape[0], self.hq, len(self.lens))
        ws.fill_(255)  # NaN everywhere
        scale = self.scale if scale is None else scale
        if self.news is None:
            kv.loopq_attn_decode(self.pool, self.slab, self.t, q, out, ws, scale, self.window, self.sinks)
        else:
            kv.loopq_attn_prefill(self.pool, self.slab, self.t, i32(self.cu), q, out, ws, scale, self.window, self.sinks)
        torch.cuda.synchronize()
        return out

    def queries(self):
        """(query token, row, position)"""
        for b, n in enumerate(self.lens):
            n = ref.clamp_len(n, self.width, self.page)
            if self.news is None:
                yield b, b, n - 1
            else:
                for i in range(self.news[b]):
                    yield self.cu[b] + i, b, n - self.news[b] + i

    def check(self, out=None, scale=None, some=None):
        out = self.run(scale=scale) if out is None else out
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        pool, q = self.pool.double().cpu().numpy(), self.q.double().cpu().numpy()
        every = list(self.queries())
        if some and len(every) > some:
            rng = random.Random(1)
            every = rng.sample(every, some) + every[:2] + every[-2:]
        for t, b, p in every:
            w, bound, absum = ref.attend(q[t], p, pool, self.slab, self.table[b], self.scale if scale is None else scale,
                                         self.window, self.sinks)
            tol = ref.tolerance(w, bound, absum, self.dtype)
            err = np.abs(got[t] - w)
            assert (err <= tol).all(), (t, b, p, float((err - tol).max()), float(err.max()))
        return out


BOTH = pytest.mark.parametrize("dtype", ["bf16", "f32"])


@BOTH
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 4), (1, 7), (2, 16), (1, 19), (1, 40)])
def test_decode_head_layouts(lq, dim, heads, group, dtype):
    Case([45, 1, 130, 16], heads, group, dim, 16, dtype=dtype).check()


@BOTH
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_decode_lengths(lq, page, dtype):
    Case([0, 1, 2, 7, 8, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300], 2, 2, 96, page, dtype=dtype).check()


@BOTH
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (17, 4), (100, 40), (64, 64), (300, 5), (1000, 0), (30, 1000)])
def test_decode_window_and_sinks(lq, window, sinks, dtype):
    Case([0, 1, 5, 30, 64, 101, 300, 517], 2, 3, 64, 16, window, sinks, dtype=dtype).check()


@BOTH
def test_decode_splits_a_long_row(lq, dtype):
    Case([5003, 9, 20001], 1, 2, 128, 32, dtype=dtype).check()
    Case([30011], 1, 8, 128, 64, window=9000, sinks=70, dtype=dtype).check()


@BOTH
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 4), (1, 7), (2, 16), (1, 19), (1, 40)])
def test_decode_head_layouts_in_a_long_table(lq, dim, heads, group, dtype):
    """Room for long rows: the work is cut into pieces, whatever the rows' lengths."""
    Case([45, 1, 0, 130, 16, 700], heads, group, dim, 16, dtype=dtype, width=190).check()


@BOTH
@pytest.mark.parametrize("page", [8, 64, 256])
def test_decode_lengths_in_a_long_table(lq, page, dtype):
    Case([0, 1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 255, 257, 300], 2, 2, 96, page, dtype=dtype, width=2600 // page).check()


@BOTH
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (17, 4), (64, 64), (300, 5), (30, 1000)])
def test_decode_window_and_sinks_in_a_long_table(lq, window, sinks, dtype):
    Case([0, 1, 5, 30, 64, 301, 517, 2011], 2, 3, 64, 16, window, sinks, dtype=dtype, width=140).check()


@BOTH
def test_decode_holes_in_a_long_table(lq, dtype):
    c = Case([900, 40, 0, 2000, 3], 2, 2, 64, 16, dtype=dtype, width=140, holes=[(0, 2), (0, 55), (1, 0), (1, 1), (1, 2), (3, 12), (3, 124)])
    c.check()
    c.check(scale=0.0)
    c.check(scale=-0.3)


@BOTH
def test_decode_of_mostly_empty_rows(lq, dtype):
    """Rows of a batch that wait for work: their results are 0."""
    c = Case([0] * 700 + [900] + [0] * 120, 1, 2, 64, 16, dtype=dtype, width=140)
    out = c.check(some=30)
    assert not out[:700].any() and not out[701:].any()


@BOTH
def test_decode_many_rows(lq, dtype):
    rng = random.Random(2)
    Case([rng.randint(0, 400) for _ in range(333)], 2, 1, 64, 16, dtype=dtype).check(some=60)


@BOTH
@pytest.mark.parametrize("news", [None, [40, 6, 20, 3]])
def test_entries_that_are_no_page(lq, news, dtype):
    """Holes in a row, a row whose every page is gone, lengths past the table or negative."""
    c = Case([100, 40, 200, 3], 2, 2, 64, 16, dtype=dtype, news=news, holes=[(0, 2), (0, 3), (1, 0), (1, 1), (1, 2), (2, 12), (2, 0)])
    c.check()
    c.lens = [100, -7, 2 ** 31 - 1, 3]
    c.t = c.t._replace(lens=i32(c.lens))
    c.check()


@BOTH
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 4), (1, 7), (1, 19)])
def test_prefill_head_layouts(lq, dim, heads, group, dtype):
    Case([70, 1, 200, 33], heads, group, dim, 16, dtype=dtype, news=[70, 1, 50, 20]).check()


@BOTH
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_prefill_lengths(lq, page, dtype):
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 255, 257, 300]
    Case(lens, 1, 2, 96, page, dtype=dtype, news=[0, 1, 2, 1, 16, 17, 30, 33, 1, 64, 127, 128, 129, 2, 257, 131]).check()


@BOTH
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (17, 4), (100, 40), (64, 64), (300, 5), (1000, 0), (30, 1000)])
def test_prefill_window_and_sinks(lq, window, sinks, dtype):
    Case([3, 64, 300, 517], 2, 1, 64, 16, window, sinks, dtype=dtype, news=[3, 20, 300, 260]).check()


@BOTH
def test_prefill_of_a_chunk_splits_a_long_row(lq, dtype):
    Case([5003, 9, 12001], 1, 1, 128, 32, dtype=dtype, news=[150, 3, 33]).check(some=60)
    Case([20011], 2, 2, 64, 64, window=7000, sinks=70, dtype=dtype, news=[70]).check(some=40)


@BOTH
def test_prefill_larger(lq, dtype):
    Case([1500, 700], 4, 1, 128, 16, dtype=dtype, news=[1500, 333]).check(some=60)


@BOTH
@pytest.mark.parametrize("window,sinks", [(0, 0), (5000, 70)])
def test_prefill_walks_many_tiles(lq, window, sinks, dtype):
    """Work-groups that go over more than 64 tiles of keys each, with pages missing."""
    Case([6100], 1, 40, 64, 16, window, sinks, dtype=dtype, news=[1500], holes=[(0, 3), (0, 200), (0, 301)]).check(some=25)


@BOTH
def test_more_queries_than_tokens(lq, dtype):
    """Queries at negative positions see nothing: 0."""
    c = Case([5, 40], 1, 2, 64, 16, dtype=dtype, news=[9, 40])
    out = c.check()
    assert not out[:4].any()


@BOTH
@pytest.mark.parametrize("news", [None, [90, 3]])
@pytest.mark.parametrize("scale", [0.0, -0.3, 40.0])
def test_scales(lq, scale, news, dtype):
    Case([130, 77], 2, 2, 64, 16, dtype=dtype, news=news).check(scale=scale)


@BOTH
@pytest.mark.parametrize("news", [None, [150, 20]])
def test_large_scores(lq, news, dtype):
    Case([150, 300], 2, 2, 128, 16, dtype=dtype, news=news, qmul=60.0).check()


@BOTH
@pytest.mark.parametrize("window", [0, 40])
def test_a_value_that_some_queries_see(lq, window, dtype):
    """NaN or infinity in a token's values reaches the queries that see it, and no other."""
    c = Case([200], 2, 1, 64, 16, window, 2, dtype=dtype, news=[200])
    j = 100
    c.pool[c.table[0][j // 16], c.slab, 1, 0, j % 16, 5] = math.nan
    c.pool[c.table[0][j // 16], c.slab, 1, 1, j % 16, 63] = math.inf
    got = c.run().float().cpu().numpy()
    sees = np.array([p >= j and (not window or p - j < window) for p in range(200)])
    assert (np.isnan(got[:, 0, 5]) == sees).all() and (np.isinf(got[:, 1, 63]) == sees).all()
    got[sees, 0, 5] = 0
    got[sees, 1, 63] = 0
    assert np.isfinite(got).all()
    c.pool[c.table[0][j // 16], c.slab, 1, :, j % 16] = 0.25
    w = c.run().float().cpu().numpy()
    assert np.array_equal(got[~sees], w[~sees])


@BOTH
def test_a_value_hidden_from_the_only_query(lq, dtype):
    c = Case([200], 1, 4, 64, 16, 40, 2, dtype=dtype, trash=False)
    want = c.check().clone()
    for j in (2, 100, 159):
        c.pool[c.table[0][j // 16], c.slab, :, :, j % 16] = math.inf
    assert torch.equal(c.run(), want)


@BOTH
@pytest.mark.parametrize("width", [13, 140])
@pytest.mark.parametrize("news", [None, [1]])
def test_a_key_of_minus_infinity(lq, news, width, dtype):
    """A score of -infinity is a weight of 0, as a score of -1e30 is."""
    c = Case([200], 1, 1, 64, 16, dtype=dtype, news=news, width=width)
    for j in (0, 77, 199):
        c.pool[c.table[0][j // 16], c.slab, 0, 0, j % 16, 9] = -1e30 * torch.sign(c.q[0, 0, 9])
    want = c.run()
    assert torch.isfinite(want).all()
    for j in (0, 77, 199):
        c.pool[c.table[0][j // 16], c.slab, 0, 0, j % 16, 9] = -math.inf * torch.sign(c.q[0, 0, 9])
    assert torch.equal(c.run(), want)


@BOTH
@pytest.mark.parametrize("news", [None, [130, 9]])
def test_slices_of_wider_rows(lq, news, dtype):
    c = Case([130, 40], 2, 2, 64, 16, dtype=dtype, news=news)
    wide_q = torch.full((c.q_tokens, 3 * c.hq * 64 + 8), math.nan, dtype=c.q.dtype, device="cuda")
    wide_o = torch.full((c.q_tokens, c.hq * 64 + 16), 5.0, dtype=c.q.dtype, device="cuda")
    wide_q[:, c.hq * 64:2 * c.hq * 64] = c.q.flatten(1)
    out = wide_o[:, 8:8 + c.hq * 64].unflatten(1, (c.hq, 64))
    got = c.run(wide_q[:, c.hq * 64:2 * c.hq * 64].unflatten(1, (c.hq, 64)), out)
    assert torch.equal(got, c.run())
    assert (wide_o[:, :8] == 5).all() and (wide_o[:, 8 + c.hq * 64:] == 5).all()


def test_queries_past_the_last_row_are_left_alone(lq):
    c = Case([30, 20], 1, 1, 64, 16, news=[10, 5])
    want = c.run()
    q = torch.cat([c.q, c.q[:4]])
    got = c.run(q)
    assert torch.equal(got[:15], want) and (got[15:] == 7).all()


def test_prefix_that_does_not_ascend_stays_inside(lq):
    """Not a valid call, but no address depends on cu: nothing outside out and the workspace is written."""
    c = Case([900] * 40, 1, 1, 64, 16, news=[10] * 40)
    need = kv.loopq_attn_workspace_bytes(400, 1, 40, 64)
    big = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    cu = i32([0, 400] * 20 + [0])
    out = torch.full((500, 1, 64), 7.0, dtype=c.q.dtype, device="cuda")
    kv.loopq_attn_prefill(c.pool, c.slab, c.t, cu, c.q, out[:400], big[:need], c.scale)
    kv.loopq_attn_prefill(c.pool, c.slab, c.t, i32([-5, 2 ** 31 - 1, -2 ** 31] * 13 + [0, 9]), c.q, out[:400], big[:need], c.scale)
    torch.cuda.synchronize()
    assert (big[need:] == 77).all() and (out[400:] == 7).all()


@BOTH
@pytest.mark.parametrize("news", [None, [300, 64, 1]])
def test_same_bits_every_time_and_on_another_stream(lq, news, dtype):
    c = Case([3000, 64, 700], 2, 4, 128, 16, dtype=dtype, news=news)
    want = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run()
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("news", [None, [200, 64]])
def test_in_a_graph_with_lengths_that_change(lq, news):
    """Lengths are read on the device: one captured call serves every step."""
    c = Case([900, 64], 2, 2, 128, 16, news=news)
    out, ws = torch.empty_like(c.q), kv.empty_attn_workspace(c.pool, c.q_tokens, c.hq, 2)
    cu = i32(c.cu) if news else None

    def step():
        if news is None:
            kv.loopq_attn_decode(c.pool, c.slab, c.t, c.q, out, ws, c.scale)
        else:
            kv.loopq_attn_prefill(c.pool, c.slab, c.t, cu, c.q, out, ws, c.scale)

    step()
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        with torch.cuda.graph(graph, stream=cap):
            step()
    torch.cuda.current_stream().wait_stream(cap)
    for lens in ([900, 64], [201, 64], [777, 64]):
        c.t.lens.copy_(i32(lens))
        step()
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_pages_past_four_gigabytes(lq):
    """A pool whose last pages lie beyond 2^32 bytes and 2^32 elements from its start."""
    page, heads, dim, slabs = 256, 4, 128, 16
    per = slabs * 2 * heads * page * dim
    pages = 2 ** 32 // per + 3
    pool = torch.empty((pages, slabs, 2, heads, page, dim), dtype=torch.bfloat16, device="cuda")
    c = Case([400, 300], heads, 1, dim, page, slabs=2)
    t = kv.KVTable(i32([[pages - 1, 0], [pages - 2, 1]]), i32([0, 0]), torch.zeros(pages, dtype=torch.int32, device="cuda"))
    t = t._replace(lens=i32([400, 300]))
    for b in range(2):
        for k in range(2):
            pool[t.table[b, k].item(), 15] = c.pool[c.table[b][k], c.slab]
    out = torch.empty_like(c.q)
    ws = kv.empty_attn_workspace(pool, 2, heads, 2)
    kv.loopq_attn_decode(pool, 15, t, c.q, out, ws, c.scale)
    assert torch.equal(out, c.run())
    cu, q = i32([0, 30, 60]), c.q.repeat_interleave(30, 0).contiguous()
    a, b = torch.empty_like(q), torch.empty_like(q)
    ws = kv.empty_attn_workspace(pool, 60, heads, 2)
    kv.loopq_attn_prefill(pool, 15, t, cu, q, a, ws, c.scale)
    kv.loopq_attn_prefill(c.pool, c.slab, c.t, cu, q, b, ws, c.scale)
    assert torch.equal(a, b)
    k = torch.randn((2, heads, dim), device="cuda")
    kv.loopq_kv_write(pool, 15, t, i32([0, 1, 2]), k, -k)
    assert torch.equal(pool[t.table[0, 1].item(), 15, 0, :, 399 - 256], k[0].to(torch.bfloat16))
    kv.loopq_kv_copy_pages(pool, i32([pages - 1]), pool, i32([pages - 3]))
    assert torch.equal(pool[pages - 3, 15], pool[pages - 1, 15])


def test_decode_of_more_items_than_one_launch_has_work_groups_for(lq):
    """8192 rows of 1024 heads, in a table with room for 1024 tokens: a work-group an item would be 2^32 work-items."""
    lens = [i % 37 for i in range(32)]
    c = Case(lens, 1024, 1, 64, 8, slabs=1, slab=0, width=126)
    assert 512 < 8 * c.width <= 2048
    t = kv.KVTable(c.t.table.repeat(256, 1), c.t.lens.repeat(256), c.t.refs)
    q = c.q.repeat(256, 1, 1)
    out = torch.full_like(q, 7.0)
    kv.loopq_attn_decode(c.pool, 0, t, q, out, kv.empty_attn_workspace(c.pool, 8192, 1024, 8192), c.scale)
    pool, q32 = c.pool.double().cpu().numpy(), c.q.double().cpu().numpy()
    each = [ref.attend(q32[b], n - 1, pool, 0, c.table[b], c.scale, 0, 0) for b, n in enumerate(lens)]
    want = torch.tensor(np.stack([w for w, _, _ in each]), device="cuda")
    tol = torch.tensor(np.stack([ref.tolerance(*x, "bf16") for x in each]), device="cuda")
    assert all(((some.double() - want).abs() <= tol).all() for some in out.split(32))


@BOTH
@pytest.mark.parametrize("window,group", [(0, 1), (0, 3), (90, 1)])
def test_keys_that_a_query_does_not_see_leave_no_trace(lq, window, group, dtype):
    """Not even in the last bit, where queries beside it see them and their scores are large."""
    c = Case([200, 130], 2, group, 64, 16, window, 3, dtype=dtype, news=[200, 100], trash=False)
    want = c.run()
    j = 100
    for b in range(2):
        c.pool[c.table[b][j // 16], c.slab, 0, :, j % 16] *= 40
        c.pool[c.table[b][j // 16], c.slab, 1, :, j % 16] *= -3
    got = c.run()
    sees = torch.tensor([p >= j and (not window or p - j < window) for _, _, p in c.queries()], device="cuda")
    assert torch.equal(got[~sees], want[~sees])
    assert not torch.equal(got[sees], want[sees])


@BOTH
@pytest.mark.parametrize("lens,news,width", [([300], None, 19), ([300], None, 140), ([5000], None, 320), ([300], [300], 20), ([5000], [40], 320)])
def test_values_that_are_not_finite_stay_so_whatever_their_weight(lq, lens, news, width, dtype):
    """Scores fall from one end of the row to the other so that weights are 0 in 32 bits at the far end."""
    c = Case(lens, 2, 1, 64, 16, dtype=dtype, news=news, width=width)
    n = lens[0]
    for j in range(n):  # scores from 0 down to -10 n, the largest at the row's last token
        c.pool[c.table[0][j // 16], c.slab, 0, :, j % 16] = 0
        c.pool[c.table[0][j // 16], c.slab, 0, :, j % 16, 0] = -80.0 * (n - 1 - j)
    c.q[:, :, 0] = 1
    want = c.run()
    assert torch.isfinite(want).all()
    odd = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
    for j, col, value in ((0, 3, math.nan), (1, 40, math.inf), (n // 2, 41, -math.inf), (n - 1, 63, math.inf)):
        c.pool[c.table[0][j // 16], c.slab, 1, :, j % 16, col] = value
        for t, _, p in c.queries():
            odd[t, :, col] |= p >= j
    got = c.run()
    assert torch.equal(~torch.isfinite(got), odd)
    assert torch.equal(got[~odd], want[~odd])


@BOTH
@pytest.mark.parametrize("news,width", [(None, 13), (None, 140), ([200], 13)])
def test_scores_that_are_not_finite(lq, news, width, dtype):
    """All scores -infinity: 0; one of +infinity or NaN: NaN in every column of that head."""
    c = Case([200], 3, 1, 64, 16, dtype=dtype, news=news, width=width, seed=5)
    c.q[:, :, 9] = 1
    want = c.run()
    for j in range(200):
        c.pool[c.table[0][j // 16], c.slab, 0, 0, j % 16, 9] = -math.inf
    c.pool[c.table[0][100 // 16], c.slab, 0, 1, 100 % 16, 9] = math.inf
    got = c.run()
    sees = torch.tensor([p >= 100 for _, _, p in c.queries()], device="cuda")
    assert not got[:, 0].any()
    assert got[sees, 1].isnan().all() and torch.equal(got[~sees, 1], want[~sees, 1])
    assert torch.equal(got[:, 2], want[:, 2])
    c.pool[c.table[0][100 // 16], c.slab, 0, 1, 100 % 16, 9] = math.nan
    got = c.run()
    assert got[sees, 1].isnan().all() and torch.equal(got[~sees, 1], want[~sees, 1])


@BOTH
@pytest.mark.parametrize("lens,news,width", [([400], None, 26), ([400], None, 140), ([400], [400], 26), ([2000, 300], [90, 300], 130)])
def test_large_values(lq, lens, news, width, dtype):
    """Values whose magnitudes add up to less than 2^119: a power of two, which scales every sum exactly."""
    c = Case(lens, 2, 2, 64, 16, dtype=dtype, news=news, width=width, qmul=4.0)
    want = c.run()
    c.pool[:, :, 1] *= 2.0 ** 105  # at most 2000 values of up to 2^2.5
    got = c.run()
    assert torch.isfinite(got).all() and torch.equal(got, want * 2.0 ** 105)


@BOTH
@pytest.mark.parametrize("news", [None, [130, 9]])
def test_out_beside_the_queries_in_one_buffer(lq, news, dtype):
    c = Case([130, 40], 2, 2, 64, 16, dtype=dtype, news=news)
    n = c.hq * 64
    wide = torch.full((c.q_tokens, 2 * n + 8), 5.0, dtype=c.q.dtype, device="cuda")
    wide[:, :n] = c.q.flatten(1)
    got = c.run(wide[:, :n].unflatten(1, (c.hq, 64)), wide[:, n + 8:].unflatten(1, (c.hq, 64)))
    assert torch.equal(got, c.run())
    assert torch.equal(wide[:, :n], c.q.flatten(1)) and (wide[:, n:n + 8] == 5).all()
