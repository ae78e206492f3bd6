"""Prefill with more tasks than work-groups: a work-group stores one task's
results after the next one's first tiles are on their way, and the two differ in
rows, positions and parts."""

import math

import pytest
import torch

from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


def one_of_every_32_rows(c, heads, group):
    """A query of every run of 32 (query, head of the group) rows, and the last of each row."""
    some = []
    for t, b, p in c.queries():
        i = t - c.cu[b]
        if i % max(32 // group, 1) == 16 // group or i == c.news[b] - 1:
            some.append((t, b, p))
    return some


# parts of an item with many rows are followed by items with fewer
@pytest.mark.parametrize("dtype,lens,news,heads,group,window,sinks", [
    ("bf16", [16333], [400], 20, 1, 0, 0), ("bf16", [2000, 5003, 16333, 2000], [400, 40, 40, 130], 8, 1, 0, 0),
    ("bf16", [12001, 2000], [40, 200], 8, 3, 0, 0), ("bf16", [2000, 5003], [400, 130], 8, 2, 3000, 70),
    ("f32", [16000, 9000, 12000, 8000], [256, 40, 200, 256], 16, 1, 0, 0), ("f32", [2000], [300], 20, 2, 0, 0),
    ("f32", [2000, 5003, 16333], [300, 400, 40], 5, 1, 0, 0), ("f32", [2000, 2000, 2000, 2000], [400, 400, 400, 40], 8, 1, 1000, 4)])
def test_parts_followed_by_a_task_with_fewer_rows(lq, dtype, lens, news, heads, group, window, sinks):
    c = Case(lens, heads, group, 64, 32, window, sinks, dtype=dtype, slabs=1, slab=0, news=news)
    some = one_of_every_32_rows(c, heads, group)
    c.queries = lambda: some
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,news,heads,group,window,sinks", [
    ([3000], [3000], 24, 1, 0, 0), ([3000], [3000], 24, 1, 700, 2), ([2500, 1111, 1800], [1500, 1111, 900], 12, 2, 0, 0)])
def test_a_value_that_some_queries_see_among_many_tasks(lq, lens, news, heads, group, window, sinks, dtype):
    """NaN or infinity in a token's values reaches the queries that see it, and no other, whatever task comes next."""
    c = Case(lens, heads, group, 64, 16, window, sinks, dtype=dtype, slabs=1, slab=0, news=news, trash=False)
    want = c.run()
    assert torch.isfinite(want).all()
    odd = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
    for b, j, col, value in ((0, 700, 63, math.inf), (len(lens) - 1, 1000, 5, math.nan)):
        c.pool[c.table[b][j // 16], 0, 1, :, j % 16, col] = value
        for t, row, p in c.queries():
            odd[t, :, col] |= row == b and p >= j and (not window or p - j < window)
    got = c.run()
    assert torch.equal(~torch.isfinite(got), odd)
    rest = ~odd.any(-1).any(-1)
    assert rest.any() and torch.equal(got[rest], want[rest])
