"""Prefill with more tasks than work-groups: a work-group stores one task's
results after the next one's first tiles are on their way, and the two differ in
rows, positions and parts."""

import pytest

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
