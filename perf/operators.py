"""Measured cases of the paged key-value cache and the attention over it.

A looped model keeps keys and values of its own for every (layer, loop), a
"slab"; the cache's pool is bf16 [pages][slabs][2][heads][page][head_dim], one
page table serves every slab.  ``run`` makes one pass of an operator: in its
plain form (elementary torch operations in 32 bits) where ``own`` is false,
through the framework's entry points where it is true.

Operators (``case["op"]``):
  decode   attention of one new token per row over the row's cached tokens
  prefill  attention of the rows' last tokens, causal, with a sliding window
           and sink tokens where the case has them
  fork     rows of the page table copied, reordered, dropped; shared pages
           counted, the partial last page copied for every further child
  evict    pages outside sinks and window freed, then the pool compacted
  append   pages reserved for new tokens, their keys and values written
"""
import math

import torch

own = False


# --------------------------------------------------------------- the cases

def _attn(name, op, rows, kv_heads, group, head_dim, page, max_len, window=0, sinks=0, dtype="bf16", new=1, ragged=True):
    c = {"op": op, "rows": rows, "kv_heads": kv_heads, "group": group, "head_dim": head_dim, "page": page,
         "max_len": max_len, "window": window, "sinks": sinks, "dtype": dtype, "ragged": ragged}
    if op == "prefill":
        c["new"] = new
    return dict(c, name=name) if name else c


def _pages(name, op, rows, slabs, kv_heads, head_dim, page, max_len, **more):
    c = {"op": op, "rows": rows, "slabs": slabs, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
         "max_len": max_len, **more}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token early in an answer: the call's latency is what counts (16 heads of 128, K = 2048)
        _attn("decode_single", "decode", 1, 16, 1, 128, 16, 391, ragged=False),
        # a serving batch in full swing, every row at another length (20 heads of 128, K = 2560)
        _attn("decode_batch", "decode", 48, 20, 1, 128, 16, 8192),
        # few rows over very long contexts with shared key heads, queries straight from an fp32 linear
        _attn("decode_long_shared", "decode", 3, 4, 8, 128, 64, 131071, dtype="f32", ragged=False),
        # a streaming batch: sinks and a sliding window, freed pages in between (55 heads of 96, K = 5280)
        _attn("decode_window", "decode", 32, 55, 1, 96, 32, 7000, window=2048, sinks=4),
        # the next chunk of one long prompt: few query rows over a long cache
        _attn("prefill_chunk", "prefill", 1, 16, 1, 128, 16, 16333, new=256, ragged=False),
        # whole prompts at once, causal: the largest amount of arithmetic
        _attn("prefill_prompt", "prefill", 2, 16, 1, 128, 64, 8192, new=8192, ragged=False),
        # ragged chunks of streaming rows with sinks and a window, shared key heads
        _attn("prefill_window", "prefill", 12, 8, 4, 96, 32, 6000, window=1000, sinks=4, new=1500),
        # parallel answers from a few prompts: small, latency-bound
        _pages("fork_small", "fork", 4, 4, 16, 128, 16, 300, rows_out=8, drop=0),
        # a beam step over many rows: reorder, drop the losers, copy the partial pages of 24 slabs
        _pages("fork_beams", "fork", 96, 24, 16, 128, 16, 500, rows_out=96, drop=8),
        # a long-running pool after many streams: free what the windows left behind, close the holes
        _pages("evict_pool", "evict", 64, 8, 16, 128, 16, 1600, window=256, sinks=4),
        # one new token for every row of a serving batch
        _pages("append_token", "append", 64, 4, 16, 128, 16, 1000, new=1, dtype="f32"),
        # prompts entering the cache
        _pages("append_prompt", "append", 9, 2, 20, 128, 32, 4000, new=3001, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "fork", "evict", "append"])
    dim, page = rng.choice([64, 96, 128]), rng.choice([16, 32, 64, 128])
    if op in ("decode", "prefill"):
        heads, group = _log(rng, 1, 55), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16])
        if heads * group > 64:
            group = 1
        window, sinks = (0, 0) if rng.random() < 0.5 else (_log(rng, 1, 4096), rng.choice([0, 1, 4, 5, 64]))
        if op == "decode":
            rows = _log(rng, 1, 96)
            top = max(2, min(131071, int(6e8 / (rows * heads * dim))))  # elements of keys in the plain form
            return _attn("", op, rows, heads, group, dim, page, _log(rng, 1, top), window, sinks, rng.choice(["bf16", "f32"]), ragged=rng.random() < 0.7)
        rows, new = _log(rng, 1, 16), _log(rng, 2, 4096)
        top = int(1.5e9 / (rows * heads * group * new))  # score pairs in the plain form
        if top < new:
            new = max(2, int(math.sqrt(1.5e9 / (rows * heads * group))))
            top = new
        top = max(new, min(16384, top, int(3e8 / (rows * heads * dim))))
        return _attn("", op, rows, heads, group, dim, page, _log(rng, min(new, top), top), window, sinks, rng.choice(["bf16", "bf16", "f32"]), new=min(new, top), ragged=rng.random() < 0.7)
    rows, slabs, heads = _log(rng, 1, 96), rng.choice([1, 2, 4, 8, 24]), _log(rng, 1, 20)
    length = _log(rng, 1, 1600)
    cap = 8e8 / (rows * (length / page + 1))  # elements a page may have
    while slabs > 1 and slabs * 2 * heads * page * dim > cap:
        slabs //= 2
    while heads > 1 and slabs * 2 * heads * page * dim > cap:
        heads //= 2
    if op == "fork":
        return _pages("", op, rows, slabs, heads, dim, page, length, rows_out=_log(rng, 1, 96), drop=rng.choice([0, 0, 3, 8]))
    if op == "evict":
        return _pages("", op, rows, slabs, heads, dim, page, length, window=_log(rng, 1, 1024), sinks=rng.choice([0, 1, 4, 40]))
    return _pages("", op, rows, slabs, heads, dim, page, length, new=rng.choice([1, 1, _log(rng, 2, 600)]), dtype=rng.choice(["bf16", "f32"]))


# ------------------------------------------------- sizes that follow from a case

def _spread(b, n):
    """A fixed fraction in [0, 1) for row b: ragged cases have the same lengths for every seed."""
    return ((b + 1) * 0.6180339887498949 + 0.11 * n) % 1.0


def _lens(case):
    """Tokens of each row, the new ones of prefill among them."""
    n, top = case["rows"], case["max_len"]
    if not case.get("ragged", True):
        return [top] * n
    return [max(1, int(round(top * (0.02 + 0.98 * _spread(b, n))))) for b in range(n - 1)] + [top]


def _news(case):
    """New tokens of each row."""
    n, new = case["rows"], case["new"]
    if case["op"] == "append":
        return [new if new == 1 else int(new * _spread(b + 7, n)) for b in range(n - 1)] + [new]
    if not case["ragged"]:
        return [new] * n
    return [min(l, int(new * _spread(b + 3, n))) for b, l in enumerate(_lens(case)[:-1])] + [new]


def _parents(case):
    n, out, drop = case["rows"], case["rows_out"], case["drop"]
    if out >= n and not drop:
        return [i % n for i in range(out)]
    return [-1 if drop and i % (drop + 1) == drop else int(n * _spread(5 * i, n)) for i in range(out)]


def _ceil(a, b):
    return -(-a // b)


def _copied(case):
    """Pages that a fork copies: every child after the first of a row whose last page is partial."""
    lens, par = _lens(case), [p for p in _parents(case) if p >= 0]
    return sum(1 for i, p in enumerate(par) if lens[p] % case["page"] and p in par[:i])


def _kept(case):
    """Pages that stay after a trim, over all rows."""
    page, w, s = case["page"], case["window"], case["sinks"]
    return sum(sum(1 for k in range(_ceil(l, page)) if (k + 1) * page > l - w + 1 or k * page < s) for l in _lens(case))


def _num_pages(case):
    page, used = case["page"], sum(_ceil(l, case["page"]) for l in _lens(case))
    if case["op"] == "fork":
        return used + _copied(case) + 8
    if case["op"] == "append":
        return used + sum(_ceil(l + n, page) - _ceil(l, page) for l, n in zip(_lens(case), _news(case))) + 16
    return used + used // 8 + 4


def _max_pages(case):
    extra = max(_news(case)) if case["op"] == "append" else 0
    return _ceil(case["max_len"] + extra, case["page"]) + 3


def _pairs(l, n, w, s):
    """Visible (query, key) pairs of a row's last n of l tokens, and the keys that some query sees."""
    p = torch.arange(l - n, l, dtype=torch.float64)
    seen = p + 1 if w == 0 else torch.minimum(p + 1, torch.full_like(p, w)) + torch.clamp(torch.minimum(p - w + 1, torch.full_like(p, s)), min=0)
    first = 0 if w == 0 else max(0, l - n - w + 1)
    return float(seen.sum()), l - first + min(s, first)


def work(case):
    op, d, h = case["op"], case["head_dim"], case["kv_heads"]
    lens, page = _lens(case), case["page"]
    if op in ("decode", "prefill"):
        news = [1] * case["rows"] if op == "decode" else _news(case)
        pk = [_pairs(l, n, case["window"], case["sinks"]) if n else (0.0, 0) for l, n in zip(lens, news)]
        hq, item = h * case["group"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": sum(k for _, k in pk) * h * d * 4 + 2 * sum(news) * hq * d * item + 4 * sum(_ceil(k, page) for _, k in pk),
                "flops": 4.0 * d * hq * sum(p for p, _ in pk)}
    page_bytes = case["slabs"] * 2 * h * page * d * 2
    pages = _num_pages(case)
    meta = 8 * pages + 4 * case["rows"] * _max_pages(case)
    if op == "fork":
        return {"bytes": 2 * _copied(case) * page_bytes + meta + 4 * case["rows_out"] * (_max_pages(case) + 3), "flops": 0}
    if op == "evict":
        live = _kept(case)  # pages lie anywhere in the pool: a live one is above the live count with this chance
        return {"bytes": 2 * live * (1 - live / pages) * page_bytes + 2 * meta, "flops": 0}
    n, item = sum(_news(case)), 4 if case["dtype"] == "f32" else 2
    return {"bytes": n * 2 * h * d * (item + 2) + 2 * meta, "flops": 0}


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rows, page, h, d = case["rows"], case["page"], case["kv_heads"], case["head_dim"]
    lens, pages, width = _lens(case), _num_pages(case), _max_pages(case)
    slabs = case.get("slabs", 2)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    pool = torch.empty((pages, slabs, 2, h, page, d), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    # every row's pages lie anywhere in the pool
    counts = i32([_ceil(l, page) for l in lens])
    start = torch.cumsum(counts, 0) - counts
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64)
    k = torch.arange(width, device=dev)
    has = k[None, :] < counts[:, None]
    table = torch.where(has, order[(start[:, None] + k[None, :]).clamp(max=pages - 1)], -1).to(torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    refs.scatter_add_(0, table.clamp(min=0).long().reshape(-1), has.reshape(-1).to(torch.int32))
    st = {"case": dict(case), "pool": pool, "table": table, "lens": i32(lens), "refs": refs}
    if case["op"] in ("decode", "prefill"):
        if case["window"]:  # what fell out of every query's window was freed before
            news = [1] * rows if case["op"] == "decode" else _news(case)
            low = i32([l - n - case["window"] + 1 for l, n in zip(lens, news)])
            gone = ((k[None, :] + 1) * page <= low[:, None]) & (k[None, :] * page >= case["sinks"])
            st["table"] = torch.where(gone, -1, table)
        total = rows if case["op"] == "decode" else sum(_news(case))
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        st["q"] = (1.5 * torch.randn((total, h * case["group"], d), generator=g, device=dev)).to(dt)
        if case["op"] == "prefill":
            st["cu"] = i32([sum(_news(case)[:b]) for b in range(rows + 1)])
            st["longest"] = max(_news(case))
    elif case["op"] == "fork":
        st["parent"] = i32(_parents(case))
    elif case["op"] == "append":
        news = _news(case)
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        qkv = torch.randn((sum(news), 3 * h * d), generator=g, device=dev).to(dt)  # the linear's q | k | v
        st["k"], st["v"] = (qkv[:, i * h * d:(i + 1) * h * d].unflatten(1, (h, d)) for i in (1, 2))
        st["grow"], st["cu"] = i32(news), i32([sum(news[:b]) for b in range(rows + 1)])
    return st


# ------------------------------------------------------- the plain forms

def _visible(case, table, lens, pos, keys, pages):
    """[rows][queries][keys]: whether the query at position pos sees the key."""
    page = table[:, (keys // case["page"]).clamp(max=table.shape[1] - 1)]
    there = ((page >= 0) & (page < pages))[:, None, :]
    seen = (keys[None, None, :] <= pos[:, :, None]) & there & (keys < table.shape[1] * case["page"])
    if case["window"]:
        seen = seen & ((pos[:, :, None] - keys < case["window"]) | (keys < case["sinks"]))
    return seen


def _plain_attention(st, q, pos):
    """q [rows][queries][heads][dim] at positions pos [rows][queries] over slab 1."""
    case, pool, table = st["case"], st["pool"], st["table"]
    rows, n, hq, d = q.shape
    h, page = case["kv_heads"], case["page"]
    keys = torch.arange(case["max_len"], device=q.device)
    seen = _visible(case, table, st["lens"], pos, keys, pool.shape[0])
    at = table[:, keys // page].clamp(0, pool.shape[0] - 1).long()
    k = pool[at, 1, 0, :, keys % page].float()  # [rows][keys][heads][dim]
    v = pool[at, 1, 1, :, keys % page].float()
    v = torch.where(seen.any(1)[:, :, None, None], v, 0.0)
    qs = q.float().reshape(rows, n, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(rows, h, hq // h * n, d)
    s = torch.matmul(qs, k.permute(0, 2, 3, 1)).reshape(rows, h, hq // h, n, -1) / math.sqrt(d)
    s = torch.where(seen[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1)
    o = torch.matmul(p.reshape(rows, h, hq // h * n, -1), v.permute(0, 2, 1, 3)).reshape(rows, h, hq // h, n, d)
    o = torch.where((l > 0)[..., None], o / l[..., None], 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(rows, n, hq, d)


def _plain_decode(st):
    q = st["q"]
    return _plain_attention(st, q[:, None], st["lens"][:, None] - 1)[:, 0].to(q.dtype)


def _plain_prefill(st):
    q, cu, lens = st["q"], st["cu"].long(), st["lens"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(st["longest"], device=q.device)
    at = (cu[:-1, None] + i[None, :]).clamp(max=q.shape[0] - 1)
    o = _plain_attention(st, q[at], torch.where(i[None, :] < n[:, None], (lens - n)[:, None] + i[None, :], -1))
    t = torch.arange(q.shape[0], device=q.device)
    row = torch.searchsorted(cu[1:], t, right=True)
    return o[row, t - cu[row]].to(q.dtype)


def _counts(table, pages):
    """How often each page stands in the table."""
    n = torch.zeros(pages + 1, dtype=torch.int32, device=table.device)
    at = torch.where(table < 0, pages, table).long().reshape(-1)
    return n.scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:pages]


def _plain_fork(st):
    pool, table, lens, refs, parent = st["pool"], st["table"], st["lens"], st["refs"], st["parent"].long()
    page, out = st["case"]["page"], parent.shape[0]
    i = torch.arange(out, device=pool.device)
    alive, par = parent >= 0, parent.clamp(min=0)
    new_lens = torch.where(alive, lens[par], 0)
    new_table = torch.where(alive[:, None], table[par], -1)
    last = ((new_lens - 1) // page).clamp(min=0).long()
    src = new_table.gather(1, last[:, None])[:, 0].long()
    first = torch.full((table.shape[0],), out, device=pool.device).scatter_reduce(0, par, torch.where(alive, i, out), "amin")
    keeps = (first[par] == i) & (refs[src.clamp(min=0)] == 1)
    needs = alive & (new_lens % page != 0) & (src >= 0) & ~keeps
    free = torch.sort((refs != 0).to(torch.int32), stable=True).indices
    dst = free[(torch.cumsum(needs, 0) - 1).clamp(min=0)]
    new_table = new_table.scatter(1, last[:, None], torch.where(needs, dst, src).to(torch.int32)[:, None])
    pool[dst[needs]] = pool[src[needs]]
    new_refs = refs - _counts(table, refs.shape[0]) + _counts(new_table, refs.shape[0])
    info = torch.stack([torch.zeros_like(needs.sum()), needs.sum()]).to(torch.int32)
    return {"table": new_table, "lens": new_lens, "refs": new_refs, "info": info, "pool": pool}


def _plain_evict(st):
    pool, table, lens, refs, case = st["pool"], st["table"], st["lens"], st["refs"], st["case"]
    page, pages = case["page"], refs.shape[0]
    k = torch.arange(table.shape[1], device=pool.device)
    gone = ((k[None, :] + 1) * page <= lens[:, None] - case["window"] + 1) & (k[None, :] * page >= case["sinks"])
    new_table = torch.where(gone, -1, table)
    refs = refs - _counts(table, pages) + _counts(new_table, pages)
    live = refs > 0
    n, p = live.sum(), torch.arange(pages, device=pool.device)
    hole, high = ~live & (p < n), live & (p >= n)
    rank = torch.cumsum(high, 0) - 1
    holes = torch.sort((~hole).to(torch.int32), stable=True).indices
    page_map = torch.where(live, torch.where(high, holes[rank.clamp(min=0)], p), -1)
    pool[page_map[high]] = pool[p[high]]
    new_refs = torch.zeros(pages + 1, dtype=torch.int32, device=pool.device)
    new_refs = new_refs.scatter(0, torch.where(live, page_map, pages), refs)[:pages]
    new_table = torch.where(new_table >= 0, page_map[new_table.clamp(min=0).long()], -1).to(torch.int32)
    info = torch.stack([n, high.sum()]).to(torch.int32)
    return {"table": new_table, "lens": lens, "refs": new_refs, "map": page_map.to(torch.int32), "info": info, "pool": pool}


def _plain_append(st):
    pool, table, lens, refs, grow, cu = st["pool"], st["table"], st["lens"], st["refs"], st["grow"], st["cu"].long()
    page = st["case"]["page"]
    have, want = (lens + page - 1) // page, (lens + grow + page - 1) // page
    need = want - have
    before = torch.cumsum(need, 0) - need
    free = torch.sort((refs != 0).to(torch.int32), stable=True).indices
    k = torch.arange(table.shape[1], device=pool.device)[None, :]
    is_new = (k >= have[:, None]) & (k < want[:, None])
    rank = (before[:, None] + k - have[:, None]).clamp(0, refs.shape[0] - 1).long()
    new_table = torch.where(is_new, free[rank].to(torch.int32), table)
    new_lens = lens + grow
    taken = need.sum()
    new_refs = refs.scatter(0, free, torch.where(torch.arange(refs.shape[0], device=pool.device) < taken, 1, refs[free]).to(torch.int32))
    t = torch.arange(st["k"].shape[0], device=pool.device)
    row = torch.searchsorted(cu[1:], t, right=True)
    pos = lens[row] + t - cu[row]
    at = new_table[row, pos // page].long()
    pool[at, 1, 0, :, pos % page] = st["k"].to(torch.bfloat16)
    pool[at, 1, 1, :, pos % page] = st["v"].to(torch.bfloat16)
    info = torch.stack([torch.zeros_like(taken), taken]).to(torch.int32)
    return {"table": new_table, "lens": new_lens, "refs": new_refs, "info": info, "pool": pool}


# ------------------------------------------------------- the framework's calls

def _own(st):
    from bit_ptq_looped_amd import kv
    case, pool, op = st["case"], st["pool"], st["case"]["op"]
    tab = kv.KVTable(st["table"], st["lens"], st["refs"])
    if op in ("decode", "prefill"):
        q = st["q"]
        if "ws" not in st:  # kept by a user's program from call to call
            st["ws"] = kv.empty_attn_workspace(pool, q.shape[0], q.shape[1], tab.lens.shape[0])
        out = torch.empty_like(q)
        scale, window, sinks = 1.0 / math.sqrt(q.shape[2]), case["window"], case["sinks"]
        if op == "decode":
            kv.loopq_attn_decode(pool, 1, tab, q, out, st["ws"], scale, window, sinks)
        else:
            kv.loopq_attn_prefill(pool, 1, tab, st["cu"], q, out, st["ws"], scale, window, sinks)
        return out
    if "ws" not in st:
        st["ws"] = kv.empty_pages_workspace(max(case["rows"], case.get("rows_out", 1)), pool.shape[0])
    info = torch.empty(2, dtype=torch.int32, device=pool.device)
    new = kv.empty_table(case.get("rows_out", case["rows"]), tab.table.shape[1], pool.shape[0], pool.device)
    got = {"table": new.table, "lens": new.lens, "refs": new.refs, "info": info, "pool": pool}
    if op == "fork":
        kv.loopq_kv_fork(pool, tab, st["parent"], new, info, st["ws"])
    elif op == "evict":
        got["map"] = torch.empty_like(tab.refs)
        kv.loopq_kv_trim(tab, case["page"], case["window"], case["sinks"], new)
        kv.loopq_kv_compact(pool, new, new, got["map"], info, st["ws"])
    else:
        kv.loopq_kv_reserve(tab, case["page"], st["grow"], new, info, st["ws"])
        kv.loopq_kv_write(pool, 1, new, st["cu"], st["k"], st["v"])
    return got


def run(state):
    if own:
        return _own(state)
    return {"decode": _plain_decode, "prefill": _plain_prefill, "fork": _plain_fork, "evict": _plain_evict,
            "append": _plain_append}[state["case"]["op"]](state)


# ------------------------------------------------------- the definition in 64 bits

def _exact_row(st, b, q, first):
    """q [queries][heads][dim], the first of them at position `first`, of row b."""
    case, pool = st["case"], st["pool"]
    page, h, w = case["page"], case["kv_heads"], case["window"]
    n, hq, d = q.shape
    table = st["table"][b].tolist()
    js = [j for j in range(first + n) if 0 <= table[j // page] < pool.shape[0] and (not w or first - j < w or j < case["sinks"])]
    o = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    if not js:
        return o
    j = torch.tensor(js, device=q.device)
    where = torch.tensor([table[x // page] for x in js], device=q.device)
    i = torch.arange(first, first + n, device=q.device)[:, None]
    hidden = (j > i) | ((i - j >= w) & (j >= case["sinks"]) if w else torch.zeros_like(j > i))
    for head in range(hq):
        k, v = (pool[where, 1, a, head // (hq // h), j % page].double() for a in (0, 1))
        s = (q[:, head].double() @ k.T) * d ** -0.5
        s.masked_fill_(hidden, -math.inf)
        o[:, head] = torch.softmax(s, -1) @ v
    return o


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "decode":
        if case["rows"] * case["kv_heads"] * case["group"] > 6000:
            return None
        return torch.cat([_exact_row(st, b, st["q"][b:b + 1], l - 1) for b, l in enumerate(_lens(case))])
    if op == "prefill":
        cu = st["cu"].tolist()
        return torch.cat([_exact_row(st, b, st["q"][cu[b]:cu[b + 1]], l - n) for b, (l, n) in enumerate(zip(_lens(case), _news(case)))])
    if op != "append":
        return None  # whole numbers, and pages moved as they are
    pool, page, cu = st["pool"].double(), case["page"], st["cu"].tolist()
    spare = (st["refs"] == 0).nonzero()[:, 0].tolist()
    taken = 0
    for b, (l, n) in enumerate(zip(_lens(case), _news(case))):
        own_pages = st["table"][b, :_ceil(l, page)].tolist()
        more = _ceil(l + n, page) - len(own_pages)
        own_pages += spare[taken:taken + more]
        taken += more
        pos = torch.arange(l, l + n, device=pool.device)
        at = torch.tensor(own_pages, device=pool.device)[pos // page]
        for a, x in ((0, st["k"]), (1, st["v"])):
            pool[at, 1, a, :, pos % page] = x[cu[b]:cu[b + 1]].double()
    return {"table": None, "lens": None, "refs": None, "info": None, "pool": pool}
