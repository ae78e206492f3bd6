"""Plain references of the paged cache and its attention, written from the
definitions in include/loopq_kv.h: Python lists for the page bookkeeping,
numpy in 64 bits for the attention."""

import numpy as np

U = 2.0 ** -24   # unit roundoff of fp32
UB = 2.0 ** -9   # half of bf16's unit roundoff (8 significant bits: 2^-8); see tolerance()


# ------------------------------------------------------------------ pages

def clamp_len(n, width, page):
    return min(max(n, 0), width * page)


def reserve(table, lens, refs, page, grow):
    """(table, lens, refs, info) as lists; the inputs are not changed."""
    width = len(table[0])
    old = [clamp_len(n, width, page) for n in lens]
    want = [-(-(n + max(g, 0)) // page) for n, g in zip(old, grow)]
    have = [-(-n // page) for n in old]
    total = sum(w - h for w, h in zip(want, have) if w <= width)
    free = [p for p, r in enumerate(refs) if r <= 0]
    table, refs = [list(r) for r in table], list(refs)
    if any(w > width for w in want):
        return table, list(lens), refs, [2, total]
    if total > len(free):
        return table, list(lens), refs, [1, total]
    at = 0
    for b, (h, w) in enumerate(zip(have, want)):
        for k in range(h, w):
            table[b][k] = free[at]
            refs[free[at]] = 1
            at += 1
    return table, [n + max(g, 0) for n, g in zip(old, grow)], refs, [0, total]


def fork(table, lens, refs, page, parent):
    """(table, lens, refs, info, [(src, dst)])"""
    width, pages = len(table[0]), len(refs)
    free = [p for p, r in enumerate(refs) if r <= 0]
    parent = [p if 0 <= p < len(table) else -1 for p in parent]
    out = [list(table[p]) if p >= 0 else [-1] * width for p in parent]
    new_lens = [lens[p] if p >= 0 else 0 for p in parent]
    moves = []
    for i, p in enumerate(parent):
        n = clamp_len(lens[p], width, page) if p >= 0 else 0
        if n % page == 0:
            continue
        src = table[p][n // page]
        if not 0 <= src < pages or (parent.index(p) == i and refs[src] == 1):
            continue
        moves.append((i, n // page, src))
    if len(moves) > len(free):
        return [[-1] * width for _ in parent], [0] * len(parent), list(refs), [1, len(moves)], []
    copies = []
    for (i, k, src), dst in zip(moves, free):
        out[i][k] = dst
        copies.append((src, dst))
    refs = list(refs)
    for row in table:
        for p in row:
            if 0 <= p < pages:
                refs[p] -= 1
    for row in out:
        for p in row:
            if 0 <= p < pages:
                refs[p] += 1
    return out, new_lens, refs, [0, len(moves)], copies


def trim(table, lens, refs, page, window, sinks):
    width = len(table[0])
    table, refs = [list(r) for r in table], list(refs)
    for b, row in enumerate(table):
        n = clamp_len(lens[b], width, page)
        for k, p in enumerate(row):
            if (k + 1) * page <= n - window + 1 and k * page >= sinks:
                if 0 <= p < len(refs):
                    refs[p] -= 1
                row[k] = -1
    return table, list(lens), refs


def compact(table, lens, refs):
    """(table, lens, refs, page_map, info, [(src, dst)])"""
    used = [p for p, r in enumerate(refs) if r > 0]
    L = len(used)
    holes = [p for p in range(L) if refs[p] <= 0]
    high = [p for p in used if p >= L]
    to = {p: p for p in used}
    to.update(zip(high, holes))
    new_refs = [0] * len(refs)
    for p in used:
        new_refs[to[p]] = refs[p]
    return ([[to.get(p, -1) for p in row] for row in table], list(lens), new_refs,
            [to.get(p, -1) for p in range(len(refs))], [L, len(high)], list(zip(high, holes)))


# -------------------------------------------------------------- attention

def visible(p, width, page, table_row, pages, window, sinks):
    """Positions that the query at position p sees, in order."""
    top = min(p, width * page - 1)
    return [j for j in range(top + 1) if 0 <= table_row[j // page] < pages and
            (window == 0 or p - j < window or j < sinks)]


def attend(q, p, pool, slab, table_row, scale, window, sinks):
    """One query: q [heads_q][D] fp64 at position p -> (out, bound) [heads_q][D].

    bound: what fp32 arithmetic may be off (no rounding of the result).  Each
    score carries (D + 8) U of its products' magnitudes and the rounding of the
    scaled argument, exp one more ulp; a relative error e of every weight moves
    the quotient by at most 2 e A, A = sum p |v| / sum p; the sums of n terms add
    (n + 8) U A each."""
    P, _, _, H, page, D = pool.shape
    hq = q.shape[0]
    js = visible(p, len(table_row), page, table_row, P, window, sinks)
    out, bound, absum = np.zeros((hq, D)), np.zeros((hq, D)), np.zeros((hq, D))
    if not js:
        return out, bound, absum
    pages = np.array([table_row[j // page] for j in js])
    at = np.array([j % page for j in js])
    for h in range(hq):
        kh = h // (hq // H)
        k, v = pool[pages, slab, 0, kh, at], pool[pages, slab, 1, kh, at]
        s = scale * (k @ q[h])
        w = np.exp(s - s.max())
        out[h] = (w @ v) / w.sum()
        absum[h] = (w @ np.abs(v)) / w.sum()
        mag = abs(scale) * (np.abs(k) @ np.abs(q[h]))
        delta = ((D + 8) * U * mag + 4 * U * (np.abs(s) + np.abs(s).max())).max() + 4 * U
        bound[h] = absum[h] * (2 * delta + 2 * (len(js) + 8) * U) + 1e-37
    return out, bound, absum


def tolerance(out, bound, absum, dtype):
    """What the kernel may be off for a result of this type.  bf16 queries: the
    weights may be rounded to bf16 before they meet the values (A UB, on average
    over them), and the result is rounded to bf16; the two together are no less
    than the rounding of the result alone, 2 UB |out|, since A >= |out|."""
    if dtype == "f32":
        return bound + U * np.abs(out)
    e = bound + UB * absum
    return e + UB * (np.abs(out) + e)
