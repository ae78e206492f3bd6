"""Measured cases of what a looped block needs between its linears and the attention.

``run`` makes one pass of an operator: in its plain form (elementary torch
operations in 32 bits, in 64 where said) where ``own`` is false, through the
framework's entry points where it is true.

Operators (``case["op"]``):
  norm     residual added, root-mean-square norm, output as numbers or as the
           Eq.(4) codes and steps that the quantized linear takes
  rope     rotary positions of one tensor at given positions
  enter    rotary positions of q and k, and k and v into their slab of the
           paged cache
  adapter  low-rank adapters of many requests, added to a shared projection
"""
import math

import torch

own = False

EPS = 2.0 ** -20  # exactly held in 32 bits


# --------------------------------------------------------------- the cases

def _norm(name, rows, width, x, res, out):
    c = {"op": "norm", "rows": rows, "width": width, "x": x, "res": res, "out": out}
    return dict(c, name=name) if name else c


def _rope(name, tokens, heads, head_dim, rot, layout, dtype, far):
    c = {"op": "rope", "tokens": tokens, "heads": heads, "head_dim": head_dim, "rot": rot, "layout": layout, "dtype": dtype, "far": far}
    return dict(c, name=name) if name else c


def _enter(name, rows, kv_heads, group, head_dim, rot, layout, page, held, new, dtype, q_dtype):
    c = {"op": "enter", "rows": rows, "kv_heads": kv_heads, "group": group, "head_dim": head_dim, "rot": rot, "layout": layout,
         "page": page, "held": held, "new": new, "dtype": dtype, "q_dtype": q_dtype}
    return dict(c, name=name) if name else c


def _adapter(name, rows, requests, adapters, rank, mixed, width, out, dtype):
    c = {"op": "adapter", "rows": rows, "requests": requests, "adapters": adapters, "rank": rank, "mixed": mixed, "width": width,
         "out": out, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token: the call's latency is what counts (K = 2048, the block's q|k|v input)
        _norm("norm_token", 1, 2048, "f32", "f32", "bf16"),
        # a serving batch: the next linear's 4-bit codes straight from the norm, a bf16 residual stream
        _norm("norm_batch_codes", 48, 2560, "f32", "bf16", "codes4"),
        # a prompt's tokens through the block's norm, 8-bit codes in groups of 32
        _norm("norm_prompt_codes", 8192, 2560, "f32", "f32", "codes8"),
        # calibration rows at a down projection's input, one step a token, no residual
        _norm("norm_rows_token", 4096, 6912, "bf16", "none", "token8"),
        # one new token for every row of a serving batch, straight from the fp32 q|k|v linear
        _enter("enter_token", 48, 20, 1, 128, 128, "half", 16, 8192, 1, "f32", "f32"),
        # whole prompts: fp32 q|k|v in, bf16 queries out for the attention
        _enter("enter_prompt", 2, 16, 1, 128, 128, "half", 64, 0, 8192, "f32", "bf16"),
        # ragged chunks of long contexts, shared key heads, two thirds of each head rotated in pairs
        _enter("enter_chunks", 12, 8, 3, 96, 64, "pairs", 32, 120000, 1500, "bf16", "bf16"),
        # calibration rows at given positions, heads of 96
        _rope("rope_rows", 4096, 55, 96, 96, "half", "bf16", 32768),
        # one token of one request (K = 2048, the fused q|k|v of N = 6144)
        _adapter("adapter_token", 1, 1, 4, 16, False, 2048, 6144, "f32"),
        # a serving batch, most rows with an adapter of their own, some with none
        _adapter("adapter_batch", 48, 48, 32, 16, False, 2560, 7680, "f32"),
        # ragged prompts of a few requests beside the down projection, ranks of many sizes
        _adapter("adapter_ragged", 1500, 12, 8, 32, True, 6912, 2560, "bf16"),
        # a full batch of prompt tokens beside the up projection
        _adapter("adapter_prompt", 8192, 9, 8, 64, False, 2560, 6912, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rope", "enter", "enter", "adapter", "adapter"])
    if op == "norm":
        out = rng.choice(["f32", "bf16", "codes4", "codes8", "token4", "token8"])
        unit = 8 if out in ("f32", "bf16") else 32
        width = unit * _log(rng, 1, 17920 // unit)
        rows = _log(rng, 1, min(16384, 20_000_000 // width))
        return _norm("", rows, width, rng.choice(["f32", "bf16"]), rng.choice(["none", "f32", "bf16"]), out)
    if op in ("rope", "enter"):
        dim, layout = rng.choice([64, 96, 128]), rng.choice(["half", "pairs"])
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        dtype = rng.choice(["f32", "bf16"])
        if op == "rope":
            heads = _log(rng, 1, 64)
            return _rope("", _log(rng, 1, min(16384, 20_000_000 // (heads * dim))), heads, dim, rot, layout, dtype, _log(rng, 16, 1_000_000))
        heads, group, rows, page = _log(rng, 1, 55), rng.choice([1, 1, 2, 3, 4, 7, 8]), _log(rng, 1, 96), rng.choice([8, 16, 32, 64, 128])
        if heads * group > 64:
            group = 1
        new = rng.choice([1, 1, _log(rng, 2, max(2, 20_000_000 // (rows * heads * (group + 2) * dim)))])
        held = _log(rng, 1, 131071)
        return _enter("", rows, heads, group, dim, rot, layout, page, held, min(new, 8192), dtype, rng.choice(["bf16", dtype]))
    rank, adapters = rng.choice([8, 16, 16, 32, 64, 128, rng.randint(1, 128)]), _log(rng, 1, 48)
    width, out = 32 * _log(rng, 4, 330), rng.choice([4, 32, 1]) * _log(rng, 64, 240)
    rows = _log(rng, 1, min(8192, int(3e10 / (adapters * rank * (width + out))), 20_000_000 // max(width, out)))
    return _adapter("", rows, rng.choice([rows, _log(rng, 1, min(rows, 96))]), adapters, rank, rng.random() < 0.5, width, out, rng.choice(["f32", "bf16"]))


# ------------------------------------------------- sizes that follow from a case

def _spread(b, n):
    """A fixed fraction in [0, 1) for number b: ragged cases have the same sizes for every seed."""
    return ((b + 1) * 0.6180339887498949 + 0.11 * n) % 1.0


def _ceil(a, b):
    return -(-a // b)


def _held(case):
    """Tokens that each row holds before the call."""
    n, top = case["rows"], case["held"]
    return [int(top * (0.02 + 0.98 * _spread(b, n))) for b in range(n - 1)] + [top]


def _news(case):
    """New tokens of each row."""
    n, new = case["rows"], case["new"]
    if new == 1 or case["held"] == 0:
        return [new] * n
    return [int(new * _spread(b + 3, n)) for b in range(n - 1)] + [new]


def _ids(case):
    """The adapter of each row: a request's rows lie one after the other; about one request in nine has none."""
    n, rows = case["requests"], case["rows"]
    cut = [0] + sorted(min(rows, int(rows * (b + 0.5 * _spread(b, n)) / n)) for b in range(1, n)) + [rows]
    pick = [-1 if n > 1 and b % 9 == 5 else int(case["adapters"] * _spread(3 * b, n)) for b in range(n)]
    return [pick[b] for b in range(n) for _ in range(cut[b + 1] - cut[b])]


def _ranks(case):
    n, r = case["adapters"], case["rank"]
    return [max(1, int(round(r * (0.2 + 0.8 * _spread(a, n))))) for a in range(n - 1)] + [r] if case["mixed"] else [r] * n


_SIZE = {"f32": 4, "bf16": 2, "none": 0}


def work(case):
    op = case["op"]
    if op == "norm":
        n, out = case["rows"] * case["width"], case["out"]
        o = n * _SIZE[out] if out in _SIZE else n * (1 if out[-1] == "8" else 0.5) + (case["rows"] * 4 if out[0] == "t" else n / 8)
        return {"bytes": n * (_SIZE[case["x"]] + 2 * _SIZE[case["res"]]) + o + 4 * case["width"], "flops": 6.0 * n}
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["head_dim"]
        return {"bytes": 2 * n * _SIZE[case["dtype"]] + 4 * case["tokens"] + 4 * case["rot"], "flops": 3.0 * n * case["rot"] / case["head_dim"]}
    if op == "enter":
        n = sum(_news(case)) * case["kv_heads"] * case["head_dim"]
        g = case["group"]
        return {"bytes": n * ((g + 2) * _SIZE[case["dtype"]] + g * _SIZE[case["q_dtype"]] + 4) + 12 * case["rows"],
                "flops": 3.0 * n * (g + 1) * case["rot"] / case["head_dim"]}
    ids, ranks, k, n = _ids(case), _ranks(case), case["width"], case["out"]
    some = [a for a in ids if a >= 0]
    return {"bytes": len(some) * (k * _SIZE[case["dtype"]] + 8 * n) + 4 * len(ids) + 2 * (k + n) * sum(ranks[a] for a in set(some)),
            "flops": 2.0 * (k + n) * sum(ranks[a] for a in some)}


# --------------------------------------------------------------- the inputs

_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _frequencies(rot, longest):
    """Radians a position; past 8192 positions the slow ones are stretched, those in between by a ramp over their turns."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if longest <= 8192:
        return f, 1.0
    turns = 8192 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return f * (keep + (1 - keep) / 16.0), 0.1 * math.log(16.0) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    rand = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    st = {"case": dict(case)}
    if op == "norm":
        rows, width = case["rows"], case["width"]
        loud = torch.where(torch.rand(width, generator=g, device=dev) < 0.01, 12.0, 1.0)  # a few columns stand out
        st["x"] = (rand(rows, width) * loud).to(_TYPE[case["x"]])
        if case["res"] != "none":
            st["res"] = (3.0 * rand(rows, width) * loud).to(_TYPE[case["res"]])
        st["w"] = 1.0 + 0.2 * rand(width)
        st["clip"] = 0.9375
        return st
    if op == "rope":
        st["x"] = rand(case["tokens"], case["heads"], case["head_dim"]).to(_TYPE[case["dtype"]])
        st["pos"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device=dev, dtype=torch.int32)
        f, st["magnitude"] = _frequencies(case["rot"], case["far"])
        st["freq"] = f.to(dev)
        return st
    if op == "enter":
        rows, page, h, d = case["rows"], case["page"], case["kv_heads"], case["head_dim"]
        held, news = _held(case), _news(case)
        lens = [a + b for a, b in zip(held, news)]  # the rows have room already
        first = i32([n // page for n in held])  # what lies before is not needed here: a window has left it behind
        counts = i32([_ceil(n, page) for n in lens]) - first
        pages, width = int(sum(_ceil(n, page) - m // page for n, m in zip(lens, held))) + 4, _ceil(max(lens), page) + 2
        start = torch.cumsum(counts, 0) - counts
        order = torch.randperm(pages, generator=g, device=dev)  # every row's pages lie anywhere in the pool
        k = torch.arange(width, device=dev)[None, :] - first[:, None]
        st["table"] = torch.where((k >= 0) & (k < counts[:, None]), order[(start[:, None] + k).clamp(0, pages - 1)], -1).to(torch.int32)
        st["lens"], st["cu"] = i32(lens), i32([sum(news[:b]) for b in range(rows + 1)])
        st["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        st["refs"][order[:pages - 4]] = 1
        st["pool"] = torch.empty((pages, 2, 2, h, page, d), dtype=torch.bfloat16, device=dev).normal_(generator=g)
        hq = h * case["group"]
        qkv = rand(sum(news), (hq + 2 * h) * d).to(_TYPE[case["dtype"]])  # the linear's q | k | v
        st["q"], st["k"], st["v"] = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, hq), (hq, hq + h), (hq + h, hq + 2 * h)))
        f, st["magnitude"] = _frequencies(case["rot"], max(lens))
        st["freq"] = f.to(dev)
        return st
    n, r, k, out = case["adapters"], case["rank"], case["width"], case["out"]
    room = _ceil(r, 8) * 8
    st["x"] = rand(case["rows"], k).to(_TYPE[case["dtype"]])
    st["a"] = (rand(n, room, k) / math.sqrt(k)).to(torch.bfloat16)
    st["b"] = (0.3 * rand(n, out, room)).to(torch.bfloat16)
    st["ids"], st["ranks"] = i32(_ids(case)), i32(_ranks(case))
    st["scales"] = 0.5 + torch.rand(n, generator=g, device=dev)
    st["y"] = rand(case["rows"], out)
    return st


# ------------------------------------------------------- the plain forms

def _plain_norm(st):
    case, x = st["case"], st["x"]
    h = x.float()
    got = {}
    if case["res"] != "none":
        got["sum"] = (h + st["res"].float()).to(st["res"].dtype)
        h = got["sum"].float()
    # the mean in 64 bits: its 32-bit root is then the same number in any order of adding up, and with it the codes next to a border
    r = (1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + EPS)).float()
    z = h * r * st["w"]
    if case["out"] in _TYPE:
        return dict(got, y=z.to(_TYPE[case["out"]]))
    rows, width = z.shape
    top = 7.0 if case["out"][-1] == "4" else 127.0
    part = z.reshape(rows, -1, 32) if case["out"][0] == "c" else z[:, None]
    amax = part.abs().amax(-1, keepdim=True)
    steps = st["clip"] * (amax / torch.full_like(amax, top))  # a division by a tensor: by a number would be a product with its reciprocal
    q = torch.round(part / torch.where(steps == 0, 1.0, steps)).clamp(-top, top)
    return dict(got, values=(q * steps).to(torch.bfloat16).reshape(rows, width), steps=steps[:, :, 0].expand(rows, width // 32).contiguous())


def _turned(st, x, pos):
    """x [tokens][heads][dim] at the positions, in 32 bits; angles in 64."""
    angle = pos.double()[:, None] * st["freq"]
    c, s = ((st["magnitude"] * t).float()[:, None] for t in (torch.cos(angle), torch.sin(angle)))
    rot = st["case"]["rot"]
    x = x.float()
    half = st["case"]["layout"] == "half"
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.cat((a, b), -1) if half else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(st):
    return _turned(st, st["x"], st["pos"]).to(st["x"].dtype)


def _places(st):
    """Position and page of each new token."""
    cu, lens, page = st["cu"].long(), st["lens"].long(), st["case"]["page"]
    t = torch.arange(st["k"].shape[0], device=cu.device)
    row = torch.searchsorted(cu[1:], t, right=True)
    pos = lens[row] - cu[row + 1] + t
    return pos, st["table"][row, pos // page].long()


def _plain_enter(st):
    pool, page = st["pool"], st["case"]["page"]
    pos, at = _places(st)
    pool[at, 1, 0, :, pos % page] = _turned(st, st["k"], pos).to(torch.bfloat16)
    pool[at, 1, 1, :, pos % page] = st["v"].to(torch.bfloat16)
    return {"q": _turned(st, st["q"], pos).to(_TYPE[st["case"]["q_dtype"]]), "pool": pool}


def _plain_adapter(st):
    a, b, ids, y = st["a"].float(), st["b"].float(), st["ids"], st["y"]
    n, room, k = a.shape
    z = (st["x"].float() @ a.reshape(n * room, k).T).reshape(-1, n, room)
    mine = ids[:, None] == torch.arange(n, device=ids.device)
    used = torch.arange(room, device=ids.device) < st["ranks"][:, None]
    z = torch.where(mine[:, :, None] & used, z * st["scales"][:, None], 0.0)
    return y.add_(z.reshape(-1, n * room) @ b.permute(0, 2, 1).reshape(n * room, -1))


# ------------------------------------------------------- the framework's calls

def _own_norm(block, st):
    case, x = st["case"], st["x"]
    rows, width = x.shape
    got, out = {}, case["out"]
    if case["res"] != "none":
        got["sum"] = torch.empty_like(st["res"])
    if out in _TYPE:
        got["y"] = torch.empty((rows, width), dtype=_TYPE[out], device=x.device)
        block.loopq_rms_norm(x, st["w"], EPS, y=got["y"], residual=st.get("res"), sum_out=got.get("sum"))
        return got
    codes = torch.empty((rows, width), dtype=torch.int8, device=x.device)
    got["steps"] = torch.empty((rows, width // 32), dtype=torch.float32, device=x.device)
    block.loopq_rms_norm(x, st["w"], EPS, codes=codes, steps=got["steps"], clip=st["clip"], bits_a=int(out[-1]), per_token=out[0] == "t",
                         residual=st.get("res"), sum_out=got.get("sum"))
    got["values"] = torch.empty((rows, width), dtype=torch.bfloat16, device=x.device)
    torch.mul(codes.view(rows, -1, 32), got["steps"][:, :, None], out=got["values"].view(rows, -1, 32))
    return got


def _own(st):
    from bit_ptq_looped_amd import block, kv
    op = st["case"]["op"]
    if op == "norm":
        return _own_norm(block, st)
    if op == "adapter":
        x, a, y = st["x"], st["a"], st["y"]
        if "ws" not in st:  # kept by a user's program from call to call
            st["ws"] = block.empty_adapter_workspace(x.shape[0], a.shape[1], x.device)
        block.loopq_adapter_apply(x, st["ids"], a, st["b"], st["scales"], y, st["ws"], ranks=st["ranks"])
        return y
    layout = block.LOOPQ_ROPE_HALF if st["case"]["layout"] == "half" else block.LOOPQ_ROPE_PAIRS
    rope = block.Rope(st["freq"], layout, st["magnitude"])
    if op == "rope":
        out = torch.empty_like(st["x"])
        block.loopq_rope(st["x"], st["pos"], rope, out)
        return out
    q = st["q"]
    out = torch.empty(q.shape, dtype=_TYPE[st["case"]["q_dtype"]], device=q.device)
    block.loopq_kv_write_rope(st["pool"], 1, kv.KVTable(st["table"], st["lens"], st["refs"]), st["cu"], rope, st["k"], st["v"], q, out)
    return {"q": out, "pool": st["pool"]}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "rope": _plain_rope, "enter": _plain_enter, "adapter": _plain_adapter}[state["case"]["op"]](state)


# ------------------------------------------------------- the definition in 64 bits

def _exact_turn(st, x, pos):
    out = x.double()
    rot = st["case"]["rot"]
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if st["case"]["layout"] == "half" else (2 * i, 2 * i + 1)
        t = (pos.double() * st["freq"][i])[:, None]
        u, v = out[..., a].clone(), out[..., b].clone()
        out[..., a] = st["magnitude"] * (u * torch.cos(t) - v * torch.sin(t))
        out[..., b] = st["magnitude"] * (u * torch.sin(t) + v * torch.cos(t))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_turn(st, st["x"], st["pos"])
    if op == "enter":
        pool, page, cu = st["pool"].double(), case["page"], st["cu"].tolist()
        q = torch.empty(st["q"].shape, dtype=torch.float64, device=pool.device)
        for b, (have, n) in enumerate(zip(_held(case), _news(case))):
            if not n:
                continue
            t, pos = slice(cu[b], cu[b + 1]), torch.arange(have, have + n, device=pool.device)
            at = st["table"][b].long()[pos // page]
            pool[at, 1, 0, :, pos % page] = _exact_turn(st, st["k"][t], pos)
            pool[at, 1, 1, :, pos % page] = st["v"][t].double()
            q[t] = _exact_turn(st, st["q"][t], pos)
        return {"q": q, "pool": pool}
    if op == "adapter":
        y = st["y"].double()
        for a, r in enumerate(_ranks(case)):
            rows = (st["ids"] == a).nonzero()[:, 0]
            z = st["x"][rows].double() @ st["a"][a, :r].double().T
            y[rows] += float(st["scales"][a]) * (z @ st["b"][a, :, :r].double().T)
        return y
    h = st["x"].double()
    got = {}
    if case["res"] != "none":
        got["sum"] = h + st["res"].double()
        h = got["sum"].to(st["res"].dtype).double()  # the norm is of the sum as it is kept
    z = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["width"] + EPS) * st["w"].double()
    if case["out"] in _TYPE:
        return dict(got, y=z)
    top = 2.0 ** (int(case["out"][-1]) - 1) - 1
    groups = z.unflatten(-1, (-1, 32))
    most = groups.abs().amax(-1) if case["out"][0] == "c" else z.abs().amax(-1, keepdim=True).expand(-1, case["width"] // 32)
    return dict(got, values=None, steps=st["clip"] * most / top)  # a code next to a border has no value of its own in 64 bits
