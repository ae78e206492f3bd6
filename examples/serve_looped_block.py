"""Serving a small looped transformer: prompts into a paged cache, answers
forked from them, one new token at a time, a sliding window with sinks.

    python examples/serve_looped_block.py

Every (layer, loop) has a slab of the cache.  A block is the quantized q|k|v
linear, the attention over the slab, and the quantized output linear, with a
residual around it; the same packed weights serve every loop.  In its full form
the block has what a served one has besides: the residual and an RMS norm that
hands the linear its 8-bit codes, rotary positions on the way into the cache, and
a low-rank adapter for each (request, loop) beside both linears.  Weights and
inputs are random: what is shown is how the calls follow each other.
"""

import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from bit_ptq_looped_amd import block, kv, loopq as lq  # noqa: E402

LAYERS, LOOPS, HEADS, DIM, PAGE = 2, 2, 4, 64, 16
HIDDEN = HEADS * DIM
ADAPTERS, RANK, EPS = 3, 16, 1e-6


class Model:
    """full: with norms, rotary positions and adapters (adapter a of loop t is number a * LOOPS + t)."""

    def __init__(self, seed=0, full=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers, self.full = [], full
        for _ in range(LAYERS):
            pack = []
            for n in (3 * HIDDEN, HIDDEN):
                w = torch.randn((n, HIDDEN), generator=g, device="cuda") / math.sqrt(HIDDEN)
                codes, scales = lq.empty_packed_weights(HIDDEN, n, 32)
                lq.loopq_pack_weights(w, 32, codes, scales)
                pack.append((n, codes, scales))
            self.layers.append(pack)
        if full:
            rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
            self.norms = [1.0 + 0.1 * rand(HIDDEN) for _ in range(LAYERS)]
            n = ADAPTERS * LOOPS
            self.adapters = [[((rand(n, RANK, HIDDEN) / math.sqrt(HIDDEN)).bfloat16(), (0.1 * rand(n, w[0], RANK)).bfloat16())
                              for w in pack] for pack in self.layers]
            self.scales = torch.full((n,), 0.5, device="cuda")
            freq = block.loopq_rope_frequencies(block.LOOPQ_ROPE_PLAIN, DIM)
            self.rope = block.Rope(torch.tensor(freq, dtype=torch.float64, device="cuda"))

    def codes_linear(self, codes, steps, which):
        """The linear on codes that the norm has formed."""
        n, w_codes, w_scales = which
        y = torch.empty((codes.shape[0], n), dtype=torch.float32, device="cuda")
        ws = lq.empty_workspace(lq.LOOPQ_OP_LINEAR, 1, codes.shape[0], HIDDEN, n, 8)
        lq.loopq_gemm_codes(codes, steps, w_codes, w_scales, 32, n, y, ws, 8)
        return y

    def full_block(self, server, layer, t, x, branch, cu, ids, one, args):
        """One block: the stream x and the branch before it in, both after it out."""
        w_qkv, w_o = self.layers[layer]
        rows, slab = x.shape[0], layer * LOOPS + t
        a_ws = block.empty_adapter_workspace(rows, RANK)
        y = torch.empty_like(x)
        codes = torch.empty((rows, HIDDEN), dtype=torch.int8, device="cuda")
        steps = torch.empty((rows, HIDDEN // 32), dtype=torch.float32, device="cuda")
        block.loopq_rms_norm(branch, self.norms[layer], EPS, y=y, residual=x, sum_out=x, codes=codes, steps=steps, bits_a=8)
        qkv = self.codes_linear(codes, steps, w_qkv)
        block.loopq_adapter_apply(y, ids, *self.adapters[layer][0], self.scales, qkv, a_ws)
        q, k, v = (qkv[:, i * HIDDEN:(i + 1) * HIDDEN].unflatten(1, (HEADS, DIM)) for i in range(3))
        block.loopq_kv_write_rope(server.pool, slab, server.table, cu, self.rope, k, v, q, q)  # q where it is
        if one:
            kv.loopq_attn_decode(server.pool, slab, server.table, q, *args)
        else:
            kv.loopq_attn_prefill(server.pool, slab, server.table, cu, q, *args)
        out = args[0].flatten(1)
        branch = self.linear(out, w_o)
        block.loopq_adapter_apply(out, ids, *self.adapters[layer][1], self.scales, branch, a_ws)
        return x, branch

    def linear(self, x, which):
        n, codes, scales = which
        y = torch.empty((x.shape[0], n), dtype=torch.float32, device="cuda")
        ws = lq.empty_workspace(lq.LOOPQ_OP_LINEAR, 1, x.shape[0], HIDDEN, n, 8)
        lq.loopq_w4a4_linear(x, None, None, 1.0, 8, codes, scales, 32, n, y, ws)
        return y


class Server:
    """Rows of a growing cache.  `table` is what the next call reads; `spare`
    receives the result of a fork, and the two change places."""

    def __init__(self, model, rows, max_tokens, num_pages, window=0, sinks=0):
        self.model, self.window, self.sinks = model, window, sinks
        self.pool = kv.empty_pool(num_pages, LAYERS * LOOPS, HEADS, PAGE, DIM)
        self.width = -(-max_tokens // PAGE)
        self.table = kv.new_table(rows, self.width, num_pages)
        self.page_map = torch.empty(num_pages, dtype=torch.int32, device="cuda")
        self.info = torch.empty(2, dtype=torch.int32, device="cuda")
        self.ws = kv.empty_pages_workspace(max(rows, 64), num_pages)
        self.ids = [b % (ADAPTERS + 1) - 1 for b in range(rows)]  # each row's adapter, -1: none

    def step(self, x, counts):
        """x [tokens][hidden]: counts[b] new tokens of each row, in order."""
        rows = len(counts)
        grow = torch.tensor(counts, dtype=torch.int32, device="cuda")
        cu = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")
        cu[1:] = torch.cumsum(grow, 0)
        kv.loopq_kv_reserve(self.table, PAGE, grow, self.table, self.info, self.ws)
        if self.info[0].item() != kv.LOOPQ_KV_DONE:
            raise RuntimeError("the cache is full")
        ws = kv.empty_attn_workspace(self.pool, x.shape[0], HEADS, rows)
        one = all(c == 1 for c in counts)
        if self.model.full:
            x, branch = x.clone(), torch.zeros_like(x)
            for t in range(LOOPS):
                ids = [a * LOOPS + t if a >= 0 else -1 for a, c in zip(self.ids, counts) for _ in range(c)]
                ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
                for layer in range(LAYERS):
                    out = torch.empty((x.shape[0], HEADS, DIM), dtype=torch.float32, device="cuda")
                    args = (out, ws, 1.0 / math.sqrt(DIM), self.window, self.sinks)
                    x, branch = self.model.full_block(self, layer, t, x, branch, cu, ids, one, args)
            return x + branch
        for t in range(LOOPS):
            for layer, (w_qkv, w_o) in enumerate(self.model.layers):
                slab = layer * LOOPS + t
                qkv = self.model.linear(x, w_qkv)
                q, k, v = (qkv[:, i * HIDDEN:(i + 1) * HIDDEN].unflatten(1, (HEADS, DIM)) for i in range(3))
                kv.loopq_kv_write(self.pool, slab, self.table, cu, k, v)
                out = torch.empty((x.shape[0], HEADS, DIM), dtype=torch.float32, device="cuda")
                args = (out, ws, 1.0 / math.sqrt(DIM), self.window, self.sinks)
                if one:
                    kv.loopq_attn_decode(self.pool, slab, self.table, q, *args)
                else:
                    kv.loopq_attn_prefill(self.pool, slab, self.table, cu, q, *args)
                x = x + self.model.linear(out.flatten(1), w_o)
        return x

    def fork(self, parent):
        """Row i goes on from row parent[i] (-1: an empty row)."""
        spare = kv.empty_table(len(parent), self.width, self.table.refs.numel())
        kv.loopq_kv_fork(self.pool, self.table, torch.tensor(parent, dtype=torch.int32, device="cuda"), spare, self.info, self.ws)
        if self.info[0].item() != kv.LOOPQ_KV_DONE:
            raise RuntimeError("the cache is full")
        self.table = spare
        self.ids = [self.ids[p] if p >= 0 else -1 for p in parent]

    def evict(self):
        """Frees what the window left behind and closes the holes; pages in use."""
        if self.window:
            kv.loopq_kv_trim(self.table, PAGE, self.window, self.sinks, self.table)
        kv.loopq_kv_compact(self.pool, self.table, self.table, self.page_map, self.info, self.ws)
        return self.info[0].item()


def run(window=0, sinks=0, seed=0, full=False):
    """Two prompts, five answers, 24 tokens each; then the first answer once more
    in one pass.  Returns (its last hidden state step by step, the same in one
    pass, pages in use before and after eviction)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    model = Model(seed, full)
    server = Server(model, 2, 256, 96, window, sinks)
    server.ids = [1, -1]
    prompts = [37, 50]
    x = torch.randn((sum(prompts), HIDDEN), generator=g, device="cuda")
    first = [x[:prompts[0]]]
    server.step(x, prompts)
    server.fork([0, 0, 1, 1, 0])
    used = []
    for n in range(24):
        x = torch.randn((5, HIDDEN), generator=g, device="cuda")
        first.append(x[:1])
        last = server.step(x, [1] * 5)
        if n % 8 == 7:
            before = int((server.table.refs > 0).sum())
            used.append((before, server.evict()))
    server.fork([0, -1])  # keep the first answer
    again = Server(model, 1, 256, 32, window, sinks)
    again.ids = [1]
    tokens = torch.cat(first)
    whole = again.step(tokens, [tokens.shape[0]])
    torch.cuda.synchronize()
    return last[0], whole[-1], used


def main():
    for window, sinks, full in ((0, 0, False), (24, 4, False), (24, 4, True)):
        step, whole, used = run(window, sinks, full=full)
        off = float((step - whole).norm() / whole.norm())
        print(f"window {window} sinks {sinks}{' with norms, rotary positions and adapters' if full else ''}: last state step by step and in one pass differ by {off:.1e}; "
              f"pages in use before and after eviction: {used}")


if __name__ == "__main__":
    main()
