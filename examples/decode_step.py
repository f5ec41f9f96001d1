"""One decode step after another with the package's operators, as a serving
program runs them.

A layer's paged cache is split over RANKS parts (each rank holds every second
page of a request, as a cache sharded over its length does; here all on one
device).  A step projects the new token, appends its key and value with the
position rotation, attends over each part, and joins the parts' results:

    cache_append -> attend_paged per rank -> fold_softmax

The step is captured into a graph once and replayed; lengths, slots and page
tables live on the device, so a replay follows them.

    python examples/decode_step.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_fixed_order_amd as detfold  # noqa: E402

RANKS, PAGE = 2, 16


class Layer:
    """One attention layer's decode state for `batch` requests of up to `longest` tokens."""

    def __init__(self, batch, longest, q_heads=8, heads=2, dim=64, cache_type=torch.bfloat16, seed=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.batch, self.q_heads, self.heads, self.dim = batch, q_heads, heads, dim
        self.hidden = q_heads * dim
        per = -(-longest // (RANKS * PAGE))               # pages of a request on each rank
        self.longest = per * PAGE                         # tokens of a request on a rank
        self.w = self._normal((self.hidden, (q_heads + 2 * heads) * dim)) / math.sqrt(self.hidden)
        rate = 10000.0 ** (-torch.arange(dim // 2, device="cuda", dtype=torch.float64) / (dim // 2))
        angle = torch.arange(per * RANKS * PAGE, device="cuda", dtype=torch.float64)[:, None] * rate
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.caches, self.tables, self.work = [], [], []
        for _ in range(RANKS):
            pages = batch * per
            k, v = (torch.zeros((pages, PAGE, heads, dim), device="cuda").to(cache_type) for _ in range(2))
            cache = detfold.PagedCache(k, v)
            self.caches.append(cache)
            self.tables.append(torch.randperm(pages, generator=self.gen, device="cuda", dtype=torch.int32).view(batch, per))
            self.work.append(detfold.attend_workspace(cache, batch, q_heads, self.longest))
        self.length = torch.zeros(batch, dtype=torch.int64, device="cuda")  # tokens of each request so far
        self.x = torch.zeros((batch, self.hidden), device="cuda", dtype=torch.bfloat16)
        self.q = torch.empty((batch, q_heads, dim), device="cuda", dtype=torch.bfloat16)
        self.outs = torch.empty((RANKS, batch, q_heads, dim), device="cuda")
        self.lses = torch.empty((RANKS, batch, q_heads), device="cuda")
        self.out = torch.empty((batch, q_heads, dim), device="cuda")

    def _normal(self, shape):
        return torch.randn(shape, generator=self.gen, device="cuda").bfloat16()

    def step(self):
        """The next token of every request: self.x -> self.out."""
        qkv = self.x @ self.w
        q, k, v = (t.unflatten(1, (-1, self.dim)) for t in
                   qkv.split([self.hidden, self.heads * self.dim, self.heads * self.dim], dim=1))
        at, page = self.length % PAGE, self.length // PAGE      # the request's page, counted over all ranks
        mine, rank = page // RANKS, page % RANKS
        for r, cache in enumerate(self.caches):
            slots = self.tables[r].gather(1, mine[:, None])[:, 0] * PAGE + at
            slots = torch.where(rank == r, slots, -1)           # another rank's token: not stored here
            detfold.cache_append(cache, k, v, slots, q=q, q_out=self.q, positions=self.length, cos=self.cos, sin=self.sin)
        total = self.length + 1
        for r, cache in enumerate(self.caches):
            whole, rest = total // (RANKS * PAGE) * PAGE, total % (RANKS * PAGE)
            lens = (whole + (rest - r * PAGE).clamp(0, PAGE)).to(torch.int32)
            detfold.attend_paged(self.outs[r], self.q, cache, self.tables[r], lens, max_len=self.longest,
                                 lse=self.lses[r], workspace=self.work[r])
        detfold.fold_softmax(self.out, self.outs, self.lses)
        self.length.add_(1)

    def plain(self, xs):
        """The last of the steps over inputs xs [n, batch, hidden], in float64 on the host, without a cache."""
        n = len(xs)
        qkv = torch.stack([x @ self.w for x in xs]).double().cpu()
        q, k, v = (t.unflatten(2, (-1, self.dim)) for t in
                   qkv.split([self.hidden, self.heads * self.dim, self.heads * self.dim], dim=2))
        cos, sin = self.cos[:n].double().cpu()[:, None, None], self.sin[:n].double().cpu()[:, None, None]

        def turned(t):
            a, b = t.chunk(2, -1)
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).bfloat16().double()

        q, k = turned(q)[-1], turned(k)
        group = self.q_heads // self.heads
        k, v = (t.repeat_interleave(group, 2) for t in (k, v))
        s = torch.einsum("bhd,tbhd->bht", q, k) / math.sqrt(self.dim)
        return torch.einsum("bht,tbhd->bhd", torch.softmax(s, -1), v)


def main(steps=200, batch=3):
    layer = Layer(batch, steps + 1)
    xs = [layer._normal((batch, layer.hidden)) for _ in range(steps)]
    layer.x.copy_(xs[0])
    layer.step()                                             # eager: nothing here synchronizes
    graph = torch.cuda.CUDAGraph()
    layer.length.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.step()
    for x in xs:
        layer.x.copy_(x)
        graph.replay()
    off = float((layer.out.double().cpu() - layer.plain(xs)).abs().max())
    print("%d steps of %d requests over %d ranks: the last output differs from the plain form by %.2g" % (steps, batch, RANKS, off))
    return off


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
