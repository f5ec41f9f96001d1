"""The example's decode loop, step by step, from what its caches hold: every token
stored once, in its rank's slot, and every step's output the attention over exactly
the tokens so far: one token more or less, in a row of 200, moves it by about 2^-8,
well past the tolerance."""
import importlib.util
import math
import os

import pytest

import decode_oracle as oracle

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(detfold_lib):
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _held(example, layer, b, n):
    """Keys and values of request b's n tokens, from the ranks' caches through their tables."""
    k, v = [], []
    for t in range(n):
        page, at = divmod(t, example.PAGE)
        r, mine = page % example.RANKS, page // example.RANKS
        c = layer.caches[r]
        slot = int(layer.tables[r][b, mine])
        k.append(c.k[slot, at].cpu())
        v.append(c.v[slot, at].cpu())
    return k, v


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("steps", [1, 2, 16, 17, 33, 70, 200])
def test_every_step(example, graph, steps):
    import torch
    batch = 3
    layer = example.Layer(batch, steps + 1)
    xs = [layer._normal((batch, layer.hidden)) for _ in range(steps)]
    replay = layer.step
    if graph:
        layer.x.copy_(xs[0])
        layer.step()
        captured = torch.cuda.CUDAGraph()
        layer.length.zero_()
        torch.cuda.synchronize()
        with torch.cuda.graph(captured):
            layer.step()
        replay = captured.replay
    for c in layer.caches:  # the capture's own step aside
        c.k.zero_(), c.v.zero_()
    for x in xs:
        layer.x.copy_(x)
        replay()
    assert layer.length.tolist() == [steps] * batch

    # what was stored: the projection, the keys turned by their positions and rounded once
    qkv = torch.stack([x @ layer.w for x in xs]).double().cpu()
    q, k, v = (t.unflatten(2, (-1, layer.dim)) for t in
               qkv.split([layer.hidden, layer.heads * layer.dim, layer.heads * layer.dim], dim=2))
    cos, sin = layer.cos[:steps].double().cpu(), layer.sin[:steps].double().cpu()
    bf = torch.bfloat16
    for b in range(batch):
        hk, hv = _held(example, layer, b, steps)
        hk, hv = torch.stack(hk), torch.stack(hv)
        want, size = oracle.rotate(k[:, b], cos, sin, False)
        oracle.close(hk, want, oracle.stored(want, size, bf)[1], "keys of request %d" % b)
        assert torch.equal(hv.double(), v[:, b])
        want, size = oracle.rotate(q[-1:, b], cos[-1:], sin[-1:], False)
        oracle.close(layer.q[b:b + 1], want, oracle.stored(want, size, bf)[1], "query of request %d" % b)
        # the output over these very keys and values
        group = layer.q_heads // layer.heads
        for h in range(layer.heads):
            i = slice(h * group, (h + 1) * group)
            out, _, tol, _ = oracle.attend(layer.q[b, i].double().cpu(), hk[:, h].double(), hv[:, h].double(),
                                           1 / math.sqrt(layer.dim), torch.float32, None)
            # the join of two ranks: their outputs and weights, each off by no more
            # than the whole's tolerance, and the fold's exp, sums and product
            values = hv[:, h].double().abs().amax()
            oracle.close(layer.out[b, i], out, 3 * tol + 2.0 ** -20 * values, "output of request %d" % b)
    # no other slot was written
    for r, c in enumerate(layer.caches):
        mine = sum(len(range(p * example.PAGE, min(steps, (p + 1) * example.PAGE)))
                   for p in range(r, -(-steps // example.PAGE), example.RANKS))
        assert int((c.k != 0).any(-1).any(-1).sum()) == batch * mine
