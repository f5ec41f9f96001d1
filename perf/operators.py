"""What is measured of the decode-step operators: the paged cache's append, the
attention of one new token over it, and the fold of attention partials.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is true, through the
package's entry points.  ``exact`` computes the same from the definition in 64
bits.  Layouts: a cache is ``[pages, page_size, heads, dim]`` (``order`` says
how it lies in memory), a row's tokens are numbered from its first page on, and
page 0 belongs to no row.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0
BIGGEST = 1.6e9  # bytes of cache of a drawn attention; the largest listed one has 2.1e9


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # one new token of one request: the smallest call, all latency
        _append("append 1 token bf16", 1, 32, 8, 128, "bf16", "bf16", 16),
        # a decode batch of 64 requests into an 8-bit cache
        _append("append 64 tokens e4m3", 64, 32, 8, 128, "bf16", "e4m3", 64),
        # an odd prompt in float32: a third of each head rotated, in pairs, pages of 7
        _append("append 1021 tokens f32 odd", 1021, 15, 3, 84, "f32", "f32", 7, rot=28, pairs=True),
        # a prompt of 8192 tokens: bandwidth
        _append("append 8192 tokens bf16", 8192, 32, 8, 128, "bf16", "bf16", 16, order="htd"),
        # one request with a short cache: latency
        _attend("attend 1 x 1000 bf16", 1, 1000, 32, 8, 128, "bf16", "bf16", 16),
        # one request with a long cache: the split over its length must fill the card
        _attend("attend 1 x 131072 bf16", 1, 131072, 32, 8, 128, "bf16", "bf16", 16),
        # a decode batch of ragged lengths, idle rows among them
        _attend("attend 64 ragged 8192 bf16", 64, 8192, 32, 8, 128, "bf16", "bf16", 64, ragged=True, idle=True),
        # a large batch over an 8-bit cache
        _attend("attend 256 x 4096 e4m3", 256, 4096, 32, 8, 128, "bf16", "e4m3", 16, order="htd"),
        # float32 with odd sizes: 5 queries a head, heads of 84, pages of 7, the last 1500 tokens
        _attend("attend 7 ragged 6001 f32 odd", 7, 6001, 15, 3, 84, "f32", "f32", 7, ragged=True, window=1500),
        # the decode join of two ranks' attention, hidden 4096
        _fold("fold 2 x 32 x 128 f32", 2, 32, 128, "f32"),
        # odd rows of 16-bit partials, some of them empty
        _fold("fold 5 x 4099 x 84 bf16", 5, 4099, 84, "bf16", empty=True),
        # a prompt's attention over eight ranks: 64 MiB a rank
        _fold("fold 8 x 131072 x 128 f32", 8, 131072, 128, "f32", empty=True),
    ]


def _append(name, tokens, q_heads, heads, dim, dtype, cache, page, rot=None, pairs=False, order="thd", idle=False):
    return dict(name=name, op="append", tokens=tokens, q_heads=q_heads, heads=heads, dim=dim, dtype=dtype,
                cache=cache, page=page, rot=dim if rot is None else rot, pairs=pairs, order=order, idle=idle)


def _attend(name, batch, longest, q_heads, heads, dim, dtype, cache, page, out=None, v_dim=None, order="thd",
            ragged=False, idle=False, window=0):
    return dict(name=name, op="attend", batch=batch, longest=longest, q_heads=q_heads, heads=heads, dim=dim,
                v_dim=dim if v_dim is None else v_dim, dtype=dtype, cache=cache, page=page,
                out=dtype if out is None else out, order=order, ragged=ragged, idle=idle, window=window)


def _fold(name, ranks, rows, dim, dtype, empty=False):
    return dict(name=name, op="fold", ranks=ranks, rows=rows, dim=dim, dtype=dtype, empty=empty)


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "fold"])
    if op == "fold":
        ranks, dim = _log(rng, 1, 16), rng.choice([64, 80, 96, 128, 128, 192, 256, rng.randint(1, 256)])
        dtype = rng.choice(["f32", "f32", "bf16", "f16"])
        rows = _log(rng, 1, int(5e8 / (ranks * dim * SIZE[dtype])))
        c = _fold("", ranks, rows, dim, dtype, empty=rng.random() < 0.5)
    else:
        heads = rng.choice([1, 2, 3, 4, 8, 8, 12, 16])
        q_heads = heads * rng.choice([1, 1, 2, 4, 4, 5, 7, 8, 16, 24])
        dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
        dtype, cache = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f16", "f16"),
                                   ("f16", "e4m3"), ("f32", "f32"), ("f32", "bf16"),
                                   ("f32", "e4m3")])
        page, order = rng.choice([1, 7, 16, 16, 32, 48, 64, 128, 256]), rng.choice(["thd", "htd"])
        if op == "append":
            tokens = _log(rng, 1, int(1.5e8 / ((q_heads + 2 * heads) * dim * SIZE[dtype])))
            c = _append("", tokens, q_heads, heads, dim, dtype, cache, page, rot=rng.choice([dim, dim, dim // 4 * 2]),
                        pairs=rng.random() < 0.4, order=order, idle=rng.random() < 0.4)
        else:
            v_dim = rng.choice([dim, dim, dim, 64, 128])
            a_token = heads * (dim + v_dim) * SIZE[cache]
            batch = _log(rng, 1, 256)
            longest = _log(rng, 1, max(1, min(131072, int(BIGGEST / (batch * a_token)))))
            ragged = rng.random() < 0.6
            c = _attend("", batch, longest, q_heads, heads, dim, dtype, cache, page,
                        out="f32" if rng.random() < 0.25 else dtype, v_dim=v_dim, order=order, ragged=ragged,
                        idle=ragged and rng.random() < 0.5,
                        window=_log(rng, 1, longest) if rng.random() < 0.2 else 0)
    del c["name"]
    return c


def _lengths(c):
    """The rows' lengths: spread evenly over (0, longest] where they are ragged,
    every ninth row without a request where some are idle."""
    b, top = c["batch"], c["longest"]
    got = [max(1, int(top * ((i * 0.6180339887498949) % 1.0))) if c["ragged"] and i else top for i in range(b)]
    return [0 if c["idle"] and i % 9 == 4 else n for i, n in enumerate(got)]


def work(case):
    c = case
    if c["op"] == "append":
        live = sum(not _is_idle(c, i) for i in range(c["tokens"]))
        q = c["tokens"] * c["q_heads"] * c["dim"]
        kv = live * c["heads"] * c["dim"] * 2
        size = 2 * q * SIZE[c["dtype"]] + kv * (SIZE[c["dtype"]] + SIZE[c["cache"]])
        return {"bytes": size + c["tokens"] * (16 + 4 * c["rot"]),
                "flops": 3 * c["rot"] * (c["tokens"] * c["q_heads"] + live * c["heads"])}
    if c["op"] == "attend":
        seen = sum(min(n, c["window"] or n) for n in _lengths(c))
        pages = sum(-(-min(n, c["window"] or n) // c["page"]) for n in _lengths(c))
        rows = c["batch"] * c["q_heads"]
        return {"bytes": seen * c["heads"] * (c["dim"] + c["v_dim"]) * SIZE[c["cache"]] + 4 * pages + 4 * c["batch"]
                + rows * (c["dim"] * SIZE[c["dtype"]] + c["v_dim"] * SIZE[c["out"]] + 4),
                "flops": 2 * seen * c["q_heads"] * (c["dim"] + c["v_dim"])}
    each = c["rows"] * (c["dim"] * SIZE[c["dtype"]] + 4)
    return {"bytes": (c["ranks"] + 1) * each, "flops": 2 * c["ranks"] * c["rows"] * c["dim"]}


# --------------------------------------------------------------------------
# inputs

def _normal(gen, shape, dtype, spread=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16 if dtype == "e4m3" else TYPES[dtype])
    if spread != 1.0:
        x.mul_(spread)
    return x.to(TYPES[dtype])


def _pool(gen, pages, page, heads, dim, c):
    """A cache that other requests have filled before."""
    if c["order"] == "htd":
        return _normal(gen, (pages, heads, page, dim), c["cache"]).transpose(1, 2)
    return _normal(gen, (pages, page, heads, dim), c["cache"])


def _bits(x):
    """An 8-bit cache as whole bytes: torch indexes those."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _scales(gen, c):
    if c["cache"] != "e4m3":
        return None, None
    s = torch.rand((2, c["heads"]), generator=gen, device="cuda") * 0.05 + 0.02
    return s[0].contiguous(), s[1].contiguous()


def _is_idle(c, i):
    return c["idle"] and i % 9 == 4


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"append": _prepare_append, "attend": _prepare_attend, "fold": _prepare_fold}[case["op"]](case, gen)


def _prepare_append(c, gen):
    t, hq, h, d = c["tokens"], c["q_heads"], c["heads"], c["dim"]
    # a projection gives queries, keys and values of a token side by side
    qkv = _normal(gen, (t, (hq + 2 * h) * d), c["dtype"])
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, h * d, h * d], dim=1))
    pages = -(-t // c["page"]) + 9
    order = torch.randperm(pages - 1, generator=gen, device="cuda") + 1
    at = torch.arange(t, device="cuda")
    slots = order[at // c["page"]] * c["page"] + at % c["page"]
    far = 32768
    positions = (at + torch.randint(0, far, (1,), generator=gen, device="cuda")) if t > 512 else \
        torch.randint(0, far, (t,), generator=gen, device="cuda")
    if c["idle"]:  # tokens that pad the batch
        idle = at % 9 == 4
        slots, positions = slots.masked_fill(idle, -1), positions.masked_fill(idle, 0)
    half = c["rot"] // 2
    rate = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(half, 1))
    angle = torch.arange(far + t, device="cuda", dtype=torch.float64)[:, None] * rate
    k_scale, v_scale = _scales(gen, c)
    s = dict(case=c, q=q, k=k, v=v, q_out=torch.empty((t, hq, d), device="cuda", dtype=TYPES[c["dtype"]]),
             k_cache=_pool(gen, pages, c["page"], h, d, c), v_cache=_pool(gen, pages, c["page"], h, d, c),
             k_scale=k_scale, v_scale=v_scale, slots=slots, positions=positions,
             cos=angle.cos().float(), sin=angle.sin().float())
    if own:
        import deterministic_fixed_order_amd as detfold
        s["cache"] = detfold.PagedCache(s["k_cache"], s["v_cache"], k_scale=k_scale, v_scale=v_scale)
    return s


def _prepare_attend(c, gen):
    b, hq, h, page = c["batch"], c["q_heads"], c["heads"], c["page"]
    lens = torch.tensor(_lengths(c), device="cuda")[torch.randperm(b, generator=gen, device="cuda")]
    held = (lens + page - 1) // page
    wide, pages = -(-c["longest"] // page), int(held.sum()) + 9
    order = (torch.randperm(pages - 1, generator=gen, device="cuda") + 1)
    col = torch.arange(wide, device="cuda")
    first = held.cumsum(0) - held
    table = torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=pages - 2)], 0)
    k_cache = _pool(gen, pages, page, h, c["dim"], c)
    v_cache = _pool(gen, pages, page, h, c["v_dim"], c)
    # the slots after a row's end hold whatever they held: here, no numbers
    last = (lens - 1).clamp(min=0) // page
    after = (torch.arange(page, device="cuda") >= (lens - last * page)[:, None]) & (lens > 0)[:, None]
    at = table.gather(1, last[:, None]).expand(-1, page)
    nan = 0x7F if c["cache"] == "e4m3" else float("nan")
    row = torch.arange(page, device="cuda").expand(b, -1)
    _bits(k_cache)[at[after], row[after]] = nan
    _bits(v_cache)[at[after], row[after]] = nan
    k_scale, v_scale = _scales(gen, c)
    if k_scale is not None:
        k_scale, v_scale = k_scale * 20, v_scale * 20  # the cache's values are about 1 already
    s = dict(case=c, q=_normal(gen, (b, hq, c["dim"]), c["dtype"], 2.0), k_cache=k_cache, v_cache=v_cache,
             k_scale=k_scale, v_scale=v_scale, table=table.to(torch.int32), lens=lens.to(torch.int32),
             scale=1.0 / math.sqrt(c["dim"]),
             out=torch.empty((b, hq, c["v_dim"]), device="cuda", dtype=TYPES[c["out"]]),
             lse=torch.empty((b, hq), device="cuda"))
    if own:
        import deterministic_fixed_order_amd as detfold
        s["cache"] = detfold.PagedCache(k_cache, v_cache, k_scale=k_scale, v_scale=v_scale)
        s["workspace"] = detfold.attend_workspace(s["cache"], b, hq, c["longest"])
    return s


def _prepare_fold(c, gen):
    w, r, d = c["ranks"], c["rows"], c["dim"]
    outs, lses = _normal(gen, (w, r, d), c["dtype"]), torch.randn((w, r), generator=gen, device="cuda") * 3 + 6
    if c["empty"]:  # ranks without a token of the row: nothing was written there
        lses[torch.rand((w, r), generator=gen, device="cuda") < 0.2] = -math.inf
        outs.masked_fill_((lses == -math.inf)[:, :, None], math.nan)
    return dict(case=c, outs=outs, lses=lses, out=torch.empty((r, d), device="cuda", dtype=TYPES[c["dtype"]]),
                lse=torch.empty(r, device="cuda"))


# --------------------------------------------------------------------------
# one pass

def run(state):
    return {"append": _run_append, "attend": _run_attend, "fold": _run_fold}[state["case"]["op"]](state)


def _run_append(s):
    if own:
        import deterministic_fixed_order_amd as detfold
        detfold.cache_append(s["cache"], s["k"], s["v"], s["slots"], q=s["q"], q_out=s["q_out"],
                             positions=s["positions"], cos=s["cos"], sin=s["sin"], pairs=s["case"]["pairs"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    cos, sin = (s[n][s["positions"]][:, None] for n in ("cos", "sin"))
    s["q_out"].copy_(_rotated(s["q"].float(), cos, sin, s["case"]))
    _stored(s["k_cache"], _rotated(s["k"].float(), cos, sin, s["case"]), s["k_scale"], s["slots"])
    _stored(s["v_cache"], s["v"].float(), s["v_scale"], s["slots"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _rotated(x, cos, sin, c):
    turned, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["pairs"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = turned.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _stored(cache, x, scale, slots):
    page, at = (slots.clamp(min=0)).div(cache.shape[1], rounding_mode="floor"), slots.clamp(min=0) % cache.shape[1]
    if scale is not None:
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    bits = _bits(cache)
    new = _bits(x.to(cache.dtype))
    # a token without a slot leaves what is there
    bits[page, at] = torch.where((slots < 0)[:, None, None], bits[page, at], new)


def _run_attend(s):
    c = s["case"]
    if own:
        import deterministic_fixed_order_amd as detfold
        detfold.attend_paged(s["out"], s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"],
                             window=c["window"], max_len=c["longest"], lse=s["lse"], workspace=s["workspace"])
        return s["out"], s["lse"]
    b, hq, h = c["batch"], c["q_heads"], c["heads"]
    k, v = (_bits(x)[s["table"].long()].flatten(1, 2).view(x.dtype).float().transpose(1, 2)
            for x in (s["k_cache"], s["v_cache"]))                      # [batch, heads, tokens, dim]
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    t, n = torch.arange(k.shape[2], device=k.device), s["lens"][:, None]
    seen = (t < n) & (t >= n - c["window"] if c["window"] else t >= 0)  # [batch, tokens]
    score = torch.matmul(s["q"].float().reshape(b, h, hq // h, -1), k.transpose(2, 3)) * s["scale"]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.masked_fill(~seen[:, None, :, None], 0.0)) / total.masked_fill(total == 0, 1.0)
    return o.reshape(b, hq, -1).to(TYPES[c["out"]]), (top + torch.log(total)).reshape(b, hq)


def _run_fold(s):
    if own:
        import deterministic_fixed_order_amd as detfold
        detfold.fold_softmax(s["out"], s["outs"], s["lses"], lse=s["lse"])
        return s["out"], s["lse"]
    top = s["lses"].amax(0)
    top = top.masked_fill(top == -math.inf, 0.0)
    a = torch.exp(s["lses"] - top)
    o = s["outs"].float().masked_fill((s["lses"] == -math.inf)[:, :, None], 0.0)
    total = a.sum(0)
    o = (a[:, :, None] * o).sum(0) / total.masked_fill(total == 0, 1.0)[:, None]
    return o.to(s["outs"].dtype), top + torch.log(total)


# --------------------------------------------------------------------------
# the definition, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attend": _exact_attend, "fold": _exact_fold}[case["op"]](s, case)


def _exact_append(s, c):
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    half = c["rot"] // 2
    if c["pairs"]:
        first, second = 2 * torch.arange(half), 2 * torch.arange(half) + 1
    else:
        first, second = torch.arange(half), half + torch.arange(half)
    turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"]]

    def rotate(x):
        y = x.double()
        z = torch.complex(y[:, :, first], y[:, :, second]) * turn[:, None, :]
        y[:, :, first], y[:, :, second] = z.real, z.imag
        return y

    def store(cache, x, scale):
        y = cache.double().contiguous()
        if scale is not None:
            x = torch.clamp(x / scale.double()[None, :, None], -E4M3_MAX, E4M3_MAX)
        y.view(-1, c["heads"], c["dim"])[s["slots"][live]] = x[live]
        return y

    k, v = rotate(s["k"]), s["v"].double()
    return rotate(s["q"]), store(s["k_cache"], k, s["k_scale"]), store(s["v_cache"], v, s["v_scale"])


def _exact_attend(s, c):
    group = c["q_heads"] // c["heads"]
    out = torch.zeros((c["batch"], c["q_heads"], c["v_dim"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    k_bits, v_bits = _bits(s["k_cache"]), _bits(s["v_cache"])
    for i, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        pages = s["table"][i, :-(-n // c["page"])].long()
        low = max(0, n - c["window"]) if c["window"] else 0
        for h in range(c["heads"]):
            k = k_bits[pages, :, h].flatten(0, 1)[low:n].contiguous().view(s["k_cache"].dtype).double()
            v = v_bits[pages, :, h].flatten(0, 1)[low:n].contiguous().view(s["v_cache"].dtype).double()
            heads = slice(h * group, (h + 1) * group)
            x = (k @ s["q"][i, heads].double().t()) * s["scale"]          # [tokens, group]
            if s["k_scale"] is not None:
                x, v = x * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            lse[i, heads] = torch.logsumexp(x, 0)
            out[i, heads] = torch.softmax(x, 0).t() @ v
    return out, lse


def _exact_fold(s, c):
    lses = s["lses"].double()
    out = torch.zeros((c["rows"], c["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.logsumexp(lses, 0)
    for r in range(c["ranks"]):
        there = lses[r] > -math.inf
        out[there] += torch.exp(lses[r] - lse)[there, None] * s["outs"][r][there].double()
    return out, lse
