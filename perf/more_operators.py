"""What is measured of the drafted step's operators: the attention of a tree of
drafted tokens over the paged cache, capped and biased scores of one new token,
the copy of pages, and the compaction of a row's kept tokens.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is true, through the
package's entry points.  ``exact`` computes the same from the definition in 64
bits.  Layouts: a cache is ``[pages, page_size, heads, dim]`` (``order`` says
how it lies in memory), a row's tokens are numbered from its first page on, its
drafted tokens are its last ones, and page 0 belongs to no row.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
BIGGEST = 1.0e9  # bytes of cache of a drawn case; the largest listed ones have 1.07e9
SCORES = 1.2e8   # scores of a drawn attention; the largest listed one has 2.7e8


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # one request with a short cache and a small tree: the smallest drafted step, all latency
        _attend("tree 1 x 8 over 1000 bf16", 1, 1000, 8, 32, 8, 128, "bf16", "bf16", 16),
        # a decode batch of ragged lengths, each with a tree of its own size, idle rows among them
        _attend("tree 64 x 8 ragged 8192 bf16", 64, 8192, 8, 32, 8, 128, "bf16", "bf16", 64, ragged=True, idle=True,
                fewer=True),
        # one request with a long cache: the split over its length must fill the card
        _attend("tree 1 x 16 over 131072 bf16", 1, 131072, 16, 32, 8, 128, "bf16", "bf16", 16),
        # the largest trees: products bound it
        _attend("tree 32 x 64 over 4096 bf16 capped", 32, 4096, 64, 32, 8, 128, "bf16", "bf16", 16, cap=50.0),
        # float32 with odd sizes: 5 queries a head, heads of 84, pages of 7, a window and a bias by distance
        _attend("tree 7 x 13 ragged 3001 f32 odd", 7, 3001, 13, 15, 3, 84, "f32", "f32", 7, ragged=True, fewer=True,
                window=1500, slopes=True),
        # one new token of one request, scores capped: latency
        _attend("capped 1 x 1000 bf16", 1, 1000, 0, 32, 8, 128, "bf16", "bf16", 16, cap=50.0),
        # a local layer of a decode batch: capped, each row its last 4096 tokens
        _attend("capped 64 ragged 8192 bf16 window", 64, 8192, 0, 32, 8, 128, "bf16", "bf16", 64, ragged=True,
                idle=True, window=4096, cap=30.0),
        # a bias by distance over an 8-bit cache
        _attend("biased 32 x 8192 e4m3", 32, 8192, 0, 32, 8, 128, "bf16", "e4m3", 16, order="htd", slopes=True),
        # a beam's fork: the last page of each of three requests, partly filled
        _copy("copy 3 pages bf16", 3, 8, 128, "bf16", 16, part=True),
        # a pool that is moved to other pages: bandwidth
        _copy("copy 2048 pages of 64 bf16", 2048, 8, 128, "bf16", 64, idle=True),
        # the accepted paths of 64 trees of 16 drafted tokens, in place: latency
        _compact("compact 64 x 16 drafted bf16", 64, 4096, 16, 5, 8, 128, "bf16", 16, drafted=True),
        # 2048 kept tokens of prompts of 8192, into pages of their own: bandwidth
        _compact("compact 32 x 2048 of 8192 bf16", 32, 8192, 8192, 2048, 8, 128, "bf16", 16),
    ]


def _attend(name, batch, longest, drafts, q_heads, heads, dim, dtype, cache, page, out=None, v_dim=None, order="thd",
            ragged=False, idle=False, fewer=False, chain=False, window=0, cap=0.0, slopes=False):
    """drafts = 0: one new token per row."""
    return dict(name=name, op="tree" if drafts else "paged", batch=batch, longest=longest, drafts=drafts, q_heads=q_heads,
                heads=heads, dim=dim, v_dim=dim if v_dim is None else v_dim, dtype=dtype, cache=cache, page=page,
                out=dtype if out is None else out, order=order, ragged=ragged, idle=idle, fewer=fewer, chain=chain,
                window=window, cap=cap, slopes=slopes)


def _copy(name, count, heads, dim, cache, page, order="thd", part=False, idle=False, other=False):
    return dict(name=name, op="copy", count=count, heads=heads, dim=dim, v_dim=dim, cache=cache, page=page, order=order,
                part=part, idle=idle, other=other)


def _compact(name, batch, longest, of, keep, heads, dim, cache, page, order="thd", drafted=False, ragged=False):
    """keep: of so many tokens (a row's last ones, in place, where they are drafted) at most so many stay."""
    return dict(name=name, op="compact", batch=batch, longest=longest, of=of, keep=keep, heads=heads, dim=dim, v_dim=dim,
                cache=cache, page=page, order=order, drafted=drafted, ragged=ragged)


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "paged", "paged", "copy", "compact"])
    heads = rng.choice([1, 2, 3, 4, 8, 8, 12, 16])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
    page, order = rng.choice([1, 7, 16, 16, 32, 48, 64, 128, 256]), rng.choice(["thd", "htd"])
    cache = rng.choice(["bf16", "bf16", "f16", "f32", "e4m3"])
    each = 2 * heads * dim * SIZE[cache]
    if op == "copy":
        count = _log(rng, 1, max(1, int(BIGGEST / 2 / (page * each))))
        c = _copy("", count, heads, dim, cache, page, order, part=rng.random() < 0.3, idle=rng.random() < 0.3,
                  other=rng.random() < 0.3)
    elif op == "compact":
        drafted = rng.random() < 0.5
        batch = _log(rng, 1, 256)
        of = rng.randint(2, 64) if drafted else _log(rng, 16, max(16, min(16384, int(BIGGEST / 2 / (batch * each)))))
        longest = max(of, _log(rng, 64, max(64, min(16384, int(BIGGEST / 2 / (batch * each)))))) if drafted else of
        c = _compact("", batch, longest, of, rng.randint(1, max(1, of // 2)), heads, dim, cache, page, order,
                     drafted=drafted, ragged=rng.random() < 0.5)
    else:
        q_heads = heads * rng.choice([1, 1, 2, 4, 4, 5, 7, 8, 16])
        dtype, cache = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f16", "f16"),
                                   ("f16", "e4m3"), ("f32", "f32"), ("f32", "bf16"), ("f32", "e4m3")])
        v_dim = rng.choice([dim, dim, dim, 64, 128])
        drafts = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 16, 32, 33, 64]) if op == "tree" else 0
        batch = _log(rng, 1, 256 if drafts < 32 else 32)
        top = min(131072, int(BIGGEST / (batch * heads * (dim + v_dim) * SIZE[cache])),
                  int(SCORES / (batch * max(drafts, 1) * q_heads)))
        longest = _log(rng, 64, max(64, top))
        ragged = rng.random() < 0.6
        score = rng.choice(["cap", "slopes", "both"]) if op == "paged" else rng.choice(["", "", "cap", "slopes", "both"])
        c = _attend("", batch, longest, drafts, q_heads, heads, dim, dtype, cache, page,
                    out="f32" if rng.random() < 0.2 else dtype, v_dim=v_dim, order=order, ragged=ragged,
                    idle=ragged and rng.random() < 0.5, fewer=drafts > 1 and rng.random() < 0.4,
                    chain=drafts > 0 and rng.random() < 0.3, window=_log(rng, 1, longest) if rng.random() < 0.25 else 0,
                    cap=rng.choice([15.0, 30.0, 50.0]) if score in ("cap", "both") else 0.0,
                    slopes=score in ("slopes", "both"))
    del c["name"]
    return c


def _lengths(c, least=1):
    """The rows' lengths: spread evenly over (0, longest] where they are ragged, every ninth row without a
    request where some are idle."""
    b, top = c["batch"], c["longest"]
    got = [max(least, int(top * ((i * 0.6180339887498949) % 1.0))) if c["ragged"] and i else top for i in range(b)]
    return [0 if c.get("idle") and i % 9 == 4 else n for i, n in enumerate(got)]


def _drafted(c):
    """The rows' numbers of drafted tokens."""
    top = max(c["drafts"], 1)
    got = [1 + (i * 5 + top - 1) % top if c["fewer"] else top for i in range(c["batch"])]
    return [min(n, m) for n, m in zip(got, _lengths(c, top))]


def _kept(c):
    """The rows' numbers of kept tokens."""
    return [1 + (i * 7 + c["keep"] - 1) % c["keep"] if c["ragged"] else c["keep"] for i in range(c["batch"])]


def work(case):
    c = case
    each = 2 * c["heads"] * c["dim"] * SIZE[c["cache"]]
    if c["op"] == "copy":
        live = [i for i in range(c["count"]) if not _no_copy(c, i)]
        tokens = sum(_part(c, i) for i in live)
        return {"bytes": 2 * tokens * each + (12 if c["part"] else 8) * c["count"], "flops": 0}
    if c["op"] == "compact":
        tokens = sum(_kept(c))
        first = c["batch"] if c["drafted"] else 0  # the first drafted token stays where it is
        return {"bytes": 2 * (tokens - first) * each + 4 * tokens + 4 * c["batch"] * (2 if c["drafted"] else 1), "flops": 0}
    lens = _lengths(c, max(c["drafts"], 1))
    drafted = _drafted(c)
    reach = [min(n, c["window"] + m - 1) if c["window"] else n for n, m in zip(lens, drafted)]
    pages = sum(-(-n // c["page"]) for n in reach)
    queries = sum(drafted) if c["op"] == "tree" else c["batch"]
    scores = sum((min(n, c["window"]) if c["window"] else n) * m for n, m in zip(lens, drafted)) * c["q_heads"]
    return {"bytes": sum(reach) * c["heads"] * (c["dim"] + c["v_dim"]) * SIZE[c["cache"]] + 4 * pages + 4 * c["batch"]
            + queries * c["q_heads"] * (c["dim"] * SIZE[c["dtype"]] + c["v_dim"] * SIZE[c["out"]] + 4)
            + (queries * 12 if c["op"] == "tree" else 0),
            "flops": 2 * scores * (c["dim"] + c["v_dim"])}


# --------------------------------------------------------------------------
# inputs

def _normal(gen, shape, dtype, spread=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16 if dtype == "e4m3" else TYPES[dtype])
    if spread != 1.0:
        x.mul_(spread)
    return x.to(TYPES[dtype])


def _pool(gen, pages, dim, c):
    """A cache that other requests have filled before."""
    if c["order"] == "htd":
        return _normal(gen, (pages, c["heads"], c["page"], dim), c["cache"]).transpose(1, 2)
    return _normal(gen, (pages, c["page"], c["heads"], dim), c["cache"])


def _bits(x):
    """An 8-bit cache as whole bytes: torch indexes those."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _table(gen, held, wide, spare):
    """Pages of rows that hold so many each, in no order, and the pages there are."""
    pages = int(held.sum()) + spare
    order = torch.randperm(pages - 1, generator=gen, device="cuda") + 1
    col = torch.arange(wide, device="cuda")
    first = held.cumsum(0) - held
    return torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=pages - 2)], 0), pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"tree": _prepare_attend, "paged": _prepare_attend, "copy": _prepare_copy, "compact": _prepare_compact}[case["op"]](case, gen)


def _trees(c, gen):
    """Each row's tree: a token's parent is one of the four before it (chain: the one before it), a root's is
    the last token of the prefix.  The tokens that each sees, as bits, and their depths."""
    b, n = c["batch"], c["drafts"]
    back = torch.ones((b, n), dtype=torch.int64) if c["chain"] else torch.randint(1, 5, (b, n), generator=gen, device="cuda").cpu()
    masks, depths = torch.zeros((b, n + 1), dtype=torch.int64), torch.full((b, n + 1), -1, dtype=torch.int32)
    rows = torch.arange(b)
    for i in range(n):  # column 0 is the prefix
        parent = (i + 1 - back[:, i]).clamp(min=0)
        masks[:, i + 1] = masks[rows, parent] | torch.tensor(1, dtype=torch.int64) << i
        depths[:, i + 1] = depths[rows, parent] + 1
    return masks[:, 1:].contiguous().cuda(), depths[:, 1:].contiguous().cuda()


def _prepare_attend(c, gen):
    b, hq, h, page, n = c["batch"], c["q_heads"], c["heads"], c["page"], max(c["drafts"], 1)
    mix = torch.randperm(b, generator=gen, device="cuda")
    lens, counts = torch.tensor(_lengths(c, n), device="cuda")[mix], torch.tensor(_drafted(c), device="cuda")[mix]
    held = (lens + page - 1) // page
    table, pages = _table(gen, held, -(-c["longest"] // page), 9)
    k_cache, v_cache = _pool(gen, pages, c["dim"], c), _pool(gen, pages, c["v_dim"], c)
    # the slots after a row's end hold whatever they held: here, no numbers
    last = (lens - 1).clamp(min=0) // page
    after = (torch.arange(page, device="cuda") >= (lens - last * page)[:, None]) & (lens > 0)[:, None]
    at = table.gather(1, last[:, None]).expand(-1, page)
    nan = 0x7F if c["cache"] == "e4m3" else float("nan")
    row = torch.arange(page, device="cuda").expand(b, -1)
    _bits(k_cache)[at[after], row[after]] = nan
    _bits(v_cache)[at[after], row[after]] = nan
    k_scale = v_scale = slopes = None
    if c["cache"] == "e4m3":
        k_scale, v_scale = torch.rand((2, h), generator=gen, device="cuda").add_(0.4)
    if c["slopes"]:  # a geometric row of slopes, one for each query head
        slopes = 2.0 ** (-8.0 * (torch.arange(hq, device="cuda") + 1) / hq)
    shape = (b, n, hq) if c["drafts"] else (b, hq)
    s = dict(case=c, q=_normal(gen, (*shape, c["dim"]), c["dtype"], 3.0 if c["cap"] else 2.0), k_cache=k_cache, v_cache=v_cache,
             k_scale=k_scale, v_scale=v_scale, table=table.to(torch.int32), lens=lens.to(torch.int32), counts=None, masks=None,
             depths=None, slopes=slopes, scale=1.0 / math.sqrt(c["dim"]),
             out=torch.zeros((*shape, c["v_dim"]), device="cuda", dtype=TYPES[c["out"]]), lse=torch.zeros(shape, device="cuda"))
    if c["drafts"]:
        s["counts"] = counts.to(torch.int32) if c["fewer"] else None
        s["masks"], s["depths"] = (None, None) if c["chain"] else _trees(c, gen)
    if own:
        import deterministic_fixed_order_amd as detfold
        s["cache"] = detfold.PagedCache(k_cache, v_cache, k_scale=k_scale, v_scale=v_scale)
        s["workspace"] = detfold.attend_workspace(s["cache"], b, hq, c["longest"], drafts=n)
    return s


def _no_copy(c, i):
    return c["idle"] and i % 9 == 4


def _part(c, i):
    return 1 + (i * 5) % c["page"] if c["part"] else c["page"]


def _prepare_copy(c, gen):
    n, page = c["count"], c["page"]
    pages = 2 * n + 5
    order = torch.randperm(pages - 1, generator=gen, device="cuda") + 1
    src, dst = order[:n].clone(), order[n:2 * n].clone()
    idle = torch.tensor([_no_copy(c, i) for i in range(n)], device="cuda")
    src[idle], dst[idle] = -1, -1  # a list that is padded
    s = dict(case=c, k_cache=_pool(gen, pages, c["dim"], c), v_cache=_pool(gen, pages, c["v_dim"], c),
             src=src.to(torch.int32), dst=dst.to(torch.int32), tokens=None, k_into=None, v_into=None)
    if c["part"]:
        s["tokens"] = torch.tensor([_part(c, i) for i in range(n)], device="cuda", dtype=torch.int32)
    if c["other"]:
        s["k_into"], s["v_into"] = _pool(gen, pages, c["dim"], c), _pool(gen, pages, c["v_dim"], c)
    if own:
        import deterministic_fixed_order_amd as detfold
        s["cache"] = detfold.PagedCache(s["k_cache"], s["v_cache"])
        s["into"] = detfold.PagedCache(s["k_into"], s["v_into"]) if c["other"] else None
    return s


def _prepare_compact(c, gen):
    b, page, of, keep = c["batch"], c["page"], c["of"], c["keep"]
    lens = torch.tensor([max(n, of) for n in _lengths(c)], device="cuda")
    counts = torch.tensor(_kept(c), device="cuda")
    held = (lens + page - 1) // page
    wide = -(-max(c["longest"], of) // page)
    fresh = torch.zeros_like(held) if c["drafted"] else (counts + page - 1) // page
    both, pages = _table(gen, torch.cat([held, fresh]), wide, 9)
    # which tokens stay, ascending: of a tree the first one and then, deeper and deeper, tokens behind its
    # widest level; of a prompt any
    low = keep if c["drafted"] else 0
    picks = torch.rand((b, of - low), generator=gen, device="cuda").argsort(1)[:, :keep].sort(1).values + low
    if c["drafted"]:
        picks = torch.cat([torch.zeros_like(picks[:, :1]), picks], 1)[:, :keep].contiguous()
    s = dict(case=c, k_cache=_pool(gen, pages, c["dim"], c), v_cache=_pool(gen, pages, c["v_dim"], c),
             table=both[:b].to(torch.int32).contiguous(), to=None, starts=None, picks=picks.to(torch.int32),
             counts=counts.to(torch.int32))
    if c["drafted"]:
        s["starts"] = (lens - of).to(torch.int32)
    else:
        s["to"] = both[b:, :-(-keep // page)].to(torch.int32).contiguous()
    if own:
        import deterministic_fixed_order_amd as detfold
        s["cache"] = detfold.PagedCache(s["k_cache"], s["v_cache"])
    return s


# --------------------------------------------------------------------------
# one pass

def run(state):
    return {"tree": _run_attend, "paged": _run_attend, "copy": _run_copy, "compact": _run_compact}[state["case"]["op"]](state)


def _run_attend(s):
    c = s["case"]
    if own:
        import deterministic_fixed_order_amd as detfold
        common = dict(scale=s["scale"], window=c["window"], max_len=c["longest"], lse=s["lse"], workspace=s["workspace"],
                      cap=c["cap"], slopes=s["slopes"])
        if c["drafts"]:
            detfold.attend_tree(s["out"], s["q"], s["cache"], s["table"], s["lens"], masks=s["masks"], counts=s["counts"],
                                depths=s["depths"], **common)
        else:
            detfold.attend_paged(s["out"], s["q"], s["cache"], s["table"], s["lens"], **common)
        return s["out"], s["lse"]
    b, hq, h, n = c["batch"], c["q_heads"], c["heads"], max(c["drafts"], 1)
    k, v = (_bits(x)[s["table"].long()].flatten(1, 2).view(x.dtype).float().transpose(1, 2)
            for x in (s["k_cache"], s["v_cache"]))                                  # [batch, heads, tokens, dim]
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    t, i = torch.arange(k.shape[2], device=k.device), torch.arange(n, device=k.device)
    lens = s["lens"].long()
    counts = torch.minimum(lens, lens.new_tensor(n) if s["counts"] is None else s["counts"].long())
    base = (lens - counts)[:, None]
    depths = i.expand(b, n) if s["depths"] is None else s["depths"].long()
    bit = (t - base).clamp(0, n - 1)                                                # [batch, tokens]: which drafted token
    drafted = (i[:, None] >= bit[:, None]) if s["masks"] is None else (s["masks"][:, :, None] >> bit[:, None] & 1).bool()
    seen = (t < lens[:, None])[:, None] & ((t < base)[:, None] | drafted)           # [batch, drafts, tokens]
    away = torch.where(t < base, t - base, depths.gather(1, bit))[:, None] - depths[:, :, None]
    if c["window"]:
        seen = seen & (away > -c["window"])
    q = s["q"].float().reshape(b, n, h, hq // h, -1).transpose(1, 2).flatten(2, 3)  # [batch, heads, drafts x group, dim]
    score = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).unflatten(2, (n, hq // h))
    if c["cap"]:
        score = torch.tanh(score / c["cap"]) * c["cap"]
    if s["slopes"] is not None:
        score = score + s["slopes"].view(h, 1, hq // h, 1) * away.float()[:, None, :, None]
    score = score.masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.masked_fill((t >= lens[:, None])[:, None, :, None], 0.0)) / total.masked_fill(total == 0, 1.0)
    o = o.unflatten(2, (n, -1)).transpose(1, 2).reshape(s["out"].shape).to(TYPES[c["out"]])
    lse = (top + torch.log(total)).unflatten(2, (n, -1)).transpose(1, 2).reshape(s["lse"].shape)
    if not c["fewer"]:
        return o, lse
    live = (i < counts[:, None])[:, :, None]
    s["out"].copy_(torch.where(live[..., None], o, s["out"]))
    s["lse"].copy_(torch.where(live, lse, s["lse"]))
    return s["out"], s["lse"]


def _run_copy(s):
    c = s["case"]
    to = (s["k_into"], s["v_into"]) if c["other"] else (s["k_cache"], s["v_cache"])
    if own:
        import deterministic_fixed_order_amd as detfold
        detfold.cache_copy(s["cache"], s["src"], s["dst"], tokens=s["tokens"], into=s["into"])
        return to
    src, dst = s["src"].long(), s["dst"].long().clamp(min=0)
    # what pads the list leaves page 0, which belongs to nobody, as it is
    there = (s["src"] >= 0)[:, None].expand(-1, c["page"])
    if c["part"]:
        there = there & (torch.arange(c["page"], device=src.device) < s["tokens"][:, None])
    x, y = _bits(s["k_cache"]), _bits(to[0])
    y[dst] = torch.where(there[:, :, None, None], x[src.clamp(min=0)], y[dst])
    x, y = _bits(s["v_cache"]), _bits(to[1])
    y[dst] = torch.where(there[:, :, None, None], x[src.clamp(min=0)], y[dst])
    return to


def _run_compact(s):
    c = s["case"]
    if own:
        import deterministic_fixed_order_amd as detfold
        detfold.cache_compact(s["cache"], s["table"], s["picks"], s["counts"], starts=s["starts"], to=s["to"])
        return s["k_cache"], s["v_cache"]
    i = torch.arange(s["picks"].shape[1], device=s["picks"].device)
    there = i < s["counts"][:, None]
    first = 0 if s["starts"] is None else s["starts"].long()[:, None]
    src, dst = first + s["picks"].long(), (first + i).expand_as(s["picks"])
    to = s["table"] if s["to"] is None else s["to"]
    # what does not stay leaves page 0, which belongs to nobody, as it is
    at, in_at = (torch.where(there, x, 0) for x in (s["table"].long().gather(1, src // c["page"]), src % c["page"]))
    on, in_on = (torch.where(there, x, 0) for x in
                 (to.long().gather(1, (dst // c["page"]).clamp(max=to.shape[1] - 1)), dst % c["page"]))
    k, v = _bits(s["k_cache"]), _bits(s["v_cache"])
    k[on, in_on] = k[at, in_at]
    v[on, in_on] = v[at, in_at]
    return s["k_cache"], s["v_cache"]


# --------------------------------------------------------------------------
# the definition, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"tree": _exact_attend, "paged": _exact_attend, "copy": _exact_copy, "compact": _exact_compact}[case["op"]](s, case)


def _exact_attend(s, c):
    group, page, n = c["q_heads"] // c["heads"], c["page"], max(c["drafts"], 1)
    out, lse = s["out"].double().view(c["batch"], n, c["q_heads"], -1), s["lse"].double().view(c["batch"], n, c["q_heads"])
    q = s["q"].view(c["batch"], n, c["q_heads"], -1)
    k_bits, v_bits = _bits(s["k_cache"]), _bits(s["v_cache"])
    for b, length in enumerate(s["lens"].tolist()):
        drafted = min(n if s["counts"] is None else int(s["counts"][b]), length)
        live = drafted if c["fewer"] else n
        out[b, :live], lse[b, :live] = 0.0, -math.inf
        if not length:
            continue
        base = length - drafted
        depth = torch.arange(n, device="cuda") if s["depths"] is None else s["depths"][b].long()
        at = torch.cat([torch.arange(base, device="cuda"), base + depth[:drafted]])             # each token's position
        seen = torch.ones((n, length), dtype=torch.bool, device="cuda")
        for i in range(n):
            for j in range(drafted):
                seen[i, base + j] = j <= i if s["masks"] is None else bool(int(s["masks"][b, i]) >> j & 1)
        away = (at[None, :] - (base + depth)[:, None]).double()                                 # [drafts, tokens]
        if c["window"]:
            seen &= away > -c["window"]
        pages = s["table"][b, :-(-length // page)].long()
        for h in range(c["heads"]):
            k = k_bits[pages, :, h].flatten(0, 1)[:length].contiguous().view(s["k_cache"].dtype).double()
            v = v_bits[pages, :, h].flatten(0, 1)[:length].contiguous().view(s["v_cache"].dtype).double()
            of = slice(h * group, (h + 1) * group)
            x = (q[b, :, of].double().flatten(0, 1) @ k.t()).view(n, group, length) * s["scale"]
            if s["k_scale"] is not None:
                x, v = x * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if s["slopes"] is not None:
                x = x + s["slopes"][of].double()[None, :, None] * away[:, None]
            x = x.masked_fill(~seen[:, None], -math.inf)
            sums = torch.logsumexp(x, -1)
            p = torch.exp(x - sums.masked_fill(sums == -math.inf, 0.0)[..., None])
            lse[b, :live, of] = sums[:live]
            out[b, :live, of] = (p.flatten(0, 1) @ v).view(n, group, -1)[:live]
    return out.view(s["out"].shape), lse.view(s["lse"].shape)


def _exact_copy(s, c):
    to = (s["k_into"], s["v_into"]) if c["other"] else (s["k_cache"], s["v_cache"])
    got = [x.double() for x in to]
    there = torch.nonzero(s["src"] >= 0)[:, 0]
    src, dst = s["src"].long()[there], s["dst"].long()[there]
    for x, y in zip((s["k_cache"], s["v_cache"]), got):
        if s["tokens"] is None:
            y[dst] = _bits(x)[src].view(x.dtype).double()
        else:
            for i, j, n in zip(src.tolist(), dst.tolist(), s["tokens"][there].tolist()):
                y[j, :n] = x[i, :n].double()
    return tuple(got)


def _exact_compact(s, c):
    got, page = [], c["page"]
    to = s["table"] if s["to"] is None else s["to"]
    for x in (s["k_cache"], s["v_cache"]):
        was, now = x.double(), x.double()
        for b, n in enumerate(s["counts"].tolist()):
            first = 0 if s["starts"] is None else int(s["starts"][b])
            src, dst = first + s["picks"][b, :n].long(), first + torch.arange(n, device="cuda")
            now[to[b, dst // page].long(), dst % page] = was[s["table"][b, src // page].long(), src % page]
        got.append(now)
    return tuple(got)
