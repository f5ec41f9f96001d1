"""The decode-step operators on a stream that the caller names (``stream=``), not
torch's current one: the same bits as on the current stream, also where a call
allocates its own workspace while the current stream allocates and writes."""
import pytest

from test_decode_gpu import _attend_case, _fold_case, _gen, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[3000, 0, 17, 2999], [70001], [40, 3, 0]])
@pytest.mark.parametrize("own", [True, False])
def test_attend_on_a_stream(env, lens, own):  # noqa: F811
    df, torch, dev = env
    c, q, table, ln, out, lse = _attend_case(env, lens, 8, 2, 128, 128, "bf16", "bf16", 16)
    need = df.attend_workspace(c, len(lens), 8, max(lens))
    s = torch.cuda.Stream()
    o, l = (torch.zeros((6, *x.shape), device=dev, dtype=x.dtype) for x in (out, lse))
    s.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        if own:
            df.attend_paged(o[i], q, c, table, ln, max_len=max(lens), lse=l[i], workspace=need, stream=s)
        else:
            df.attend_paged(o[i], q, c, table, ln, max_len=max(lens), lse=l[i], stream=s)
            # of the size that the call has just given back
            torch.full((need.nbytes,), 255, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    for i in range(6):
        assert torch.equal(o[i], out) and torch.equal(l[i], lse), i


def test_a_workspace_is_not_handed_to_another_stream(env):  # noqa: F811
    """The block of a call's own workspace is the named stream's."""
    df, torch, dev = env
    c, q, table, ln, out, lse = _attend_case(env, [3000, 2999], 8, 2, 128, 128, "bf16", "bf16", 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    made, alloc = [], df.decode.attend_workspace

    def seen(*a, **k):
        made.append(torch.cuda.current_stream().cuda_stream)
        return alloc(*a, **k)
    df.decode.attend_workspace = seen
    try:
        df.attend_paged(torch.empty_like(out), q, c, table, ln, max_len=3000, stream=s)
        df.attend_paged(torch.empty_like(out), q, c, table, ln, max_len=3000)
    finally:
        df.decode.attend_workspace = alloc
    torch.cuda.synchronize()
    assert made == [s.cuda_stream, torch.cuda.current_stream().cuda_stream]


def test_append_on_a_stream(env):  # noqa: F811
    df, torch, dev = env
    gen = _gen(torch, 31)
    k, v, q = (torch.randn((67, h, 64), generator=gen).bfloat16().to(dev) for h in (2, 2, 8))
    angle = torch.arange(200.0, device=dev)[:, None] * torch.linspace(1, 0.1, 32, device=dev)
    cos, sin, pos = angle.cos(), angle.sin(), torch.arange(67, device=dev)
    slots = torch.randperm(128, generator=gen)[:67].to(dev)
    got = []
    for s in (None, torch.cuda.Stream()):
        pools = [torch.zeros((8, 16, 2, 64), device=dev, dtype=torch.bfloat16) for _ in range(2)]
        qo = torch.zeros_like(q)
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        df.cache_append(df.PagedCache(*pools), k, v, slots, q=q, q_out=qo, positions=pos, cos=cos, sin=sin, stream=s)
        torch.cuda.synchronize()
        got.append(pools + [qo])
    for a, b in zip(*got):
        assert bool(a.any()) and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_fold_on_a_stream(env, dtype):  # noqa: F811
    df, torch, dev = env
    outs, lses, out, lse = _fold_case(env, 5, (700,), 84, dtype, empty=0.2)
    s = torch.cuda.Stream()
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    s.wait_stream(torch.cuda.current_stream())
    df.fold_softmax(o, outs, lses, lse=l, stream=s)
    s.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
