"""A ``PagedCache`` is used where its tensors lie at the time of a call, also where
they were given other memory since it was made, or share theirs with a lazy copy."""
import pytest

from test_decode_copy_on_write_gpu import _setup
from test_decode_gpu import env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["lazy copy", "other memory"])
def test_a_cache_is_used_where_it_is(env, how):  # noqa: F811
    df, torch, dev = env
    pools, k, v, q, table, lens = _setup(torch, dev)
    c = df.PagedCache(*pools)
    held = [x.clone() for x in pools]
    if how == "lazy copy":
        kept = [torch._lazy_clone(x) for x in pools]
    else:
        kept = [x.detach() for x in pools]  # the old memory, which stays here
        for x in pools:
            x.data = x.clone()
    slots = torch.tensor([3, 17, 127, 64, 40], device=dev)
    df.cache_append(c, k, v, slots)
    for x, new, was, old in zip(pools, (k, v), held, kept):
        assert torch.equal(x.flatten(0, 1)[slots], new)
        assert torch.equal(old, was)
    out, want = torch.empty_like(q), torch.empty_like(q)
    df.attend_paged(out, q, c, table, lens, max_len=128)
    df.attend_paged(want, q, df.PagedCache(*(x.clone() for x in pools)), table, lens, max_len=128)
    assert torch.equal(out, want)


def test_a_cache_of_another_layout_is_refused(env):  # noqa: F811
    df, torch, dev = env
    pools, k, v, q, table, lens = _setup(torch, dev)
    c = df.PagedCache(*pools)
    pools[1].data = pools[1][:4].clone()
    for call in (lambda: df.cache_append(c, k, v, torch.arange(5, device=dev)),
                 lambda: df.attend_paged(torch.empty_like(q), q, c, table, lens, max_len=128)):
        with pytest.raises(ValueError, match="cache"):
            call()


@pytest.mark.parametrize("how", ["contiguous", "head-major"])
def test_scales_and_strides_as_they_are_now(env, how):  # noqa: F811
    df, torch, dev = env
    pools, k, v, q, table, lens = _setup(torch, dev)
    pools = [x.to(torch.float8_e4m3fn) for x in pools]
    scales = [torch.rand(2, device=dev) + 0.5 for _ in range(2)]
    c = df.PagedCache(*pools, k_scale=scales[0], v_scale=scales[1])
    kept = pools[0].detach(), pools[1].detach(), scales[0].detach(), scales[1].detach()
    was = [x.clone() for x in kept]
    for x in pools:
        x.data = x.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(x.dtype) if how == "head-major" else x.clone()
    for x in scales:
        x.data = x * 2
    slots = torch.tensor([3, 17, 127, 64, 40], device=dev)
    df.cache_append(c, k, v, slots)
    fresh = df.PagedCache(*pools, k_scale=scales[0], v_scale=scales[1])
    out, want = torch.empty_like(q), torch.empty_like(q)
    df.attend_paged(out, q, c, table, lens, max_len=128)
    df.attend_paged(want, q, fresh, table, lens, max_len=128)
    assert torch.equal(out, want)
    new = (k.float() / scales[0][:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(pools[0].view(torch.uint8).reshape(128, 2, 64)[slots], new.view(torch.uint8))
    for x, y in zip(kept, was):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
