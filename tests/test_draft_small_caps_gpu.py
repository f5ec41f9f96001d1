"""Caps that binary32 does not hold as a normal number are refused, not taken for none."""
import pytest

from test_decode_gpu import env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [1e-50, -1e-50, 1e-46, 1e-40, 5e-324, -5e-324])
@pytest.mark.parametrize("kept", [False, True])
def test_small_caps_are_refused(env, cap, kept):  # noqa: F811
    df, torch, dev = env
    c = df.PagedCache(*(torch.zeros((4, 16, 2, 64), device=dev) for _ in range(2)))
    q = torch.zeros((1, 2, 4, 64), device=dev)
    out, table = torch.full_like(q, 7.0), torch.zeros((1, 4), dtype=torch.int32, device=dev)
    lens = torch.ones(1, dtype=torch.int32, device=dev)
    work = df.attend_workspace(c, 1, 4, 64, drafts=2) if kept else None
    for call in (lambda: df.attend_tree(out, q, c, table, lens, cap=cap, max_len=64, workspace=work),
                 lambda: df.attend_paged(out[:, 0], q[:, 0], c, table, lens, cap=cap, max_len=64, workspace=work)):
        with pytest.raises((ValueError, df.DetfoldError)) as e:
            call()
        assert getattr(e.value, "rc", df.EINVAL) == df.EINVAL
    assert bool((out == 7.0).all())
