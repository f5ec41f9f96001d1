"""``fold_softmax`` of float32 partials rounds as it says: the sum in order, each step
once, and one division by the sum of the weights."""
import pytest

from test_decode_gpu import _gen, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("W", [1, 2, 3, 5, 6, 7, 8, 9, 11, 13, 17])
@pytest.mark.parametrize("rows,dim", [(1, 128), (700, 84), (3, 7), (9001, 256)])
def test_equal_weights_give_the_mean_of_the_sum_in_order(env, W, rows, dim):  # noqa: F811
    """With equal lses every weight is exactly 1 and their sum exactly W."""
    df, torch, dev = env
    outs = torch.randn((W, rows, dim), generator=_gen(torch, 81, W))
    lses = torch.full((W, rows), 2.5)
    lses[:, rows // 2] = -3e4
    out = torch.empty((rows, dim), device=dev)
    df.fold_softmax(out, outs.to(dev), lses.to(dev))
    want = outs[0].clone()
    for w in range(1, W):
        want = want + outs[w]
    assert torch.equal(out.cpu(), want / W)
