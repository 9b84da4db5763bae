"""MoeLayer.forward_train with y over x: refused where x itself is kept for the
backward pass, and the same outputs and gradients where it is not."""
import pytest
import torch

from gpu_util import need_gpu
from test_gpu_kept_layer import _moe, moe_layer, rand

pytestmark = pytest.mark.gpu
T = 70


@pytest.mark.parametrize("with_norm,keep", [(False, None), (False, "fp8"), (True, None)])
def test_refused_where_x_is_kept(with_norm, keep):
    moe = _moe()
    need_gpu()
    layer, cfg = moe_layer(T, norm=moe.LayerNorm() if with_norm else None)
    x = rand(T, cfg.d, seed=1)
    before = x.clone()
    with pytest.raises(ValueError, match="kept for backward"):
        layer.forward_train(x, y=x, keep=keep)
    assert torch.equal(x, before)


def test_the_same_results_where_x_is_not_kept():
    moe = _moe()
    need_gpu()
    layer, cfg = moe_layer(T, norm=moe.LayerNorm())
    x, dy = rand(T, cfg.d, seed=1), rand(T, cfg.d, seed=2)

    def step(x, y):
        out = [layer.forward_train(x, y=y, keep="fp8").clone()]
        return out + [v.clone() for v in layer.backward(dy, wgrad=True)] + [layer.norm.dweight, layer.norm.dbias]
    want = step(x, None)
    z = x.clone()
    for a, b in zip(want, step(z, z)):
        assert torch.equal(a, b)
