"""One LayerNorm in front of two layers: each layer's backward pass goes through
what its own forward_train kept, whichever ran last."""
import pytest
import torch

from gpu_util import need_gpu
from test_gpu_kept_layer import _moe, moe_layer, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keep", ["fp8", "full"])
def test_two_layers_with_one_norm(keep):
    moe = _moe()
    need_gpu()
    T = 70
    weight = None

    def layers(one):
        nonlocal weight
        expert, cfg = moe_layer(T)
        if weight is None:
            weight = 1 + rand(cfg.d, seed=3, scale=0.1, dt=torch.float32)
        norms = [moe.LayerNorm(weight)] * 2 if one else [moe.LayerNorm(weight), moe.LayerNorm(weight)]
        expert.norm = norms[0]
        w13, w2 = rand(512, cfg.d, seed=1, scale=cfg.d ** -0.5), rand(cfg.d, 256, seed=2, scale=0.06)
        return [expert, moe.GatedFfn(w13, w2, norms[1])], cfg.d

    def run(one):
        pair, d = layers(one)
        x = [rand(T, d, seed=5 + k) for k in range(2)]
        dy = rand(T, d, seed=9)
        out = []
        for order in ((0, 1), (1, 0)):
            for k in (0, 1):
                pair[k].forward_train(x[k], **({} if keep == "full" and k == 0 else {"keep": keep}))
            for k in order:
                out += [v.clone() for v in pair[k].backward(dy)]
                out += [pair[k].norm.dweight, pair[k].norm.dbias]
        return out
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
