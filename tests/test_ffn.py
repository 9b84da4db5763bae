"""The dense gated block: refusals before any CUDA call (no GPU)."""
import pytest
import torch

from test_norm_ckpt import A, ALIGN, ARG, NULL, SHAPE, moe  # noqa: F401


def test_forward_refusals(moe):  # noqa: F811
    L = moe.lib()

    def f(x=A, w13=A, w2=A, ty=1, T=4, d=64, I=32, h=A, y=A, ac=None, at=3, s=None):
        return L.moe_ffn_forward(x, w13, w2, ty, T, d, I, h, y, ac, at, s, None, None)
    assert f(ty=0) == ARG and f(ty=3) == ARG
    assert f(T=-1) == SHAPE and f(T=(1 << 24) + 1) == SHAPE
    for n in (0, 4, 12, -8, (1 << 20) + 8):
        assert f(d=n) == SHAPE and f(I=n) == SHAPE
    for k in ("x", "w13", "w2", "h", "y"):
        assert f(**{k: None}) == NULL and f(**{k: A + 8}) == ALIGN
    assert f(ac=A, at=3) == NULL and f(ac=A, at=2) == ARG and f(ac=A, at=0) == ARG
    assert f(ac=A + 8, at=1) == ALIGN
    assert f(T=0, x=None, y=None) == 0


def test_backward_refusals(moe):  # noqa: F811
    L = moe.lib()

    def f(dy=A, x=A, w13=A, w2=A, ac=A, at=3, s=A, ty=1, T=4, d=64, I=32, dac=A, h=A, dx=A, dw13=A,
          dw2=A):
        return L.moe_ffn_backward(dy, x, w13, w2, ac, at, s, ty, T, d, I, dac, h, dx, dw13, dw2, None,
                                  None)
    assert f(ty=0) == ARG and f(at=0) == ARG and f(at=2) == ARG
    assert f(d=12) == SHAPE and f(I=4) == SHAPE and f(T=-1) == SHAPE
    for k in ("dy", "x", "w13", "w2", "ac", "s", "dac", "h"):
        assert f(**{k: None}) == NULL
    for k in ("dy", "x", "w13", "w2", "ac", "dac", "h", "dx", "dw13", "dw2"):
        assert f(**{k: A + 8}) == ALIGN
    assert f(T=0, dy=None, dw13=None, dw2=None) == 0


def test_binding_refusals(moe):  # noqa: F811
    x, w13, w2 = torch.zeros(4, 64), torch.zeros(64, 64), torch.zeros(64, 32)
    with pytest.raises(ValueError, match="current CUDA device"):
        moe.moe_ffn_forward(x.bfloat16(), w13.bfloat16(), w2.bfloat16(), x, x)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_ffn_forward(x.double(), w13, w2, x, x)
    for ac, s in ((None, x), (torch.zeros(4, 256, dtype=torch.uint8), None), (x, x)):
        with pytest.raises(ValueError, match="ac_scales goes with"):
            moe._lib._kept_ac(ac, s, torch.float32, 4, 32)
