"""The norm's backward pass for rows whose mean is far above their spread: xh =
(x - mean) rstd is the difference first, whose error is relative to xh and not
to |mean| rstd, whatever form the row's alignment and width select.

Tolerances as in test_gpu_norm_ckpt.py, with xh off by at most 3 U |xh|: the
difference (of a kept value: code times scale less the mean, rounded once), the
product, and one spare."""
import pytest
import torch

from gpu_util import DEV, need_gpu
from test_gpu_norm_ckpt import DT, U, half, pack, rand, unpack64

pytestmark = pytest.mark.gpu


def reference(dy, X, w, mean, rstd):
    dy, X = dy.double(), X.double()
    r = rstd.double()[:, None]
    xh = (X - mean.double()[:, None]) * r
    g = dy * w.double()
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - m1 - xh * m2)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    dxh = 3 * U * xh.abs()
    err2 = 64 * U * a2 + (g.abs() * dxh).mean(1, keepdim=True)
    tol = r * (8 * U * g.abs() + 64 * U * a1 + xh.abs() * err2 + m2.abs() * dxh
               + 8 * U * (xh * m2).abs() + 4 * U * m1.abs())
    depth = -(-dy.shape[0] // 100) + 40  # rows of a CTA, then the CTAs' partial rows
    dw = (dy * xh).sum(0)
    return dx, tol, dw, depth * U * (dy * xh).abs().sum(0) + (dy.abs() * dxh).sum(0)


# whole 16-byte pieces, odd rows, and the widths and bases that are not streamed
@pytest.mark.parametrize("kept", ["full", "fp8"])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,shift", [(300, 1024, 0), (300, 1000, 0), (40, 7168, 0), (300, 333, 0),
                                             (5, 9000, 0), (5, 9001, 0), (300, 1024, 1)])
def test_norm_backward_far_from_zero(rows, cols, shift, t, kept):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    dt = DT[t]
    # bf16 steps at 4096 are 32: spread over a few of them
    x = (4096 + (64 if t == "bf16" else 1) * rand(rows, cols, seed=1)).to(dt)
    w = 1 + 0.1 * rand(cols, seed=4)
    base = torch.empty(rows * cols + 8, dtype=dt, device=DEV)
    dy = base[shift:shift + rows * cols].view(rows, cols)
    dy.copy_(rand(rows, cols, seed=6) + 1)
    xs, X = None, x
    if kept == "fp8":
        x, xs = pack(moe, x)
        X = unpack64(x, xs, cols)
    # any fp32 number may stand for the mean: this one has all its bits
    mean = (X.double().mean(1) + 0.3 * rand(rows, seed=8).double()).float()
    rstd = ((X.double() - mean.double()[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    dx, dw, db = torch.empty_like(dy), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(moe.moe_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
    moe.moe_layernorm_backward(dy, x, xs, w, mean, rstd, dx, dw, db, ws)
    rx, tx, rw, tw = reference(dy, X, w, mean, rstd)
    tx = tx + half(dt) * (rx.abs() + tx)
    assert ((dx.double() - rx).abs() <= tx).all()
    assert ((dw.double() - rw).abs() <= tw).all()
