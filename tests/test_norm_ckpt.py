"""Layer norm and 8-bit checkpoints: refusals before any CUDA call (no GPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_block_scaled_affinity_b200 as m
    return m


A, ODD = 1 << 20, (1 << 20) + 2  # addresses that no call reaches
NULL, SHAPE, ALIGN, WS, ARG = -1, -2, -5, -6, -7


def test_norm_refusals(moe):
    L = moe.lib()

    def fwd(x=A, ty=1, rows=4, cols=64, w=A, b=A, eps=1e-5, y=A):
        return L.moe_layernorm_forward(x, ty, rows, cols, w, b, eps, y, A, A, None, None)
    assert fwd(ty=3) == ARG and fwd(ty=-1) == ARG
    assert fwd(eps=-1.0) == ARG and fwd(eps=float("nan")) == ARG
    assert fwd(cols=0) == SHAPE and fwd(cols=16385) == SHAPE and fwd(rows=-1) == SHAPE
    assert fwd(rows=1 << 31) == SHAPE
    assert fwd(x=None) == NULL and fwd(y=None) == NULL
    assert fwd(x=A + 1) == ALIGN and fwd(ty=0, x=ODD) == ALIGN and fwd(w=ODD) == ALIGN
    assert fwd(rows=0, x=None, y=None) == 0

    def bwd(dy=A, ty=1, x=A, xt=1, xs=None, rows=4, cols=64, w=A, m=A, r=A, dx=A, dw=A, ws=A, n=1 << 30):
        return L.moe_layernorm_backward(dy, ty, x, xt, xs, rows, cols, w, m, r, dx, dw, dw, ws, n, None,
                                        None)
    assert bwd(ty=3) == ARG and bwd(ty=1, xt=0) == ARG and bwd(ty=1, xt=2) == ARG
    assert bwd(cols=16385) == SHAPE
    for k in ("dy", "x", "m", "r", "dx"):
        assert bwd(**{k: None}) == NULL
    assert bwd(xt=3) == NULL  # codes without scales
    assert bwd(xt=3, xs=A, x=A + 8) == ALIGN and bwd(dy=A + 1) == ALIGN
    assert bwd(ws=None) == WS and bwd(n=16) == WS and bwd(ws=A + 8) == ALIGN
    assert L.moe_layernorm_backward_workspace_size(-1, 64) == 0
    assert L.moe_layernorm_backward_workspace_size(3, 64) == 3 * 2 * 64 * 4


def test_checkpoint_refusals(moe):
    L = moe.lib()
    assert [L.moe_ckpt_row_bytes(n) for n in (0, 1, 128, 129, -1)] == [0, 128, 128, 256, -1]

    def pack(x=A, ty=1, rows=4, cols=64, q=A, s=A):
        return L.moe_ckpt_pack(x, ty, rows, cols, q, s, None, None)

    def unpack(q=A, s=A, rows=4, cols=64, y=A, ty=1):
        return L.moe_ckpt_unpack(q, s, rows, cols, y, ty, None, None)
    for f in (pack, unpack):
        assert f(ty=3) == ARG and f(rows=-1) == SHAPE and f(cols=-1) == SHAPE
        assert f(q=None) == NULL and f(s=None) == NULL and f(q=A + 8) == ALIGN
        assert f(rows=0, q=None) == 0 and f(cols=0, s=None) == 0
    assert pack(x=None) == NULL and pack(x=A + 1) == ALIGN and unpack(ty=0, y=ODD) == ALIGN

    def swiglu(dh=A, q=A, s=A, rows=4, inter=128, total=4, o=A, os=A):
        return L.moe_swiglu_backward_quant_ckpt(dh, q, s, rows, inter, total, o, os, None, None)
    assert swiglu(inter=100) == SHAPE and swiglu(total=3) == SHAPE and swiglu(rows=-1) == SHAPE
    assert swiglu(rows=0, dh=None) == 0 and swiglu(q=None) == NULL and swiglu(q=A + 8) == ALIGN
    assert L.moe_wgrad_quant_h_ckpt(A, A, 4, 100, A, 1, A, A, None, None) == SHAPE
    assert L.moe_wgrad_quant_h_ckpt(None, A, 4, 128, A, 1, A, A, None, None) == NULL
    assert L.moe_wgrad_quant_dac_ckpt(A, A, None, 4, 128, A, 1, A, A, None, None) == NULL
    assert L.moe_wgrad_quant_dac_ckpt(A, A + 8, A, 4, 128, A, 1, A, A, None, None) == ALIGN
    def gemm(out=A, os=A, q=A, s=A, n=256, rows=8):
        return L.moe_grouped_gemm_fp8_ckpt(1, A, rows, A, A, 128, A, A, n, out, os, q, s, None, None)
    assert gemm(q=None) == NULL and gemm(s=None) == NULL and gemm(os=None) == NULL
    assert gemm(q=A + 8) == ALIGN and gemm(n=384) == SHAPE and gemm(rows=0, q=None, s=None) == 0
    sh = moe.make_shape(4, 128, 8, 1, 1, 2, 128)
    assert L.moe_gate_backward_ckpt(ctypes.byref(sh), A, A, None, A, A, A, A, None, None) == NULL
    assert L.moe_gate_backward_ckpt(ctypes.byref(sh), A, A + 8, A, A, A, A, A, None, None) == ALIGN


def test_bindings_refuse_what_the_library_cannot_see(moe):
    """Host tensors, other shapes and strides, other dtypes."""
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="current CUDA device"):
        moe.moe_layernorm_forward(x, None, None, 1e-5, x)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_layernorm_forward(x.double(), None, None, 1e-5, x)
    with pytest.raises(ValueError, match="current CUDA device"):
        moe.moe_ckpt_pack(x, torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4))
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_ckpt_unpack(x, x, torch.zeros(4, 128, dtype=torch.uint8))
    # what a tensor on the right device is refused for
    class Fake:
        is_cuda, device, shape, dtype = True, torch.device("cuda:0"), (4, 64), torch.float32

        def is_contiguous(self):
            return False
    real = torch.cuda.current_device
    try:
        torch.cuda.current_device = lambda: 0
        with pytest.raises(ValueError, match="shape"):
            moe._lib._mat("x", Fake(), (4, 65))
        with pytest.raises(ValueError, match="contiguous"):
            moe._lib._mat("x", Fake(), (4, 64))
        torch.cuda.current_device = lambda: 1
        with pytest.raises(ValueError, match="current CUDA device"):
            moe._lib._mat("x", Fake(), (4, 64))
    finally:
        torch.cuda.current_device = real
