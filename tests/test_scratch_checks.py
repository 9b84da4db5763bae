"""Workspaces and status words of the norm's, the checkpoints' and the dense
block's calls: refused on another device than the call's, or in pieces, before
the library gets an address that the GPU cannot use (no GPU: stand-ins for
tensors on a device)."""
import pytest
import torch

import fp8_block_scaled_affinity_b200 as moe
from fp8_block_scaled_affinity_b200 import _lib


class OnDevice:
    """What the bindings read of a contiguous tensor on CUDA device 0."""
    is_cuda, device = True, torch.device("cuda:0")

    def __init__(self, *shape, dtype=torch.bfloat16, dense=True):
        self.shape, self.dtype, self.dense = torch.Size(shape), dtype, dense

    def get_device(self):
        return 0

    def is_contiguous(self):
        return self.dense

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1


@pytest.fixture
def calls(monkeypatch):
    """The arguments that reach the library."""
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: seen.append(args) or 0
    monkeypatch.setattr(_lib, "lib", Library)
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    monkeypatch.setattr(_lib, "_stream", lambda stream: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return seen


def all_calls(word):
    T, d, I = 4, 64, 32
    f32, u8 = torch.float32, torch.uint8
    x, y, col, row = OnDevice(T, d), OnDevice(T, d), OnDevice(d, dtype=f32), OnDevice(T, dtype=f32)
    w13, w2, h, ac = OnDevice(2 * I, d), OnDevice(d, I), OnDevice(T, I), OnDevice(T, 2 * I)
    q, s = OnDevice(T, 128, dtype=u8), OnDevice(1, T, dtype=f32)
    aq, a_s = OnDevice(T, 256, dtype=u8), OnDevice(2, T, dtype=f32)
    ws = OnDevice(64, dtype=u8)
    return [lambda: moe.moe_layernorm_forward(x, col, col, 1e-5, y, row, row, word),
            lambda: moe.moe_layernorm_backward(x, x, None, col, row, row, y, col, col, ws, word),
            lambda: moe.moe_ckpt_pack(x, q, s, word), lambda: moe.moe_ckpt_unpack(q, s, x, word),
            lambda: moe.moe_swiglu_backward_quant_ckpt(OnDevice(T, 128, dtype=f32), aq, a_s, T, 128, T, aq, a_s,
                                                       word),
            lambda: moe.moe_ffn_forward(x, w13, w2, h, y, ac, None, word),
            lambda: moe.moe_ffn_backward(x, x, w13, w2, ac, None, ac, h, y, w13, w2, word)]


def test_status_words(calls):
    for word, at in ((OnDevice(1, dtype=torch.int32), 1 << 20), (None, None), (4096, 4096)):
        for call in all_calls(word):
            call()
            assert calls.pop()[-2] == at
    for call in all_calls(torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="dev_status.*current CUDA device"):
            call()
    assert not calls


def test_workspace_of_the_norms_backward_pass(calls):
    x, row, col = OnDevice(4, 64), OnDevice(4, dtype=torch.float32), OnDevice(64, dtype=torch.float32)

    def call(ws):
        moe.moe_layernorm_backward(x, x, None, None, row, row, OnDevice(4, 64), col, col, ws)
    call(OnDevice(4096, dtype=torch.uint8))
    assert calls.pop()[13:15] == (1 << 20, 4096)
    with pytest.raises(ValueError, match="ws.*current CUDA device"):
        call(torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="ws.*contiguous"):
        call(OnDevice(4096, dtype=torch.uint8, dense=False))
    assert not calls
