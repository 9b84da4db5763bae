"""Which status word the norm's backward pass reports on: its own, or that of the
layer whose norm it is (the library's calls recorded, no GPU)."""
import pytest
import torch

import fp8_block_scaled_affinity_b200 as moe


@pytest.fixture
def words(monkeypatch):
    """The status words that moe_layernorm_backward is given."""
    seen = []

    def backward(dy, x, scales, weight, mean, rstd, dx, dweight, dbias, ws, dev_status=None, stream=None):
        seen.append(dev_status)
    monkeypatch.setattr(moe, "moe_layernorm_backward", backward)
    for name in ("moe_layernorm_forward", "moe_ffn_forward", "moe_ffn_backward"):
        monkeypatch.setattr(moe, name, lambda *a, **k: None)
    monkeypatch.setattr(moe, "moe_layernorm_backward_workspace_size", lambda rows, cols: 64)
    return seen


@pytest.mark.parametrize("weight", [None, torch.ones(8)])
def test_a_norm_alone_reports_on_its_own_word(words, weight):
    norm = moe.LayerNorm(weight)
    x = torch.zeros(2, 8)
    norm.forward_train(x)
    norm.backward(x)
    assert words[0] is norm.dev_status
    assert words[0].dtype == torch.int32 and words[0].tolist() == [0]
    other = torch.zeros(1, dtype=torch.int32)
    norm.backward(x, dev_status=other)
    assert words[1] is other
    norm.backward(x)
    assert words[2] is words[0]


def test_status_reads_the_word(words, monkeypatch):
    monkeypatch.setattr(moe, "moe_read_status", lambda word, stream: int(word))
    norm = moe.LayerNorm()
    assert norm.status() == 0  # nothing has run
    x = torch.zeros(2, 8)
    norm.forward_train(x)
    norm.backward(x)
    norm.dev_status.fill_(moe.MOE_DEV_TIMEOUT)
    assert norm.status() == moe.MOE_DEV_TIMEOUT


def test_a_dense_blocks_norm_reports_on_the_blocks_word(words):
    ffn = moe.GatedFfn(torch.zeros(16, 8), torch.zeros(8, 8), moe.LayerNorm(torch.ones(8)))
    x = torch.zeros(2, 8)
    ffn.forward_train(x, keep="full")
    ffn.backward(x)
    assert words[0] is ffn.dev_status


def test_an_expert_layers_norm_reports_on_the_layers_word(words, monkeypatch):
    """MoeLayer.backward with every stage's call recorded only."""
    for name in ("moe_combine_backward_quant", "moe_grouped_gemm_fp8", "moe_swiglu_backward_quant",
                 "moe_gate_backward", "moe_router_backward", "moe_dx_combine", "moe_route_scores",
                 "moe_quant_permute", "moe_combine", "fp8_transpose_w_128x128"):
        monkeypatch.setattr(moe, name, lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: None)
    for name in ("moe_layer_workspace_size", "moe_route_workspace_size", "moe_permute_workspace_size",
                 "moe_router_backward_workspace_size"):
        monkeypatch.setattr(moe, name, lambda shape: 256)
    T, d, N = 4, 128, 8
    layer = moe.MoeLayer(moe.make_shape(T, d, N, 1, 1, 2, 128), torch.zeros(N, d, dtype=torch.bfloat16),
                         torch.zeros(N), norm=moe.LayerNorm(torch.ones(d)))
    x = torch.zeros(T, d, dtype=torch.bfloat16)
    layer.forward_train(x)
    layer.backward(x)
    assert words[0] is layer.dev_status
