"""What a MoeLayer with a norm refuses before its norm runs: the norm takes fp32
and any number of rows, the layer behind it reads bf16 [T, d] at an address."""
import pytest
import torch

import fp8_block_scaled_affinity_b200 as moe


@pytest.fixture
def layer(monkeypatch):
    for name in ("moe_layer_workspace_size", "moe_route_workspace_size", "moe_permute_workspace_size"):
        monkeypatch.setattr(moe, name, lambda shape: 256)
    ran = []
    for name in ("moe_layernorm_forward", "moe_layer_forward", "moe_route_scores", "moe_quant_permute",
                 "moe_grouped_gemm_fp8", "moe_combine"):
        monkeypatch.setattr(moe, name, lambda *a, **k: ran.append(a))
    T, d, N = 4, 128, 8
    it = moe.MoeLayer(moe.make_shape(T, d, N, 1, 1, 2, 128), torch.zeros(N, d, dtype=torch.bfloat16),
                      torch.zeros(N), norm=moe.LayerNorm(torch.ones(d)))
    it.ran = ran
    return it


@pytest.mark.parametrize("how", ["forward", "forward_train"])
@pytest.mark.parametrize("shape,dtype", [((4, 128), torch.float32), ((4, 128), torch.float16),
                                         ((3, 128), torch.bfloat16), ((5, 128), torch.bfloat16),
                                         ((4, 256), torch.bfloat16), ((1, 4, 128), torch.bfloat16)])
def test_refused(layer, how, shape, dtype):
    with pytest.raises(ValueError, match="x must be bf16"):
        getattr(layer, how)(torch.zeros(shape, dtype=dtype))
    assert not layer.ran and layer.norm._kept is None


@pytest.mark.parametrize("how", ["forward", "forward_train"])
def test_taken(layer, how):
    getattr(layer, how)(torch.zeros(4, 128, dtype=torch.bfloat16))
    assert layer.ran
