"""The SwiGLU gradient from kept codes has the bits of the same step from those
codes' values in fp32: one arithmetic, two sources."""
import pytest
import torch

from gpu_util import DEV, need_gpu
from test_gpu_norm_ckpt import kept_ac, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,I", [(1, 128), (33, 256), (1280, 256), (700, 2048)])
def test_codes_and_scales_of_both_forms_are_equal(rows, I):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    q0, s0, v = kept_ac(moe, rows, I)
    v[0, :4] = torch.tensor([0.0, -200.0, 200.0, -88.5], device=DEV)  # e^-a from 0 to infinity
    moe.moe_ckpt_pack(v, q0, s0)
    moe.moe_ckpt_unpack(q0, s0, v)
    dh = rand(rows, I, seed=7)

    def out():
        return (torch.empty(rows, 2 * I, dtype=torch.uint8, device=DEV),
                torch.empty(2 * I // 128, rows, device=DEV))
    a, b = out(), out()
    moe.moe_swiglu_backward_quant_ckpt(dh, q0, s0, rows, I, rows, *a)
    moe.moe_swiglu_backward_quant(dh, v, rows, I, rows, *b)
    assert torch.equal(a[1], b[1])
    # (a zero's sign is no matter)
    differ = (a[0] != b[0]) & ((a[0] | b[0]) & 0x7F != 0)
    assert not differ.any(), int(differ.sum())
