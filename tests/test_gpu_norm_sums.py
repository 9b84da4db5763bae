"""The norm's parameter gradients when calls follow one another on one stream and
share a workspace: the second kernel of a call starts under the first, and must
add up that call's partial sums and not what the workspace held before."""
import pytest
import torch

from gpu_util import DEV, need_gpu
from test_gpu_norm_ckpt import rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(3, 64), (700, 520), (1500, 7168), (400, 9001)])
def test_calls_in_turn_on_one_workspace(rows, cols):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    x = rand(rows, cols, seed=1)
    mean, rstd = x.mean(1), x.var(1, correction=0).add(1e-5).rsqrt()
    w = 1 + 0.1 * rand(cols, seed=2)
    ws = torch.full((moe.moe_layernorm_backward_workspace_size(rows, cols),), 0xFF, dtype=torch.uint8, device=DEV)
    dys = [rand(rows, cols, seed=3 + k) for k in range(3)]

    def call(dy):
        dx, dw, db = torch.empty_like(dy), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        moe.moe_layernorm_backward(dy, x, None, w, mean, rstd, dx, dw, db, ws)
        return dw, db
    want = []
    for dy in dys:
        want.append(call(dy))
        torch.cuda.synchronize()
    got = [(k % 3, call(dys[k % 3])) for k in range(60)]
    torch.cuda.synchronize()
    for k, (dw, db) in got:
        assert torch.equal(dw, want[k][0]) and torch.equal(db, want[k][1])
