"""The first call of a host thread: nothing has made a CUDA context current in it."""
import threading

import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


def in_a_new_thread(call):
    errors = []

    def run():
        try:
            call()
        except Exception as e:  # reported by the test's own thread
            errors.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors


@pytest.mark.parametrize("T", [1, 40, 600])
def test_dense_block(T):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    d, I = 512, 256
    x, w13 = (torch.randn(n, d, device=DEV).bfloat16() for n in (T, 2 * I))
    w2 = torch.randn(d, I, device=DEV).bfloat16()
    h, ac = (torch.empty(T, n, dtype=x.dtype, device=DEV) for n in (I, 2 * I))
    want, y = torch.empty_like(x), torch.zeros_like(x)
    stream = torch.cuda.current_stream()
    moe.moe_ffn_forward(x, w13, w2, h, want, ac)
    in_a_new_thread(lambda: moe.moe_ffn_forward(x, w13, w2, h, y, ac, stream=stream))
    assert torch.equal(y, want)
    grads = [[torch.zeros_like(v) for v in (x, w13, w2)] for _ in range(2)]
    dac = torch.empty_like(ac)
    moe.moe_ffn_backward(x, x, w13, w2, ac, None, dac, h, *grads[0])
    in_a_new_thread(lambda: moe.moe_ffn_backward(x, x, w13, w2, ac, None, dac, h, *grads[1], stream=stream))
    for a, b in zip(*grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("keep", [False, True])
def test_expert_gemm(keep):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    R, k, n = 40, 256, 256
    a, w = (torch.randint(0, 0x70, (m, k), device=DEV).to(torch.uint8) for m in (R, n))
    a_s, w_s = torch.ones(k // 128, R, device=DEV), torch.ones(n // 128, k // 128, device=DEV)
    off = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    stream = torch.cuda.current_stream()

    def call(out):
        h, hs, q, qs = out
        if keep:
            moe.moe_grouped_gemm_fp8_ckpt(1, off, R, a, a_s, k, w, w_s, n, h, hs, q, qs, stream=stream)
        else:
            moe.moe_grouped_gemm_fp8(1, off, R, a, a_s, k, w, w_s, n, moe.MOE_EPI_SWIGLU_QUANT, h, hs,
                                     stream=stream)
    outs = [(torch.zeros(R, n // 2, dtype=torch.uint8, device=DEV), torch.zeros(1, R, device=DEV),
             torch.zeros(R, n, dtype=torch.uint8, device=DEV), torch.zeros(2, R, device=DEV)) for _ in range(2)]
    call(outs[0])
    in_a_new_thread(lambda: call(outs[1]))
    for u, v in zip(*outs):
        assert torch.equal(u, v)


def test_norm_and_checkpoint():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    x = torch.randn(50, 512, device=DEV)
    stream = torch.cuda.current_stream()
    outs = []
    for run in (lambda f: f(), in_a_new_thread):
        y, mean, rstd = torch.zeros_like(x), torch.zeros(50, device=DEV), torch.zeros(50, device=DEV)
        q, s = torch.zeros(50, 512, dtype=torch.uint8, device=DEV), torch.zeros(4, 50, device=DEV)
        dx, dw, db = torch.zeros_like(x), torch.zeros(512, device=DEV), torch.zeros(512, device=DEV)
        ws = torch.empty(moe.moe_layernorm_backward_workspace_size(50, 512), dtype=torch.uint8, device=DEV)
        run(lambda: moe.moe_layernorm_forward(x, None, None, 1e-5, y, mean, rstd, stream=stream))
        run(lambda: moe.moe_ckpt_pack(x, q, s, stream=stream))
        run(lambda: moe.moe_layernorm_backward(x, q, s, None, mean, rstd, dx, dw, db, ws, stream=stream))
        outs.append((y, mean, rstd, q, s, dx, dw, db))
    for u, v in zip(*outs):
        assert torch.equal(u, v)
