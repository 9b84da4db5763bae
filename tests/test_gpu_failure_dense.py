"""Waits that run out in the dense block and in the norm's backward pass, made on
the host as in test_gpu_failure.py: MOEFP8_FAULT withholds the loads of a
kernel's first stage and MOEFP8_WAIT_LIMIT_NS shortens its waits.  The kernel
ends by itself with loads of its other stages in flight, the status word says
so, and the next call gives the first one's bits."""
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


def rand(*shape, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).bfloat16()


def runs_out_and_recovers(monkeypatch, fault, call, outs, status):
    import fp8_block_scaled_affinity_b200 as moe
    call()
    torch.cuda.synchronize()
    assert int(status) == 0
    good = [v.clone() for v in outs]
    for _ in range(2):
        monkeypatch.setenv("MOEFP8_FAULT", fault)
        monkeypatch.setenv("MOEFP8_WAIT_LIMIT_NS", "20000")
        call()
        torch.cuda.synchronize()  # returns: the kernels ended by themselves
        assert int(status) == moe.MOE_DEV_TIMEOUT
        monkeypatch.delenv("MOEFP8_FAULT")
        monkeypatch.delenv("MOEFP8_WAIT_LIMIT_NS")
        status.zero_()
        for v in outs:
            v.zero_()
        call()
        torch.cuda.synchronize()
        assert int(status) == 0
        for v, w in zip(outs, good):
            assert torch.equal(v, w)


# few tokens in one and in several parts of K, with fewer K steps than stages
# and with more; pairs of CTAs with one tile each and with several
SIZES = [(40, 256, 136), (40, 4096, 136), (200, 2048, 192), (777, 520, 264), (1500, 4096, 1024)]


@pytest.mark.parametrize("keep", [None, "fp8", "full"])
@pytest.mark.parametrize("T,d,I", SIZES)
def test_dense_block(T, d, I, keep, monkeypatch):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    x, w13, w2 = (rand(T, d, seed=1), rand(2 * I, d, seed=2, scale=d ** -0.5),
                  rand(d, I, seed=3, scale=I ** -0.5))
    h, y = torch.empty(T, I, dtype=x.dtype, device=DEV), torch.empty_like(x)
    wide = (I + 127) // 128 * 128
    ac, s = {None: (None, None), "full": (torch.empty(T, 2 * I, dtype=x.dtype, device=DEV), None),
             "fp8": (torch.empty(T, 2 * wide, dtype=torch.uint8, device=DEV),
                     torch.empty(2 * wide // 128, T, device=DEV))}[keep]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    runs_out_and_recovers(monkeypatch, "ffn_producer",
                          lambda: moe.moe_ffn_forward(x, w13, w2, h, y, ac, s, st),
                          [v for v in (h, y, ac, s) if v is not None], st)
    if keep is None:
        return
    dy = rand(T, d, seed=4)
    dac, h2 = torch.empty(T, 2 * I, dtype=x.dtype, device=DEV), torch.empty_like(h)
    grads = [torch.empty_like(v) for v in (x, w13, w2)]
    runs_out_and_recovers(monkeypatch, "ffn_producer",
                          lambda: moe.moe_ffn_backward(dy, x, w13, w2, ac, s, dac, h2, *grads, st),
                          [dac, h2, *grads], st)


@pytest.mark.parametrize("kept", ["full", "fp8"])
@pytest.mark.parametrize("rows,cols", [(5, 64), (700, 7168), (2000, 520), (900, 333)])
def test_norm_backward(rows, cols, kept, monkeypatch):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    norm = moe.LayerNorm(1 + rand(cols, seed=3, scale=0.1).float())
    x, dy = rand(rows, cols, seed=1), rand(rows, cols, seed=2)
    norm.forward_train(x, keep=kept)
    outs = [torch.empty_like(dy), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)]

    def call():
        for v, w in zip(outs, (norm.backward(dy), norm.dweight, norm.dbias)):
            v.copy_(w)
    runs_out_and_recovers(monkeypatch, "norm_rows", call, outs, norm.dev_status)
    assert norm.status() == 0


def test_a_blocks_status_shows_its_norms_wait(monkeypatch):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    T, d, I = 100, 512, 256
    ffn = moe.GatedFfn(rand(2 * I, d, seed=1, scale=d ** -0.5), rand(d, I, seed=2, scale=I ** -0.5),
                       moe.LayerNorm())
    x, dy = rand(T, d, seed=3), rand(T, d, seed=4)
    ffn.forward_train(x)
    monkeypatch.setenv("MOEFP8_FAULT", "norm_rows")
    monkeypatch.setenv("MOEFP8_WAIT_LIMIT_NS", "200000")  # the dense block's own waits stay below it
    ffn.backward(dy)
    assert ffn.status() == moe.MOE_DEV_TIMEOUT
