"""Calls of host threads on their own streams and buffers, large and small sizes
of the same kernels: none may change what another's launch is allowed
(concurrent calls on different buffers are independent).

The threads call the library itself with arguments laid out before: most of a
turn is then spent outside the interpreter's lock, and the calls overlap."""
import threading

import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16 = 1


def rand(*shape, scale=1.0):
    return (torch.randn(*shape, device=DEV) * scale).bfloat16()


def norm_call(moe, rows, cols):
    dy, x, dx = rand(rows, cols), rand(rows, cols), torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    args = (dy.data_ptr(), BF16, x.data_ptr(), BF16, None, rows, cols, None, mean.data_ptr(), rstd.data_ptr(),
            dx.data_ptr(), None, None, None, 0, None)
    return moe.lib().moe_layernorm_backward, args, dx, (dy, x, mean, rstd)


def dense_call(moe, T, d, I):
    x, w13, w2 = rand(T, d), rand(2 * I, d, scale=d ** -0.5), rand(d, I, scale=I ** -0.5)
    h, y = torch.empty(T, I, dtype=x.dtype, device=DEV), torch.empty_like(x)
    args = (x.data_ptr(), w13.data_ptr(), w2.data_ptr(), BF16, T, d, I, h.data_ptr(), y.data_ptr(), None, BF16,
            None, None)
    return moe.lib().moe_ffn_forward, args, y, (x, w13, w2, h)


@pytest.mark.parametrize("which", ["norm", "dense"])
def test_threads_with_large_and_small_calls(which):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    # rows of 28 KB and of 1 KB; stages for one CTA an SM and for two
    sizes = [(64, 7168), (64, 256)] if which == "norm" else [(256, 4096, 1024), (40, 512, 192)]
    make = norm_call if which == "norm" else dense_call
    calls = [make(moe, *s) for s in sizes * 2]
    want = []
    for f, args, out, _ in calls:
        assert f(*args, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        want.append(out.clone())
    failed = []

    def loop(f, args, stream):
        torch.cuda.set_device(0)
        handle = stream.cuda_stream
        for i in range(20):
            bad = 0
            for _ in range(500):
                bad += f(*args, handle) != 0
            stream.synchronize()
            if bad:
                failed.append(bad)
                return
    threads = [threading.Thread(target=loop, args=(f, args, torch.cuda.Stream())) for f, args, _, _ in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for (_, _, out, _), w in zip(calls, want):
        assert torch.equal(out, w)
