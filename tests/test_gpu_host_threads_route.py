"""test_gpu_host_threads.py's threads with the router's kernels: two shapes whose
rows and logits take different amounts of shared memory above 48 KB."""
import ctypes
import threading

import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


def route_call(moe, T, d, N, K=8):
    shape = moe.make_shape(T, d, N, 8, 4, K, 128)
    x, e = torch.randn(T, d, device=DEV).bfloat16(), (torch.randn(N, d, device=DEV) * 0.01).bfloat16()
    bias = torch.zeros(N, device=DEV)
    idx = torch.empty(T, K, dtype=torch.int32, device=DEV)
    gate, counts = torch.empty(T, K, device=DEV), torch.empty(N, dtype=torch.int32, device=DEV)
    ws = torch.empty(moe.moe_route_workspace_size(shape), dtype=torch.uint8, device=DEV)
    args = (ctypes.byref(shape), x.data_ptr(), e.data_ptr(), bias.data_ptr(), None, idx.data_ptr(),
            gate.data_ptr(), counts.data_ptr(), ws.data_ptr(), ws.numel(), None)
    return moe.lib().moe_route, args, (idx, gate, counts), (shape, x, e, bias, ws)


def test_threads_with_two_shapes():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    calls = [route_call(moe, 8, d, N) for d, N in ((12288, 1024), (6272, 768)) * 2]
    want = []
    for f, args, outs, _ in calls:
        assert f(*args, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        want.append([v.clone() for v in outs])
    failed = []

    def loop(f, args, stream):
        torch.cuda.set_device(0)
        handle = stream.cuda_stream
        for _ in range(10):
            bad = 0
            for _ in range(100):
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
    for (_, _, outs, _), ws in zip(calls, want):
        for v, w in zip(outs, ws):
            assert torch.equal(v, w)
