"""test_gpu_failure.py's withheld loads in expert GEMMs with fewer K blocks than
the ring has stages: the producer never waits there, so it is the MMA warp's
wait that runs out, with the later blocks' loads in flight."""
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nkb", [1, 2, 3])
@pytest.mark.parametrize("form", ["f32", "swiglu", "kept"])
def test_wait_runs_out_then_next_call_is_correct(form, nkb, monkeypatch):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    monkeypatch.setenv("MOEFP8_GEMM_PAIR", "0")  # the injection is for single CTAs
    R, k, n = 300, 128 * nkb, 512
    g = torch.Generator(device=DEV)
    g.manual_seed(nkb)
    codes = lambda *s: torch.randint(0, 0x60, s, generator=g, device=DEV).to(torch.uint8)  # noqa: E731
    a, w = codes(R, k), codes(n, k)
    a_s, w_s = torch.full((nkb, R), 2.0 ** -8, device=DEV), torch.full((n // 128, nkb), 2.0 ** -8, device=DEV)
    off = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    h, hs = torch.zeros(R, n // 2, dtype=torch.uint8, device=DEV), torch.zeros(n // 256, R, device=DEV)
    if form == "f32":
        outs = [torch.zeros(R, n, device=DEV)]
        call = lambda: moe.moe_grouped_gemm_fp8(1, off, R, a, a_s, k, w, w_s, n, moe.MOE_EPI_F32,  # noqa: E731
                                                outs[0], None, st)
    elif form == "swiglu":
        outs = [h, hs]
        call = lambda: moe.moe_grouped_gemm_fp8(1, off, R, a, a_s, k, w, w_s, n,  # noqa: E731
                                                moe.MOE_EPI_SWIGLU_QUANT, h, hs, st)
    else:
        outs = [h, hs, torch.zeros(R, n, dtype=torch.uint8, device=DEV), torch.zeros(n // 128, R, device=DEV)]
        call = lambda: moe.moe_grouped_gemm_fp8_ckpt(1, off, R, a, a_s, k, w, w_s, n, *outs, st)  # noqa: E731
    call()
    torch.cuda.synchronize()
    assert int(st) == 0
    good = [v.clone() for v in outs]
    for _ in range(3):
        monkeypatch.setenv("MOEFP8_FAULT", "gemm_producer")
        monkeypatch.setenv("MOEFP8_WAIT_LIMIT_NS", "20000")
        call()
        torch.cuda.synchronize()  # returns: the kernel ended by itself
        assert int(st) == moe.MOE_DEV_TIMEOUT
        monkeypatch.delenv("MOEFP8_FAULT")
        monkeypatch.delenv("MOEFP8_WAIT_LIMIT_NS")
        st.zero_()
        for v in outs:
            v.zero_()
        call()
        torch.cuda.synchronize()
        assert int(st) == 0
        for v, u in zip(outs, good):
            assert torch.equal(v, u)
