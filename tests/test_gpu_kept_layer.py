"""The layers with their norm and with 8-bit checkpoints: MoeLayer and GatedFfn
built from the layer norm, the kept values and the backward steps that read
them, and a run of all of them together."""
import numpy as np
import pytest
import torch

import synthetic as S
from gpu_util import DEV, bf16_dev, expert_bf16, need_gpu, shape_of, to_dev

pytestmark = pytest.mark.gpu


def _moe():
    import fp8_block_scaled_affinity_b200 as moe
    return moe


def rand(*shape, seed, scale=1.0, dt=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dt)


def moe_layer(T, norm=None):
    moe, cfg = _moe(), S.CONFIGS["tiny"]
    inp = S.make_layer_inputs_host(cfg)
    layer = moe.MoeLayer(shape_of(cfg, T), bf16_dev(inp["router_w"]), to_dev(inp["bias"]), device=DEV,
                         norm=norm)
    for e in range(cfg.n_routed + 1):
        layer.set_expert(e, *expert_bf16(cfg, e))
    return layer, cfg


def unpack(moe, q, s, cols):
    y = torch.empty(q.shape[0], cols, device=DEV)
    moe.moe_ckpt_unpack(q, s, y)
    return y


@pytest.mark.parametrize("sizes", [[128, 7, 0, 300], [1], [256, 129]])
def test_gemm_that_keeps_gate_and_up(sizes):
    """The plain call's bits, and codes of the fp32 epilogue's values; rows
    outside every group stay as they were."""
    moe = _moe()
    need_gpu()
    rng = np.random.default_rng(3)
    k, n, G = 512, 768, len(sizes)
    off = to_dev(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32))
    R = sum(sizes) + 5
    aq, a_s = (torch.empty(R, k, dtype=torch.uint8, device=DEV), torch.empty(k // 128, R, device=DEV))
    moe.fp8_quant_act_1x128(rand(R, k, seed=1), aq, a_s, True)
    wq = torch.empty(G * n, k, dtype=torch.uint8, device=DEV)
    w_s = torch.empty(G * n // 128, k // 128, device=DEV)
    moe.fp8_quant_w_128x128(bf16_dev(S.host_normal_bf16(rng, (G * n, k), 0.1)), wq, w_s)
    h0, h1 = (torch.full((R, n // 2), 0xAB, dtype=torch.uint8, device=DEV) for _ in range(2))
    s0, s1 = (torch.full((n // 256, R), -7.0, device=DEV) for _ in range(2))
    ac = torch.zeros(R, n, device=DEV)
    q = torch.full((R, n), 0xAB, dtype=torch.uint8, device=DEV)
    qs = torch.full((n // 128, R), -7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    a = (G, off, R, aq, a_s, k, wq, w_s, n)
    moe.moe_grouped_gemm_fp8(*a, moe.MOE_EPI_SWIGLU_QUANT, h0, s0, st)
    moe.moe_grouped_gemm_fp8(*a, moe.MOE_EPI_F32, ac, None, st)
    moe.moe_grouped_gemm_fp8_ckpt(*a, h1, s1, q, qs, st)
    assert int(st) == 0
    assert torch.equal(h0, h1) and torch.equal(s0, s1)
    n_rows = sum(sizes)
    assert (q[n_rows:] == 0xAB).all() and (qs[:, n_rows:] == -7.0).all()
    # the same accumulator: the same codes as packing its values
    rq, rs = torch.empty_like(q), torch.empty_like(qs)
    moe.moe_ckpt_pack(ac, rq, rs)
    assert torch.equal(q[:n_rows], rq[:n_rows]) and torch.equal(qs[:, :n_rows], rs[:, :n_rows])


@pytest.mark.parametrize("T", [256, 37, 1])
def test_moe_layer_that_keeps_8_bits(T, monkeypatch):
    """y is forward()'s; the gradients are those of the kept values: weight
    gradients the same bits as from the unpacked fp32 values, the others to
    what two forms of the same fp32 arithmetic differ by before a rounding to
    E4M3 (a code apart in few places) or to fp32."""
    moe = _moe()
    need_gpu()
    layer, cfg = moe_layer(T)
    x, dy = rand(T, cfg.d, seed=5), rand(T, cfg.d, seed=6)
    y = layer.forward(x)
    assert torch.equal(layer.forward_train(x, keep="fp8").view(torch.int16), y.view(torch.int16))
    assert layer.status() == 0
    dx, dE, dW13, dW2 = layer.backward(dy, wgrad=True)
    dg, du = layer.last_dgate.clone(), layer.last_du.clone()
    I, d = cfg.inter, cfg.d

    def swiglu(dh, q, s, rows, inter, total, o, os_, st, stream):
        moe.moe_swiglu_backward_quant(dh, unpack(moe, q, s, 2 * I), rows, inter, total, o, os_, st, stream)

    def dac(dh, q, s, inter, blocks, o, os_, st, stream):
        moe.moe_wgrad_quant_dac(dh, unpack(moe, q, s, 2 * I), inter, blocks, o, os_, st, stream)

    def h(q, s, inter, blocks, o, os_, st, stream):
        moe.moe_wgrad_quant_h(unpack(moe, q, s, 2 * I), inter, blocks, o, os_, st, stream)

    def gate(sh, dy, q, s, row, score, dg, du, st, stream):
        moe.moe_gate_backward(sh, dy, unpack(moe, q, s, d), row, score, dg, du, st, stream)
    monkeypatch.setattr(moe, "moe_swiglu_backward_quant_ckpt", swiglu)
    monkeypatch.setattr(moe, "moe_wgrad_quant_dac_ckpt", dac)
    monkeypatch.setattr(moe, "moe_wgrad_quant_h_ckpt", h)
    monkeypatch.setattr(moe, "moe_gate_backward_ckpt", gate)
    rx, rE, r13, r2 = layer.backward(dy, wgrad=True)
    assert torch.equal(dW13, r13) and torch.equal(dW2, r2)
    # the unpacked outputs are rounded to fp32 once: 2^-24 of each product
    scale = float(dg.abs().max())
    assert ((dg - layer.last_dgate).abs() <= 2.0 ** -23 * d ** 0.5 * scale + 2.0 ** -22 * dg.abs()).all()
    # a code of E4M3 apart (2^-3) in at most 2e-4 of the entries is 2e-3 of the norm
    assert float((dx - rx).norm() / rx.norm()) <= 2e-3
    assert float((du - layer.last_du).norm()) <= 1e-5 * float(du.norm() + 1e-30)
    assert float((dE - rE).norm()) <= 1e-5 * float(rE.norm())


def test_moe_layer_kept_and_recomputed_gradients_agree():
    """Against the layer that keeps fp32 and recomputes, and back to it on the
    same layer.  A kept value is off by at most 2^-4 of itself, uniformly, so
    by 2^-4 / sqrt(3) of the norm; each gradient has two such factors (a and c,
    or o alone)."""
    moe = _moe()
    need_gpu()
    layer, cfg = moe_layer(200)
    x, dy = rand(200, cfg.d, seed=5), rand(200, cfg.d, seed=6)

    def grads(keep):
        layer.forward_train(x, keep=keep)
        return [v.clone() for v in layer.backward(dy, wgrad=True)]
    full, kept, again = grads(None), grads("fp8"), grads(None)
    for a, b in zip(full, again):
        assert torch.equal(a, b)
    for a, b in zip(full, kept):
        assert 0 < float((a - b).norm() / a.norm()) <= 2 * 2.0 ** -4 / 3 ** 0.5


@pytest.mark.parametrize("keep", [None, "fp8"])
def test_moe_layer_with_a_norm_is_the_two_in_turn(keep):
    moe = _moe()
    need_gpu()
    d = S.CONFIGS["tiny"].d
    w, b = 1 + rand(d, seed=7, scale=0.1, dt=torch.float32), rand(d, seed=8, scale=0.1, dt=torch.float32)
    layer, cfg = moe_layer(100, norm=moe.LayerNorm(w, b))
    plain, _ = moe_layer(100)
    norm = moe.LayerNorm(w, b)
    x, dy = rand(100, d, seed=5, scale=3.0), rand(100, d, seed=6)
    y = layer.forward_train(x, keep=keep)
    n = norm.forward_train(x, keep=keep or "full")
    assert torch.equal(y, plain.forward_train(n, keep=keep)) and torch.equal(y, layer.forward(x))
    got, ref = layer.backward(dy, wgrad=True), plain.backward(dy, wgrad=True)
    for u, v in zip(got[1:], ref[1:]):
        assert torch.equal(u, v)
    assert torch.equal(got[0], norm.backward(ref[0]))
    assert torch.equal(layer.norm.dweight, norm.dweight) and torch.equal(layer.norm.dbias, norm.dbias)


@pytest.mark.parametrize("keep", ["fp8", "full"])
@pytest.mark.parametrize("T", [1, 70, 300])
def test_gated_ffn_is_its_calls_in_turn(T, keep):
    moe = _moe()
    need_gpu()
    d, I = 520, 264
    w13, w2 = rand(2 * I, d, seed=1, scale=d ** -0.5), rand(d, I, seed=2, scale=I ** -0.5)
    w = 1 + rand(d, seed=3, scale=0.1, dt=torch.float32)
    ffn = moe.GatedFfn(w13, w2, norm=moe.LayerNorm(w))
    x, dy = rand(T, d, seed=4, scale=2.0), rand(T, d, seed=5)
    norm = moe.LayerNorm(w)
    n = norm.forward_train(x, keep=keep)
    h, y, y2 = torch.empty(T, I, dtype=x.dtype, device=DEV), torch.empty_like(x), torch.empty_like(x)
    ac, s = ((torch.empty(T, 2 * 384, dtype=torch.uint8, device=DEV), torch.empty(6, T, device=DEV))
             if keep == "fp8" else (torch.empty(T, 2 * I, dtype=x.dtype, device=DEV), None))
    moe.moe_ffn_forward(n, w13, w2, h, y2)
    moe.moe_ffn_forward(n, w13, w2, h, y, ac, s)
    assert torch.equal(ffn.forward(x), y2) and torch.equal(ffn.forward_train(x, keep=keep), y)
    dac = torch.empty(T, 2 * I, dtype=x.dtype, device=DEV)
    dx, dw13, dw2 = torch.empty_like(x), torch.empty_like(w13), torch.empty_like(w2)
    moe.moe_ffn_backward(dy, n, w13, w2, ac, s, dac, h, dx, dw13, dw2)
    got = ffn.backward(dy)
    assert torch.equal(got[1], dw13) and torch.equal(got[2], dw2)
    assert torch.equal(got[0], norm.backward(dx)) and torch.equal(ffn.norm.dweight, norm.dweight)
    assert torch.equal(ffn.backward(dy, wgrad=False), got[0])
    assert ffn.status() == 0


def test_a_dense_and_an_expert_layer_together_eager_and_captured():
    """x + GatedFfn(norm(x)), then + MoeLayer(norm(.)), kept in 8 bits, and
    both backward passes: eagerly on a side stream and replayed from a graph on
    new inputs, the same bits each way."""
    moe = _moe()
    need_gpu()
    d, T = S.CONFIGS["tiny"].d, 130
    ln = lambda seed: moe.LayerNorm(1 + rand(d, seed=seed, scale=0.1, dt=torch.float32))  # noqa: E731
    ffn = moe.GatedFfn(rand(512, d, seed=1, scale=d ** -0.5), rand(d, 256, seed=2, scale=0.06), ln(3))
    layer, _ = moe_layer(T, norm=ln(4))
    x, dy = rand(T, d, seed=5), rand(T, d, seed=6)

    def step():
        a = x + ffn.forward_train(x)
        y = a + layer.forward_train(a, keep="fp8")
        da, dE, dW13, dW2 = layer.backward(dy, wgrad=True)
        da = (da + dy.float()).bfloat16()
        dx, dw13, dw2 = ffn.backward(da)
        return [y, dx + da, dE, dW13, dW2, dw13, dw2, ffn.norm.dweight, layer.norm.dweight]
    want = [v.clone() for v in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b) and b.isfinite().all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    x.copy_(rand(T, d, seed=15))
    dy.copy_(rand(T, d, seed=16))
    g.replay()
    torch.cuda.synchronize()
    replayed = [v.clone() for v in out]
    for a, b in zip(replayed, step()):
        assert torch.equal(a, b)
    assert layer.status() == 0 and ffn.status() == 0


def test_empty_batches():
    moe = _moe()
    need_gpu()
    layer, cfg = moe_layer(0, norm=moe.LayerNorm())
    x = rand(0, cfg.d, seed=1)
    layer.forward_train(x, keep="fp8")
    dx, dE, dW13, dW2 = layer.backward(x, wgrad=True)
    assert dx.shape == (0, cfg.d) and not dE.any() and not dW13.any() and not dW2.any()
    ffn = moe.GatedFfn(rand(64, 32, seed=2), rand(32, 32, seed=3), moe.LayerNorm())
    e = rand(0, 32, seed=4)
    ffn.forward_train(e)
    dx, dw13, dw2 = ffn.backward(e)
    assert dx.shape == (0, 32) and not dw13.any() and not dw2.any() and not ffn.norm.dbias.any()


def test_refusals():
    moe = _moe()
    need_gpu()
    w13, w2 = rand(64, 32, seed=2), rand(32, 32, seed=3)
    ffn = moe.GatedFfn(w13, w2)
    with pytest.raises(RuntimeError, match="forward_train"):
        ffn.backward(rand(4, 32, seed=1))
    with pytest.raises(RuntimeError, match="forward_train"):
        moe.LayerNorm().backward(rand(4, 32, seed=1))
    with pytest.raises(ValueError, match="keep"):
        ffn.forward_train(rand(4, 32, seed=1), keep="int8")
    with pytest.raises(ValueError, match="w13 must be"):
        moe.GatedFfn(w13, rand(32, 40, seed=3))
    for bad, match in ((rand(4, 40, seed=1), "shape"), (rand(4, 32, seed=1, dt=torch.float16), "dtype"),
                       (rand(32, 4, seed=1).t(), "contiguous"), (rand(4, 32, seed=1).cpu(), "CUDA device")):
        with pytest.raises(ValueError, match=match):
            ffn.forward(bad, y=torch.empty(4, 32, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(moe.MoeError):
        moe.moe_ffn_forward(rand(2, 12, seed=1), rand(16, 12, seed=2), rand(12, 8, seed=3), rand(2, 8, seed=4),
                            rand(2, 12, seed=5))
    layer, cfg = moe_layer(4)
    with pytest.raises(ValueError, match="keep"):
        layer.forward_train(rand(4, cfg.d, seed=1), keep="full")
    with pytest.raises(ValueError, match="norm"):
        moe.MoeLayer(shape_of(cfg, 4), layer.router_w, layer.bias, device=DEV, host_io=True,
                     norm=moe.LayerNorm())


@pytest.mark.parametrize("which", ["dense", "experts"])
def test_buffers_of_a_call_belong_to_its_stream(which):
    """stream= names a stream that is still busy when the call returns: memory
    that the current stream takes meanwhile is none of the call's."""
    moe = _moe()
    need_gpu()
    T, d = 300, S.CONFIGS["tiny"].d
    norm = moe.LayerNorm(1 + rand(d, seed=3, scale=0.1, dt=torch.float32))
    if which == "dense":
        run = moe.GatedFfn(rand(512, d, seed=1, scale=d ** -0.5), rand(d, 256, seed=2, scale=0.06), norm)
    else:
        run, _ = moe_layer(T, norm=norm)
    x, dy = rand(T, d, seed=5), rand(T, d, seed=6)

    def step(stream=None):
        y = run.forward_train(x, keep="fp8", stream=stream)
        return [y, *run.backward(dy, wgrad=True, stream=stream), norm.dweight, norm.dbias]
    want = [v.clone() for v in step()]
    side = torch.cuda.Stream()
    step(side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = step(side)
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
            for n in [1 << k for k in range(9, 24)] * 8]
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    del junk


def test_in_place_outputs():
    """y may be x where x itself is not kept, and is refused where it is."""
    moe = _moe()
    need_gpu()
    T, d = 70, 256
    x, dy = rand(T, d, seed=1), rand(T, d, seed=2)
    ln = moe.LayerNorm(1 + rand(d, seed=3, scale=0.1, dt=torch.float32))
    ffn = moe.GatedFfn(rand(512, d, seed=4, scale=d ** -0.5), rand(d, 256, seed=5, scale=0.06), ln)
    for run in (ln, ffn):
        want = [run.forward_train(x, keep="fp8")]
        want += [v.clone() for v in torch.utils._pytree.tree_leaves(run.backward(dy))]
        z = x.clone()
        got = [run.forward_train(z, y=z, keep="fp8")]
        got += torch.utils._pytree.tree_leaves(run.backward(dy))
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        with pytest.raises(ValueError, match="kept for backward"):
            run.forward_train(z, y=z, keep="full")
    with pytest.raises(ValueError, match="kept for backward"):
        moe.GatedFfn(ffn.w13, ffn.w2).forward_train(z, y=z, keep="fp8")
    q, s = torch.zeros(4, 256, dtype=torch.int8, device=DEV), torch.zeros(2, 4, device=DEV)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_swiglu_backward_quant_ckpt(torch.zeros(4, 128, device=DEV), q, s, 4, 128, 4, q.view(torch.uint8), s)
