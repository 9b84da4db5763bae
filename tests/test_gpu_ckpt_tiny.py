"""Tiles whose largest value is so small that 448 / amax passes the fp32 range
(below about 1.3e-36): what is kept is finite and near what was there, wherever
the checkpoints' scale rule is applied.

The rule takes an amax below 2^-119 as 2^-119: scale 2^-119 / 448 (a subnormal
number, off by at most 2^-150, 2^-22 of itself), inverse 448 2^119, exact.  So a
value is off by half a step of E4M3, 2^-4 of itself or 2^-10 scales, and 2^-21
of itself for scale and product."""
import pytest
import torch

from gpu_util import DEV, need_gpu
from test_gpu_norm_ckpt import DT, U, kept_ac, pack, pack_by_rule, rand, unpack64

pytestmark = pytest.mark.gpu
LEAST = 2.0 ** -119


def near(q, s, x):
    """The kept values against what was kept."""
    got = unpack64(q, s, x.shape[1])
    sc = s.t().repeat_interleave(128, 1)[:, :x.shape[1]].double()
    assert got.isfinite().all()
    v = x.double()
    assert ((got - v).abs() <= v.abs() * (2.0 ** -4 + 2.0 ** -21) + sc * 2.0 ** -10 * (1 + 2.0 ** -20)).all()
    assert (got[v == 0] == 0).all()


@pytest.mark.parametrize("cols", [5, 128, 300])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_pack(cols, t):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    least = 2.0 ** -149 if t == "f32" else 2.0 ** -133  # the type's smallest number
    x = torch.zeros(8, cols, device=DEV)
    x[0, 3] = 1e-37
    x[1, 0], x[1, 1], x[1, 2] = 1.2e-36, -3e-38, 2.0 ** -133
    x[2] = 1e-38 * rand(1, cols, seed=1)
    x[3, 4] = least
    x[4] = -1.0e-36
    x[5, 2] = LEAST
    x[6, 2], x[6, 3] = 2.0 ** -118, 2.0 ** -128
    x = x.to(DT[t])
    q, s = pack(moe, x)
    near(q, s, x)
    pad = (q[:, cols:] & 0x7F)
    assert not pad.any()
    y = torch.empty_like(x)
    moe.moe_ckpt_unpack(q, s, y)
    assert y.isfinite().all() and (y[x == 0] == 0).all()
    # from 2^-119 on, and for zeros, the rule is what it was
    rq, rs = pack_by_rule(x[5:])
    assert torch.equal(q[5:].cpu(), rq) and torch.equal(s[:, 5:].cpu(), rs)


@pytest.mark.parametrize("T,d,I", [(3, 64, 200), (200, 2048, 192), (777, 2056, 1000)])
def test_dense_block_keeps_tiny_gate_and_up(T, d, I):
    """Few tokens and pairs of CTAs: a and c of 2^-122 beside zeros."""
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    dt = torch.bfloat16
    x, w13 = torch.zeros(T, d, dtype=dt, device=DEV), torch.zeros(2 * I, d, dtype=dt, device=DEV)
    x[:, 0] = 2.0 ** -100
    w13[::2, 0] = 2.0 ** -22
    w2 = torch.zeros(d, I, dtype=dt, device=DEV)
    wide = (I + 127) // 128 * 128
    ac = torch.full((T, 2 * wide), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.empty(2 * wide // 128, T, device=DEV)
    h, y = torch.empty(T, I, dtype=dt, device=DEV), torch.empty_like(x)
    moe.moe_ffn_forward(x, w13, w2, h, y, ac, s)
    want = torch.zeros(1, 2 * wide, device=DEV)
    want[:, 0:I:2] = 2.0 ** -122  # (I is even: row I of w13 is an even row)
    want[:, wide:wide + I:2] = 2.0 ** -122
    near(ac, s, want.expand(T, -1))


def test_expert_gemm_keeps_tiny_gate_and_up():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    R, k, n = 40, 128, 256
    one = 0x38  # E4M3 1.0
    a = torch.full((R, k), one, dtype=torch.uint8, device=DEV)
    w = torch.zeros(n, k, dtype=torch.uint8, device=DEV)
    w[::2] = one
    a_s = torch.full((1, R), 2.0 ** -61, device=DEV)
    w_s = torch.full((n // 128, 1), 2.0 ** -68, device=DEV)
    off = torch.tensor([0, R], dtype=torch.int32, device=DEV)
    h, hs = torch.empty(R, n // 2, dtype=torch.uint8, device=DEV), torch.empty(1, R, device=DEV)
    q, qs = torch.empty(R, n, dtype=torch.uint8, device=DEV), torch.empty(n // 128, R, device=DEV)
    moe.moe_grouped_gemm_fp8_ckpt(1, off, R, a, a_s, k, w, w_s, n, h, hs, q, qs)
    want = torch.zeros(R, n, device=DEV)
    want[:, ::2] = 2.0 ** -122
    near(q, qs, want)


def test_swiglu_backward_of_tiny_gradients():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    rows, I = 37, 256
    q0, s0, v = kept_ac(moe, rows, I)
    dh = rand(rows, I, seed=7)
    dh[:, ::3] = 0
    dh[::2] *= 2.0 ** -122  # every other row
    q = torch.empty(rows, 2 * I, dtype=torch.uint8, device=DEV)
    qs = torch.empty(2 * I // 128, rows, device=DEV)
    moe.moe_swiglu_backward_quant_ckpt(dh, q0, s0, rows, I, rows, q, qs)
    a, c, D = v[:, :I].double(), v[:, I:].double(), dh.double()
    sg = torch.sigmoid(a)
    ref = torch.cat([D * c * sg * (1 + a * (1 - sg)), D * a * sg], 1)
    mag = torch.cat([(D * c * sg).abs() * (1 + a.abs()), (D * a * sg).abs()], 1)
    got = unpack64(q, qs, 2 * I)
    sc = qs.t().repeat_interleave(128, 1).double()
    assert got.isfinite().all()
    # exp and reciprocal of a few ulps each, eight products (64 U of the
    # magnitudes they act on), each product below 2^-126 off by half the
    # smallest step
    err = 64 * U * mag + 8 * 2.0 ** -150
    assert ((got - ref).abs() <= 2.0 ** -4 * ref.abs() * (1 + 2.0 ** -20) + sc * 2.0 ** -10 * (1 + 2.0 ** -20)
            + 2 * err).all()
