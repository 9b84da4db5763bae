"""The dense gated block on the GPU against the formulas in 64 bits.

Tolerances.  half(t) = finfo(t).eps / 2 is a rounding's largest relative error
(plus half of the smallest step for fp16).  A product over n terms whose one
factor was rounded adds n independent errors, each at most c_i = half |v_i w_i|:
by Hoeffding's bound their sum passes 8 sqrt(sum c_i^2) with probability below
3e-14.  The tensor cores add 16 products at a time into an fp32 accumulator, an
error of at most 2^-22 of the running sum each, and a running sum of terms of
random sign stays below 8 sqrt(sum of squares)."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def rnd(t, v):
    return torch.finfo(t).eps / 2 * v.abs() + (2.0 ** -25 if t == torch.float16 else 0.0)


def rand(*shape, seed, scale=1.0, dt=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dt)


def up(n):
    return (n + 127) // 128 * 128


def prod(a, b):
    """a b^T in 64 bits, and the accumulator's error."""
    a, b = a.double(), b.double()
    k = a.shape[1]
    return a @ b.t(), 8 * (k / 16 + 1) * 2.0 ** -22 * (a.square() @ b.square().t()).sqrt()


def spread(err, b):
    """Error of err's independent elements through a product with b^T."""
    return 8 * (err.square() @ b.double().square().t()).sqrt()


def unpack64(q, s):
    v = q.view(torch.float8_e4m3fn).double().view(q.shape[0], -1, 128) * s.t().double()[:, :, None]
    return v.view(q.shape[0], -1)


class Case:
    def __init__(self, T, d, I, dt, seed=0):
        self.T, self.d, self.I, self.dt = T, d, I, dt
        self.x = rand(T, d, seed=seed + 1, dt=dt)
        self.w13 = rand(2 * I, d, seed=seed + 2, scale=d ** -0.5, dt=dt)
        self.w2 = rand(d, I, seed=seed + 3, scale=I ** -0.5, dt=dt)
        self.dy = rand(T, d, seed=seed + 4, dt=dt)

    def kept(self, how):
        T, I = self.T, self.I
        if how == "fp8":
            return (torch.full((T, 2 * up(I)), 0xAB, dtype=torch.uint8, device=DEV),
                    torch.full((2 * up(I) // 128, T), -7.0, device=DEV))
        if how == "full":
            return torch.full((T, 2 * I), 7.0, dtype=self.dt, device=DEV), None
        return None, None


# tokens from one to several row tiles; d and inter at, below and beside the
# tiles' 64, 128 and 256
SIZES = [(1, 8, 8), (1, 512, 256), (2, 64, 128), (7, 520, 264), (16, 1024, 384), (17, 200, 136),
         (64, 512, 512), (65, 136, 1000), (100, 1096, 72), (128, 768, 640), (255, 264, 520),
         (256, 512, 256), (257, 512, 256), (300, 1032, 600), (777, 2056, 1000)]


@pytest.mark.parametrize("keep", ["none", "fp8", "full"])
@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("T,d,I", SIZES)
def test_forward(T, d, I, t, keep):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    c = Case(T, d, I, DT[t])
    y_all = torch.full((T + 3, d), 7.0, dtype=c.dt, device=DEV)
    h_all = torch.full((T + 3, I), 7.0, dtype=c.dt, device=DEV)
    y, h = y_all[:T], h_all[:T]
    ac, s = c.kept(keep)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_ffn_forward(c.x, c.w13, c.w2, h, y, ac, s, dev_status=st)
    assert int(st) == 0
    assert (y_all[T:] == 7).all() and (h_all[T:] == 7).all()
    check_forward(c, h, y, ac, s, keep)


def check_forward(c, h, y, ac, s, keep):
    T, I = c.x.shape[0], c.I
    A, ea = prod(c.x, c.w13[:I])
    C, ec = prod(c.x, c.w13[I:])
    H = A * torch.sigmoid(A) * C
    eh = 1.1 * C.abs() * ea + (A * torch.sigmoid(A)).abs() * ec + 1.1 * ea * ec + 2e-6 * H.abs()
    th = eh + rnd(c.dt, H.abs() + eh)
    assert ((h.double() - H).abs() <= th).all()
    Y, ey = prod(H, c.w2)
    ty = spread(th, c.w2) + ey
    ty = ty + rnd(c.dt, Y.abs() + ty)
    assert ((y.double() - Y).abs() <= ty).all()
    if keep == "full":
        ref, e = torch.cat([A, C], 1), torch.cat([ea, ec], 1)
        assert ((ac.double() - ref).abs() <= e + rnd(c.dt, ref.abs() + e)).all()
    if keep == "fp8":
        W = up(I)
        for v, e, at in ((A, ea, 0), (C, ec, W)):
            pad = torch.zeros(T, W, device=DEV, dtype=torch.float64)
            E = pad.clone()
            pad[:, :I], E[:, :I] = v, e
            amax = pad.abs().view(T, -1, 128).amax(2)
            sc = s[at // 128:(at + W) // 128].t().double()
            assert ((sc * 448 - amax).abs() <= E.view(T, -1, 128).amax(2) + 2.0 ** -22 * amax).all()
            got = unpack64(ac[:, at:at + W], s[at // 128:(at + W) // 128])
            sc = sc.repeat_interleave(128, 1)
            assert ((got - pad).abs() <= (2.0 ** -4 + 2.0 ** -20) * (pad.abs() + E) + 2.0 ** -10 * sc
                    + 2 * E)[:, :I].all()
            assert (ac[:, at:at + W].view(torch.uint8)[:, I:] & 0x7F == 0).all()  # padding: zeros


def backward_ref(c, A, C):
    I = c.I
    dh, eh = prod(c.dy, c.w2.t())
    sg = torch.sigmoid(A)
    da, dc, H = dh * C * sg * (1 + A * (1 - sg)), dh * A * sg, A * sg * C
    # five fp32 roundings and the fast exponential's and reciprocal's 2e-6;
    # 1 + a (1 - s) may cancel
    gain = torch.cat([(C * sg).abs() * (1 + A.abs()), (A * sg).abs()], 1)
    eh2 = torch.cat([eh, eh], 1)
    dac = torch.cat([da, dc], 1)
    e = gain * (eh2 + 4e-6 * torch.cat([dh, dh], 1).abs())
    return dac, e + rnd(c.dt, dac.abs() + e), H, rnd(c.dt, H) + 4e-6 * H.abs()


def check_backward(c, A, C, dac, h, dx, dw13, dw2):
    DAC, td, H, th = backward_ref(c, A, C)
    assert ((dac.double() - DAC).abs() <= td).all()
    assert ((h.double() - H).abs() <= th).all()
    for got, (a, ta), b in ((dx, (DAC, td), c.w13.t()), (dw13, (DAC.t(), td.t()), c.x.t())):
        if got is None:
            continue
        ref, e = prod(a, b)
        tol = e + spread(ta, b)
        assert ((got.double() - ref).abs() <= tol + rnd(c.dt, ref.abs() + tol)).all()
    if dw2 is None:
        return
    ref, e = prod(c.dy.t(), H.t())
    tol = e + spread(th.t(), c.dy.t()).t()
    assert ((dw2.double() - ref).abs() <= tol + rnd(c.dt, ref.abs() + tol)).all()


@pytest.mark.parametrize("keep", ["fp8", "full"])
@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("T,d,I", SIZES)
def test_backward(T, d, I, t, keep):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    c = Case(T, d, I, DT[t], seed=50)
    A, C = rand(T, I, seed=61), rand(T, I, seed=62)
    ac, s = c.kept(keep)
    if keep == "fp8":
        W = up(I)
        for v, at in ((A, 0), (C, W)):
            q = torch.empty(T, W, dtype=torch.uint8, device=DEV)
            moe.moe_ckpt_pack(v, q, s[at // 128:(at + W) // 128])
            ac[:, at:at + W] = q
        full = unpack64(ac, s)
        A, C = full[:, :I], full[:, W:W + I]
    else:
        ac[:, :I], ac[:, I:] = A, C
        A, C = ac[:, :I].double(), ac[:, I:].double()
    dac, h = torch.empty(T, 2 * I, dtype=c.dt, device=DEV), torch.empty(T, I, dtype=c.dt, device=DEV)
    dx, dw13, dw2 = torch.empty_like(c.x), torch.empty_like(c.w13), torch.empty_like(c.w2)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_ffn_backward(c.dy, c.x, c.w13, c.w2, ac, s, dac, h, dx, dw13, dw2, dev_status=st)
    assert int(st) == 0
    check_backward(c, A, C, dac, h, dx, dw13, dw2)
    # one gradient at a time gives the same bits
    for k in range(3):
        out = [torch.empty_like(v) if i == k else None for i, v in enumerate((dx, dw13, dw2))]
        moe.moe_ffn_backward(c.dy, c.x, c.w13, c.w2, ac, s, dac, h, *out)
        assert torch.equal(out[k], (dx, dw13, dw2)[k])


# few tokens with a long K: one to eight parts of K, one and two tiles of
# tokens, features that leave the last 64 or more of a tile of 128 empty
FEW = [(1, 6800, 408), (6, 392, 1536), (40, 4096, 136), (48, 1032, 328), (100, 264, 2048), (200, 2048, 192),
       (300, 4104, 136), (500, 2048, 512), (64, 4096, 2048)]


@pytest.mark.parametrize("keep", ["fp8", "full"])
@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("T,d,I", FEW)
def test_few_tokens_kept(T, d, I, t, keep):
    test_forward(T, d, I, t, keep)


@pytest.mark.parametrize("keep", ["fp8", "full"])
@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("T,d,I", FEW)
def test_few_tokens_backward(T, d, I, t, keep):
    test_backward(T, d, I, t, keep)


def test_many_tiles_per_pair():
    """More tiles than CTA pairs, so that pairs walk several, and the widths
    of the full-size layer."""
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    T, d, I = 1100, 7168, 2048
    c = Case(T, d, I, torch.bfloat16, seed=80)
    y, h = torch.empty_like(c.x), torch.empty(T, I, dtype=c.dt, device=DEV)
    ac, s = c.kept("fp8")
    moe.moe_ffn_forward(c.x, c.w13, c.w2, h, y, ac, s)
    dac, dx, dw13, dw2 = (torch.empty(T, 2 * I, dtype=c.dt, device=DEV), torch.empty_like(c.x),
                          torch.empty_like(c.w13), torch.empty_like(c.w2))
    A, ea = prod(c.x, c.w13[:I])
    C, ec = prod(c.x, c.w13[I:])
    H = A * torch.sigmoid(A) * C
    eh = 1.1 * C.abs() * ea + (A * torch.sigmoid(A)).abs() * ec + 1.1 * ea * ec + 2e-6 * H.abs()
    th = eh + rnd(c.dt, H.abs() + eh)
    Y, ey = prod(H, c.w2)
    ty = spread(th, c.w2) + ey
    assert ((y.double() - Y).abs() <= ty + rnd(c.dt, Y.abs() + ty)).all()
    moe.moe_ffn_backward(c.dy, c.x, c.w13, c.w2, ac, s, dac, h, dx, dw13, dw2)
    kept = unpack64(ac, s)
    DAC, td, H, th = backward_ref(c, kept[:, :I], kept[:, I:])
    for got, (a, ta), b in ((dx, (DAC, td), c.w13.t()), (dw13, (DAC.t(), td.t()), c.x.t())):
        ref, e = prod(a, b)
        tol = e + spread(ta, b)
        assert ((got.double() - ref).abs() <= tol + rnd(c.dt, ref.abs() + tol)).all()
    ref, e = prod(c.dy.t(), H.t())
    tol = e + spread(th.t(), c.dy.t()).t()
    assert ((dw2.double() - ref).abs() <= tol + rnd(c.dt, ref.abs() + tol)).all()


def test_gradient_against_differences():
    """The formulas that the gradients are held to, against central
    differences of the block in 64 bits, and the kernel's loss against both."""
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    T, d, I = 3, 16, 24
    c = Case(T, d, I, torch.bfloat16, seed=90)
    x, w13, w2, dy = (v.double() for v in (c.x, c.w13, c.w2, c.dy))

    def loss(x, w13, w2):
        a, b = x @ w13[:I].t(), x @ w13[I:].t()
        return ((a * torch.sigmoid(a) * b) @ w2.t() * dy).sum()
    ac, s = c.kept("full")
    h, y = torch.empty(T, I, dtype=c.dt, device=DEV), torch.empty_like(c.x)
    moe.moe_ffn_forward(c.x, c.w13, c.w2, h, y, ac, s)
    dac, dx, dw13, dw2 = (torch.empty(T, 2 * I, dtype=c.dt, device=DEV), torch.empty_like(c.x),
                          torch.empty_like(c.w13), torch.empty_like(c.w2))
    moe.moe_ffn_backward(c.dy, c.x, c.w13, c.w2, ac, s, dac, h, dx, dw13, dw2)
    step = 1e-5
    for k, got in enumerate((dx, dw13, dw2)):
        args = [x, w13, w2]
        num = torch.empty_like(args[k])
        for i in np.ndindex(*num.shape):
            hi, lo = args[k].clone(), args[k].clone()
            hi[i] += step
            lo[i] -= step
            num[i] = (loss(*[hi if j == k else v for j, v in enumerate(args)])
                      - loss(*[lo if j == k else v for j, v in enumerate(args)])) / (2 * step)
        # kept a and c, [da | dc] or h, and the result are rounded: with the
        # derivative of each at most about 1.1 the kept values' count twice,
        # and the sums' terms add up to more than the sum: the norm of the
        # error is below six halves of a step of the norm
        assert float((got.double() - num).norm() / num.norm()) <= 6 * 2.0 ** -8


def test_no_tokens():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    c = Case(0, 64, 32, torch.bfloat16)
    e = torch.empty(0, 32, dtype=c.dt, device=DEV)
    moe.moe_ffn_forward(c.x, c.w13, c.w2, e, c.x)
    ac, s = c.kept("fp8")
    dw13, dw2 = torch.ones_like(c.w13), torch.ones_like(c.w2)
    moe.moe_ffn_backward(c.x, c.x, c.w13, c.w2, ac, s, torch.empty(0, 64, dtype=c.dt, device=DEV), e,
                         c.x, dw13, dw2)
    assert not dw13.any() and not dw2.any()


@pytest.mark.parametrize("T", [3, 300])
def test_nan_and_infinity_stay_in_their_token(T):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    c = Case(T, 264, 136, torch.bfloat16, seed=5)
    h, y, y2 = torch.empty(T, 136, dtype=c.dt, device=DEV), torch.empty_like(c.x), torch.empty_like(c.x)
    moe.moe_ffn_forward(c.x, c.w13, c.w2, h, y)
    x = c.x.clone()
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    moe.moe_ffn_forward(x, c.w13, c.w2, h, y2)
    keep = [i for i in range(T) if i not in (1, 2)]
    assert y2[1].isnan().all() and not y2[2].isfinite().any()
    assert torch.equal(y[keep], y2[keep])


@pytest.mark.parametrize("T", [1, 40, 500])
def test_side_streams_at_once_and_captured(T):
    """Two calls on two streams at once, each with its own buffers, and a
    captured training step replayed on new inputs."""
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    d, I = 520, 264

    def buffers(seed):
        c = Case(T, d, I, torch.bfloat16, seed=seed)
        ac, s = c.kept("fp8")
        e = lambda *sh: torch.empty(*sh, dtype=c.dt, device=DEV)  # noqa: E731
        return c, ac, s, [e(T, I), e(T, d), e(T, 2 * I), e(T, I), e(T, d), e(2 * I, d), e(d, I)]

    def step(b, stream=None):
        c, ac, s, (h, y, dac, h2, dx, dw13, dw2) = b
        moe.moe_ffn_forward(c.x, c.w13, c.w2, h, y, ac, s, stream=stream)
        moe.moe_ffn_backward(c.dy, c.x, c.w13, c.w2, ac, s, dac, h2, dx, dw13, dw2, stream=stream)
    two = [buffers(100), buffers(200)]
    for b in two:
        step(b)
    torch.cuda.synchronize()
    want = [[v.clone() for v in b[3]] for b in two]
    for b in two:
        for v in b[3]:
            v.zero_()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for b, st in zip(two, side):
            step(b, st)
    torch.cuda.synchronize()
    for b, w in zip(two, want):
        for got, ref in zip(b[3], w):
            assert torch.equal(got, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(two[0])
    two[0][0].x.copy_(two[1][0].x)
    two[0][0].dy.copy_(two[1][0].dy)
    g.replay()
    torch.cuda.synchronize()
    got = [v.clone() for v in two[0][3]]
    step(two[0])
    torch.cuda.synchronize()
    for a, b in zip(got, two[0][3]):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Tokens whose elements lie beyond 2^31, against the formulas."""
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    d, I, dt = 4096, 64, torch.bfloat16
    T = 2 ** 31 // d + 4096
    c = Case(0, d, I, dt)
    c.w13, c.w2 = rand(2 * I, d, seed=2, scale=d ** -0.5, dt=dt), rand(d, I, seed=3, dt=dt)
    x = torch.zeros(T, d, dtype=dt, device=DEV)
    x[-4096:] = rand(4096, d, seed=1, dt=dt)
    e = lambda *s: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    h, y, dac, h2, dx = e(T, I), e(T, d), e(T, 2 * I), e(T, I), e(T, d)
    ac, s = torch.empty(T, 256, dtype=torch.uint8, device=DEV), torch.empty(2, T, device=DEV)
    moe.moe_ffn_forward(x, c.w13, c.w2, h, y, ac, s)
    moe.moe_ffn_backward(x, x, c.w13, c.w2, ac, s, dac, h2, dx)
    n = 600
    c.x = c.dy = x[-n:]
    check_forward(c, h[-n:], y[-n:], ac[-n:], s[:, -n:], "fp8")
    kept = unpack64(ac[-n:], s[:, -n:])
    check_backward(c, kept[:, :I], kept[:, 128:128 + I], dac[-n:], h2[-n:], dx[-n:], None, None)
