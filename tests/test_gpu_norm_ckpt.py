"""Layer norm and 8-bit activation checkpoints on the GPU against plain
implementations in 64 bits.

Tolerances: u = 2^-24 is half a step of fp32, half(t) = finfo(t).eps / 2 that
of a stored type.  A sum whose longest chain of additions is D long is off by
at most D u times the sum of its terms' absolute values; the kernels' row sums
have chains of at most 32 (a thread) + 5 + 5 (shuffles) additions, counted as
64 with the few roundings of the terms themselves."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half(t):
    return torch.finfo(t).eps / 2


def rand(*shape, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV)


def tiles(n):
    return (n + 127) // 128


def pack(moe, x):
    q = torch.full((x.shape[0], moe.moe_ckpt_row_bytes(x.shape[1])), 0xAB, dtype=torch.uint8,
                   device=DEV)
    s = torch.full((tiles(x.shape[1]), x.shape[0]), -7.0, device=DEV)
    moe.moe_ckpt_pack(x, q, s)
    return q, s


def unpack64(q, s, cols):
    v = q.view(torch.float8_e4m3fn).double().view(q.shape[0], -1, 128) * s.t().double()[:, :, None]
    return v.view(q.shape[0], -1)[:, :cols]


# ------------------------------------------------------------------ norm
SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (256, 512), (33, 520), (130, 1000), (7, 1477),
          (4, 1032), (200, 7168), (3, 8200), (2, 16384), (2, 16383), (149, 96)]


@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_forward(rows, cols, t):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    dt = DT[t]
    x = (rand(rows, cols, seed=1) * (0.5 + rand(rows, 1, seed=2).abs()) + rand(rows, 1, seed=3)).to(dt)
    w, b = 1 + 0.1 * rand(cols, seed=4), 0.1 * rand(cols, seed=5)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    for wt, bs in ((w, b), (None, None)):
        moe.moe_layernorm_forward(x, wt, bs, 1e-5, y, mean, rstd)
        X = x.double()
        mu = X.mean(1, keepdim=True)
        r = ((X - mu).square().mean(1, keepdim=True) + 1e-5).rsqrt()
        xh = (X - mu) * r
        W = torch.ones(cols, device=DEV).double() if wt is None else wt.double()
        ref = xh * W + (0 if bs is None else bs.double())
        dmu = 64 * U * X.abs().mean(1, keepdim=True)
        tol = W.abs() * (64 * U * xh.abs() + dmu * r) + 2 * U * ref.abs() + U
        tol = tol + half(dt) * (ref.abs() + tol)
        if dt == torch.float16:
            tol = tol + 2.0 ** -25  # half a step below the smallest normal
        # r is off by at most 64 u from its own sum, and by the mean's error,
        # which enters the variance squared
        tol = tol + W.abs() * xh.abs() * (dmu * r) ** 2
        assert ((y.double() - ref).abs() <= tol).all()
        assert ((mean.double() - mu[:, 0]).abs() <= dmu[:, 0]).all()
        assert ((rstd.double() / r[:, 0] - 1).abs() <= 64 * U + (dmu * r)[:, 0] ** 2).all()


def norm_back_ref(dy, X, w, mean, rstd):
    dy, X = dy.double(), X.double()
    r = rstd.double()[:, None]
    xh = (X - mean.double()[:, None]) * r
    g = dy * w.double()
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - m1 - xh * m2)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    dxh = U * (2 * xh.abs() + X.abs() * r)  # of a stored or kept x
    err2 = 64 * U * a2 + (g.abs() * dxh).mean(1, keepdim=True)
    tol = r * (8 * U * g.abs() + 64 * U * a1 + xh.abs() * err2 + m2.abs() * dxh
               + 8 * U * (xh * m2).abs() + 4 * U * m1.abs())
    rows = dy.shape[0]
    depth = -(-rows // 100) + 40  # rows of a CTA, then the CTAs' partial rows
    dw, db = (dy * xh).sum(0), dy.sum(0)
    dwt = depth * U * (dy * xh).abs().sum(0) + (dy.abs() * dxh).sum(0)
    dbt = depth * U * dy.abs().sum(0)
    return dx, tol, dw, dwt, db, dbt


@pytest.mark.parametrize("kept", ["full", "fp8"])
@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_backward(rows, cols, t, kept):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    dt = DT[t]
    x = (rand(rows, cols, seed=1) * 2 + rand(rows, 1, seed=3)).to(dt)
    w = 1 + 0.1 * rand(cols, seed=4)
    dy = rand(rows, cols, seed=6).to(dt)
    mean = x.double().mean(1).float()
    rstd = (x.double().var(1, correction=0) + 1e-5).rsqrt().float()
    xs, X = None, x
    if kept == "fp8":
        x, xs = pack(moe, x)
        X = unpack64(x, xs, cols)
    dx, dw, db = torch.empty_like(dy), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(moe.moe_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8,
                     device=DEV)
    moe.moe_layernorm_backward(dy, x, xs, w, mean, rstd, dx, dw, db, ws)
    rx, tx, rw, tw, rb, tb = norm_back_ref(dy, X, w, mean, rstd)
    tx = tx + half(dt) * (rx.abs() + tx) + (2.0 ** -25 if dt == torch.float16 else 0)
    assert ((dx.double() - rx).abs() <= tx).all()
    assert ((dw.double() - rw).abs() <= tw).all()
    assert ((db.double() - rb).abs() <= tb).all()
    # the same call gives the same bits; without the sums nothing else changes
    dx2, dw2, db2 = (torch.empty_like(v) for v in (dx, dw, db))
    moe.moe_layernorm_backward(dy, x, xs, w, mean, rstd, dx2, dw2, db2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    moe.moe_layernorm_backward(dy, x, xs, w, mean, rstd, dx2, None, None, None)
    assert torch.equal(dx, dx2)


def test_norm_backward_mixed_types_in_place_and_no_rows():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    rows, cols = 37, 512
    dy = rand(rows, cols, seed=6)
    for dt in (torch.bfloat16, torch.float16):
        x = rand(rows, cols, seed=1).to(dt)
        mean = x.double().mean(1).float()
        rstd = (x.double().var(1, correction=0) + 1e-5).rsqrt().float()
        w = 1 + 0.1 * rand(cols, seed=4)
        dx, dw, db = dy.clone(), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        ws = torch.empty(moe.moe_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8,
                         device=DEV)
        moe.moe_layernorm_backward(dx, x, None, w, mean, rstd, dx, dw, db, ws)  # dx is dy
        rx, tx, rw, tw, rb, tb = norm_back_ref(dy, x, w, mean, rstd)
        assert ((dx.double() - rx).abs() <= tx + U * rx.abs()).all()
        assert ((dw.double() - rw).abs() <= tw).all()
        y, y2 = x.clone(), torch.empty_like(x)
        moe.moe_layernorm_forward(x, w, None, 1e-5, y2)
        moe.moe_layernorm_forward(y, w, None, 1e-5, y)
        assert torch.equal(y, y2)
    e = torch.empty(0, cols, device=DEV)
    dw.fill_(3.0)
    db.fill_(3.0)
    z = torch.empty(0, device=DEV)
    moe.moe_layernorm_forward(e, w, None, 1e-5, e, z, z)
    moe.moe_layernorm_backward(e, e, None, w, z, z, e, dw, db, ws)
    assert not dw.any() and not db.any()


def test_norm_gradient_against_differences():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    rows, cols = 2, 24
    x, w, b = rand(rows, cols, seed=1), 1 + 0.1 * rand(cols, seed=2), rand(cols, seed=3)
    dy = rand(rows, cols, seed=4)

    def loss(xx, ww, bb):
        y = torch.empty_like(xx)
        moe.moe_layernorm_forward(xx, ww, bb, 1e-5, y)
        return float((y.double() * dy.double()).sum())
    mean, rstd, y = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty_like(x)
    moe.moe_layernorm_forward(x, w, b, 1e-5, y, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(moe.moe_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
    moe.moe_layernorm_backward(dy, x, None, w, mean, rstd, dx, dw, db, ws)
    # central differences of step h: the loss is a sum of rows * cols values off
    # by about 8 u |y| each, over 2 h; the cubic term of a norm is of order h^2
    h = 2.0 ** -7
    tol = 48 * 8 * U * float(y.abs().max() + 1) * float(dy.abs().max()) / h + 40 * h * h
    for grad, v, at in ((dx, x, (0, 5)), (dx, x, (1, 23)), (dw, w, (7,)), (db, b, (11,))):
        hi, lo = v.clone(), v.clone()
        hi[at] += h
        lo[at] -= h
        args = [(hi if u is v else u, lo if u is v else u) for u in (x, w, b)]
        step = float(hi[at].double() - lo[at].double())
        d = (loss(*[a[0] for a in args]) - loss(*[a[1] for a in args])) / step
        assert abs(d - float(grad[at])) <= tol


def test_norm_nan_stays_in_its_row():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    x = rand(4, 1000, seed=1)
    clean = torch.empty_like(x)
    moe.moe_layernorm_forward(x, None, None, 1e-5, clean)
    x[1, 3], x[3, 0] = float("nan"), float("inf")
    y = torch.empty_like(x)
    moe.moe_layernorm_forward(x, None, None, 1e-5, y)
    assert y[1].isnan().all() and y[3].isnan().all()
    assert torch.equal(y[[0, 2]], clean[[0, 2]])


# ------------------------------------------------------------ checkpoints
def pack_by_rule(x):
    """The checkpoints' scale rule in fp32, on the host."""
    v = x.float().cpu().numpy()
    rows, cols = v.shape
    w = np.zeros((rows, tiles(cols) * 128), np.float32)
    w[:, :cols] = v
    w = w.reshape(rows, -1, 128)
    amax = np.abs(w).max(2)
    one = np.float32(1)
    with np.errstate(divide="ignore"):
        s = np.where(amax == 0, one, amax / np.float32(448))
        inv = np.where(amax == 0, one, (one / amax) * np.float32(448))
    t = torch.from_numpy(w * inv[:, :, None])
    return t.to(torch.float8_e4m3fn).view(torch.uint8).view(rows, -1), torch.from_numpy(s.T.copy())


@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 7), (31, 130), (32, 512), (33, 513),
                                       (777, 1000), (65, 7168), (2, 1029)])
def test_pack_and_unpack(rows, cols, t):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    x = rand(rows, cols, seed=rows + cols) * torch.exp2(6 * rand(rows, 1, seed=9))
    x[:, cols // 2:] *= 0 if rows == 31 else 1  # tiles of zeros
    x = x.to(DT[t])
    q, s = pack(moe, x)
    rq, rs = pack_by_rule(x)
    assert torch.equal(s.cpu(), rs)
    # codes of zero keep their sign: both give it.  fp16 rows may hold an
    # infinity (2^(6 n) above 65504), whose tile is NaN: 0x7f and 0xff are the
    # same value, a NaN's sign says nothing
    nan = rq & 0x7F == 0x7F
    assert torch.equal(q.cpu() & 0x7F == 0x7F, nan)
    assert torch.equal(q.cpu()[~nan], rq[~nan])
    y = torch.empty_like(x)
    moe.moe_ckpt_unpack(q, s, y)
    v = unpack64(q, s, cols).float()  # code times scale, rounded to fp32
    assert torch.equal(y.nan_to_num(1234.0), v.to(DT[t]).nan_to_num(1234.0))
    # what is kept is within half a step of E4M3 (2^-4 of the value; 2^-10
    # scales for a subnormal code), and the two roundings of scale and product
    err = (unpack64(q, s, cols) - x.double()).abs()
    sc = s.t().repeat_interleave(128, 1)[:, :cols].double()
    lost = ~sc.isfinite()  # the tiles with an infinity
    assert y[lost].isnan().all()
    assert (err <= x.double().abs() * (2.0 ** -4 + 4 * U) + sc * 2.0 ** -10)[~lost].all()


def test_pack_unaligned_views_and_specials():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    base = rand(1 + 40 * 256, seed=5)
    x = base[1:].view(40, 256)  # 4-byte aligned only
    q, s = pack(moe, x)
    q2, s2 = pack(moe, x.clone())
    assert torch.equal(q, q2) and torch.equal(s, s2)
    x = rand(3, 256, seed=6)
    x[0, 5], x[1, 130] = float("nan"), float("inf")
    q, s = pack(moe, x)
    y = torch.empty_like(x)
    moe.moe_ckpt_unpack(q, s, y)
    assert y[0, 5].isnan() and y[0].isfinite().sum() == 255  # a NaN leaves its tile alone
    assert y[1, 128:].isnan().all() and y[1, :128].isfinite().all()  # an infinity does not
    assert y[2].isfinite().all()


def test_pack_scale_extremes():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    x = torch.zeros(4, 128, device=DEV)
    x[0] = torch.finfo(torch.float32).max
    x[1] = 1e-30
    x[2, 0], x[2, 1] = 448.0, 2.0 ** -9
    x[3] = -0.0
    q, s = pack(moe, x)
    rq, rs = pack_by_rule(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)


def kept_ac(moe, R, I, seed=0):
    ac = rand(R, 2 * I, seed=seed) * torch.exp2(rand(R, 1, seed=seed + 1))
    q, s = pack(moe, ac)
    v = torch.empty_like(ac)
    moe.moe_ckpt_unpack(q, s, v)
    return q, s, v


@pytest.mark.parametrize("rows,I,total", [(1, 128, 1), (33, 256, 40), (500, 384, 500), (1280, 256, 1280)])
def test_swiglu_backward_from_a_checkpoint(rows, I, total):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    q0, s0, v = kept_ac(moe, total, I)
    v[0, :8] = 0
    dh = rand(rows, I, seed=7)
    q = torch.full((total, 2 * I), 0xAB, dtype=torch.uint8, device=DEV)
    qs = torch.full((2 * I // 128, total), -7.0, device=DEV)
    moe.moe_swiglu_backward_quant_ckpt(dh, q0, s0, rows, I, total, q, qs)
    ac = unpack64(q0, s0, 2 * I)[:rows]
    a, c, D = ac[:, :I], ac[:, I:], dh.double()
    sg = torch.sigmoid(a)
    ref = torch.cat([D * c * sg * (1 + a * (1 - sg)), D * a * sg], 1)
    # the magnitudes the roundings act on: 1 + a (1 - sg) may cancel
    mag = torch.cat([(D * c * sg).abs() * (1 + a.abs()), (D * a * sg).abs()], 1)
    err = 64 * U * mag  # exp and reciprocal of a few ulps each, eight products
    amax = ref.abs().view(rows, -1, 128).amax(2)
    merr = err.view(rows, -1, 128).amax(2)
    assert ((qs[:, :rows].t().double() * 448 - amax).abs() <= merr + 2 * U * amax).all()
    got = unpack64(q[:rows], qs[:, :rows], 2 * I)
    sc = qs[:, :rows].t().repeat_interleave(128, 1).double()
    assert ((got - ref).abs() <= 2.0 ** -4 * ref.abs() * (1 + 8 * U) + 2.0 ** -10 * sc + 2 * err).all()
    # rows behind the last stay as they were
    assert (q[rows:] == 0xAB).all() and (qs[:, rows:] == -7.0).all()


def test_wgrad_quantisers_from_a_checkpoint_equal_those_from_its_values():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    I, sizes = 256, [0, 130, 1, 255, 128]
    off = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device=DEV)
    R, G = sum(sizes), len(sizes)
    q, s, v = kept_ac(moe, R, I, seed=3)
    dh = rand(R, I, seed=9)
    nb = moe.moe_wgrad_max_blocks(R, G)
    kb, blocks = (torch.empty(G + 1, dtype=torch.int32, device=DEV),
                  torch.empty(nb, 2, dtype=torch.int32, device=DEV))
    moe.moe_wgrad_layout(G, off, kb, blocks)

    def out(F):
        return (torch.zeros(F, nb * 128, dtype=torch.uint8, device=DEV),
                torch.zeros(nb, F, device=DEV))
    h0, h1, d0, d1 = out(I), out(I), out(2 * I), out(2 * I)
    moe.moe_wgrad_quant_h(v, I, blocks, *h0)
    moe.moe_wgrad_quant_h_ckpt(q, s, I, blocks, *h1)
    moe.moe_wgrad_quant_dac(dh, v, I, blocks, *d0)
    moe.moe_wgrad_quant_dac_ckpt(dh, q, s, I, blocks, *d1)
    for a, b in zip(h0 + d0, h1 + d1):
        assert torch.equal(a, b)
    assert int(h0[0].ne(0).sum()) > 0


@pytest.mark.parametrize("K", [1, 4, 8, 11, 20])
def test_gate_backward_from_a_checkpoint(K):
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    T, d = 37, 384
    shape = moe.make_shape(T, d, 32, 1, 1, K, 128)
    R = T * K + T
    o = rand(R, d, seed=1)
    q, s = pack(moe, o)
    dy = rand(T, d, seed=2).bfloat16()
    g = torch.Generator().manual_seed(3)
    row = torch.randperm(T * K, generator=g).to(torch.int32).view(T, K).to(DEV)
    row[5, 0] = -1
    score = (0.1 + torch.rand(T, K, generator=g)).to(DEV)
    dg, du = torch.empty(T, K, device=DEV), torch.empty(T, K, device=DEV)
    moe.moe_gate_backward_ckpt(shape, dy, q, s, row, score, dg, du)
    O = unpack64(q, s, d)
    ref = torch.where(row >= 0, torch.einsum("td,tkd->tk", dy.double(), O[row.clamp_min(0).long()]), 0.0)
    sc = score.double()
    S = sc.sum(1, keepdim=True)
    ref_du = (ref - (sc / S * ref).sum(1, keepdim=True)) / S * sc * (1 - sc)
    # 16 exact products are summed in fp32 by pairs and scaled (8 + 1 + 1
    # roundings, each of at most U of the terms' absolute values), those sums
    # in FP64, the result rounded once; du is linear in dg
    terms = torch.where(row >= 0, torch.einsum("td,tkd->tk", dy.double().abs(),
                                               O[row.clamp_min(0).long()].abs()), 0.0)
    err = 10 * U * terms
    err_du = ((err + (sc / S * err).sum(1, keepdim=True)) / S * sc * (1 - sc)).abs()
    assert ((dg.double() - ref).abs() <= err + U * ref.abs() + 1e-12).all()
    assert ((du.double() - ref_du).abs() <= err_du + U * ref_du.abs() + 1e-11).all()


def test_norm_and_checkpoint_on_another_stream_and_in_a_graph():
    """A run of them together: norm, kept input, backward from it; eagerly on a
    side stream, and captured and replayed on new inputs."""
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    rows, cols = 300, 1000
    x, dy = rand(rows, cols, seed=1).bfloat16(), rand(rows, cols, seed=2).bfloat16()
    w = 1 + 0.1 * rand(cols, seed=3)
    f = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    bufs = dict(y=torch.empty_like(x), mean=f(rows), rstd=f(rows), dx=torch.empty_like(x), dw=f(cols),
                db=f(cols), s=f(tiles(cols), rows),
                q=torch.empty(rows, moe.moe_ckpt_row_bytes(cols), dtype=torch.uint8, device=DEV))
    ws = torch.empty(moe.moe_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        b = bufs
        moe.moe_layernorm_forward(x, w, None, 1e-5, b["y"], b["mean"], b["rstd"], stream=stream)
        moe.moe_ckpt_pack(x, b["q"], b["s"], stream=stream)
        moe.moe_layernorm_backward(dy, b["q"], b["s"], w, b["mean"], b["rstd"], b["dx"], b["dw"], b["db"],
                                   ws, stream=stream)
    step()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in bufs.items()}
    side = torch.cuda.Stream()
    for v in bufs.values():
        v.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    for k, v in bufs.items():
        assert torch.equal(v, want[k]), k
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x2 = rand(rows, cols, seed=11).bfloat16()
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in bufs.items()}
    step()
    torch.cuda.synchronize()
    for k, v in bufs.items():
        assert torch.equal(v, got[k]), k


def test_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31 give what the same rows give alone."""
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    cols = 7168
    rows = 2 ** 31 // cols + 700
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x.copy_(rand(1, cols, seed=1).expand(rows, cols))
    x[-600:] = rand(600, cols, seed=2).bfloat16()
    w = 1 + 0.1 * rand(cols, seed=3)

    def step(x):
        n = x.shape[0]
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        moe.moe_layernorm_forward(x, w, None, 1e-5, y, mean, rstd)
        q, s = pack(moe, x)
        back = torch.empty_like(x)
        moe.moe_ckpt_unpack(q, s, back)
        moe.moe_layernorm_backward(y, q, s, w, mean, rstd, dx, None, None, None)
        dx2 = torch.empty_like(x)
        moe.moe_layernorm_backward(y, x, None, w, mean, rstd, dx2, None, None, None)
        return y[-600:], q[-600:], s[:, -600:], back[-600:], mean[-600:], rstd[-600:], dx[-600:], dx2[-600:]
    for a, b in zip(step(x), step(x[-600:].clone())):
        assert torch.equal(a, b)


def test_swiglu_backward_offsets_past_32_bits():
    import fp8_block_scaled_affinity_b200 as moe
    need_gpu()
    inter = 2048
    rows = 2 ** 31 // (2 * inter) + 300
    ac = torch.zeros(rows, 2 * inter, dtype=torch.uint8, device=DEV)
    ac[-200:] = torch.randint(0, 0x7F, (200, 2 * inter), device=DEV).to(torch.uint8)
    s = 0.01 + torch.rand(2 * inter // 128, rows, device=DEV)
    dh = torch.zeros(rows, inter, device=DEV)
    dh[-200:] = rand(200, inter, seed=2)

    def step(dh, ac, s):
        n = dh.shape[0]
        q, qs = torch.empty_like(ac), torch.empty_like(s)
        moe.moe_swiglu_backward_quant_ckpt(dh, ac, s, n, inter, n, q, qs)
        return q[-200:], qs[:, -200:]
    for a, b in zip(step(dh, ac, s), step(dh[-200:].clone(), ac[-200:].clone(), s[:, -200:].contiguous())):
        assert torch.equal(a, b)
