"""What is measured of the layer norm, the 8-bit activation checkpoints and the
dense gated feed-forward block: the cases, their inputs, the plain forms of the
operators in elementary torch operations, and the calls of the framework.

A checkpoint holds a matrix in E4M3 codes, one fp32 scale for each 1x128 tile
of a row: scale = amax / 448, code = E4M3(v * (448 / amax)), scale 1 for a tile
of zeros.  Codes lie in [rows, cols rounded up to 128] bytes, scales in
[tiles, rows].
"""
import math

import torch

own = False  # False: the plain forms; True: the framework's kernels

DEV = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
TILE = 128
E4M3_MAX = 448.0


def up(n, m):
    return (n + m - 1) // m * m


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the normalisation in front of a small layer: latency counts
        {"name": "norm_forward_tiny", "op": "norm_forward", "rows": 256, "cols": 512, "type": "bf16"},
        # the largest batch of hidden states
        {"name": "norm_forward_large", "op": "norm_forward", "rows": 16384, "cols": 7168, "type": "bf16"},
        # rows that start at no multiple of 16 bytes
        {"name": "norm_backward_odd", "op": "norm_backward", "rows": 1001, "cols": 1477, "type": "fp32",
         "kept": "full"},
        # a training step's norm with its input kept in 8 bits
        {"name": "norm_backward_kept", "op": "norm_backward", "rows": 4096, "cols": 7168, "type": "bf16",
         "kept": "fp8"},
        # keeping a small ragged activation and taking it back
        {"name": "keep_ragged", "op": "keep", "rows": 777, "cols": 1000, "type": "bf16"},
        # the expert outputs of 4096 tokens with 8 + 1 experts each, kept for the gates' gradient
        {"name": "keep_expert_out", "op": "keep", "rows": 36864, "cols": 7168, "type": "fp32"},
        # the experts' activation gradient from kept gate and up values: a small layer's rows
        {"name": "swiglu_backward_tiny", "op": "swiglu_backward", "rows": 1280, "inter": 256},
        # the same for 4096 tokens with 8 + 1 experts each
        {"name": "swiglu_backward_large", "op": "swiglu_backward", "rows": 36864, "inter": 2048},
        # one token through a dense block: the weights' bytes
        {"name": "ffn_forward_token", "op": "ffn_forward", "rows": 1, "d": 7168, "inter": 2048, "type": "bf16"},
        # a ragged batch in fp16
        {"name": "ffn_forward_odd", "op": "ffn_forward", "rows": 777, "d": 2056, "inter": 1000, "type": "fp16"},
        # a small training step: forward that keeps gate and up in 8 bits, then the backward pass
        {"name": "ffn_train_tiny", "op": "ffn_train", "rows": 256, "d": 512, "inter": 256, "type": "bf16"},
        # a training step of 4096 tokens
        {"name": "ffn_train_large", "op": "ffn_train", "rows": 4096, "d": 7168, "inter": 2048, "type": "bf16"},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "keep", "swiglu_backward", "ffn_forward",
                     "ffn_train"])
    if op in ("norm_forward", "norm_backward", "keep"):
        c = {"op": op, "rows": _log(rng, 1, 16384), "cols": _log(rng, 64, 7168),
             "type": rng.choice(["bf16", "fp16", "fp32"])}
        if op == "norm_backward":
            c["kept"] = rng.choice(["full", "fp8"])
        return c
    if op == "swiglu_backward":
        return {"op": op, "rows": _log(rng, 1, 36864), "inter": 128 * rng.randint(1, 16)}
    c = {"op": op, "rows": _log(rng, 1, 4096), "d": 8 * _log(rng, 16, 896),
         "inter": 8 * _log(rng, 8, 256), "type": "bf16"}
    if op == "ffn_forward":
        c["type"] = rng.choice(["bf16", "fp16"])
    return c


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    op, rows = case["op"], case["rows"]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    def kept(v):
        q, s = _pack(v.float())
        return _codes_out(q, v.shape[1]), s

    s = {"case": dict(case)}
    if op in ("norm_forward", "norm_backward"):
        t, cols = TYPES[case["type"]], case["cols"]
        # hidden states: every row has its own scale and offset
        x = (torch.randn(rows, cols, generator=g, device=DEV)
             * (0.5 + torch.rand(rows, 1, generator=g, device=DEV))
             + torch.randn(rows, 1, generator=g, device=DEV)).to(t)
        s["weight"] = 1.0 + normal(cols, scale=0.1)
        if op == "norm_forward":
            s["x"], s["bias"] = x, normal(cols, scale=0.1)
            s["y"] = torch.empty_like(x)
            s["mean"] = torch.empty(rows, device=DEV)
            s["rstd"] = torch.empty(rows, device=DEV)
            return s
        x64 = x.double()
        mean = x64.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = ((x64 - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        s["dy"] = normal(rows, cols, dtype=t)
        s["dx"] = torch.empty_like(s["dy"])
        s["dweight"], s["dbias"] = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        s["x"], s["x_scales"] = kept(x) if case["kept"] == "fp8" else (x, None)
        return s
    if op == "keep":
        t, cols = TYPES[case["type"]], case["cols"]
        # activations: a few columns are ten times as large as the others
        scale = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.01, 10.0, 1.0)
        s["x"] = (torch.randn(rows, cols, generator=g, device=DEV) * scale).to(t)
        s["q"] = torch.empty(rows, up(cols, TILE), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(up(cols, TILE) // TILE, rows, device=DEV)
        s["back"] = torch.empty_like(s["x"])
        return s
    if op == "swiglu_backward":
        inter = case["inter"]
        s["ac"], s["ac_scales"] = kept(normal(rows, 2 * inter))
        s["dh"] = normal(rows, inter, scale=0.5)
        s["q"] = torch.empty(rows, 2 * inter, dtype=torch.uint8, device=DEV)
        s["q_scales"] = torch.empty(2 * inter // TILE, rows, device=DEV)
        return s
    t, d, inter = TYPES[case["type"]], case["d"], case["inter"]
    # weights scaled so that gate and up values are of order one
    s["x"] = normal(rows, d, dtype=t)
    s["w13"] = normal(2 * inter, d, scale=1.0 / math.sqrt(d), dtype=t)
    s["w2"] = normal(d, inter, scale=1.0 / math.sqrt(inter), dtype=t)
    s["h"] = torch.empty(rows, inter, dtype=t, device=DEV)
    s["y"] = torch.empty(rows, d, dtype=t, device=DEV)
    if op == "ffn_train":
        wide = up(inter, TILE)
        s["dy"] = normal(rows, d, dtype=t)
        s["ac"] = torch.empty(rows, 2 * wide, dtype=torch.uint8, device=DEV)
        s["ac_scales"] = torch.empty(2 * wide // TILE, rows, device=DEV)
        s["dac"] = torch.empty(rows, 2 * inter, dtype=t, device=DEV)
        s["dx"], s["dw13"], s["dw2"] = (torch.empty_like(s[k]) for k in ("x", "w13", "w2"))
    return s


# ------------------------------------------------------------ plain forms
def _pack(v):
    """fp32 [rows, cols] -> E4M3 [rows, tiles, 128] (zeros past the last column), scales [tiles, rows]."""
    rows, cols = v.shape
    t = torch.zeros(rows, up(cols, TILE), device=v.device)
    t[:, :cols] = v
    t = t.view(rows, -1, TILE)
    amax = t.abs().amax(2)
    none = amax == 0
    scale = torch.where(none, torch.ones_like(amax), amax / E4M3_MAX)
    inverse = torch.where(none, torch.ones_like(amax), E4M3_MAX / amax)
    return (t * inverse[:, :, None]).to(torch.float8_e4m3fn), scale.t().contiguous()


def _codes_out(q, cols):
    return q.view(q.shape[0], -1).view(torch.uint8)


def _unpack(codes, scales, cols):
    q = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, TILE)
    return (q * scales.t()[:, :, None]).view(codes.shape[0], -1)[:, :cols]


def _value(codes, cols):
    """Codes as the E4M3 numbers they stand for."""
    return codes.view(torch.float8_e4m3fn)[:, :cols]


def _gated(a, c):
    return a / (1.0 + torch.exp(-a)) * c


def _gated_backward(dh, a, c):
    sig = 1.0 / (1.0 + torch.exp(-a))
    return dh * c * sig * (1.0 + a * (1.0 - sig)), dh * a * sig


def _plain(s):
    op = s["case"]["op"]
    if op == "norm_forward":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = 1.0 / torch.sqrt(xc.square().mean(1, keepdim=True) + EPS)
        y = xc * rstd * s["weight"] + s["bias"]
        return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "norm_backward":
        cols = s["weight"].numel()
        x = s["x"].float() if s["x_scales"] is None else _unpack(s["x"], s["x_scales"], cols)
        dy = s["dy"].float()
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        gr = dy * s["weight"]
        dx = s["rstd"][:, None] * (gr - gr.mean(1, keepdim=True) - xh * (gr * xh).mean(1, keepdim=True))
        return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
    if op == "keep":
        cols = s["x"].shape[1]
        q, scales = _pack(s["x"].float())
        codes = _codes_out(q, cols)
        return {"codes": _value(codes, cols), "scales": scales,
                "back": _unpack(codes, scales, cols).to(s["x"].dtype)}
    if op == "swiglu_backward":
        inter = s["dh"].shape[1]
        ac = _unpack(s["ac"], s["ac_scales"], 2 * inter)
        da, dc = _gated_backward(s["dh"], ac[:, :inter], ac[:, inter:])
        q, scales = _pack(torch.cat([da, dc], 1))
        return {"codes": _value(_codes_out(q, 2 * inter), 2 * inter), "scales": scales}
    t, inter = s["x"].dtype, s["w2"].shape[1]
    x, w13, w2 = s["x"].float(), s["w13"].float(), s["w2"].float()
    ac = x @ w13.t()
    a, c = ac[:, :inter], ac[:, inter:]
    h = _gated(a, c)
    y = (h @ w2.t()).to(t)
    if op == "ffn_forward":
        return {"y": y}
    qa, sa = _pack(a)
    qc, sc = _pack(c)
    dy = s["dy"].float()
    ka = _unpack(_codes_out(qa, inter), sa, inter)
    kc = _unpack(_codes_out(qc, inter), sc, inter)
    da, dc = _gated_backward(dy @ w2, ka, kc)
    dac = torch.cat([da, dc], 1)
    return {"y": y, "dx": (dac @ w13).to(t), "dw13": (dac.t() @ x).to(t),
            "dw2": (dy.t() @ _gated(ka, kc)).to(t)}


# ------------------------------------------------------ framework's calls
def _framework(s):
    import fp8_block_scaled_affinity_b200 as moe
    op = s["case"]["op"]
    if op == "norm_forward":
        moe.moe_layernorm_forward(s["x"], s["weight"], s["bias"], EPS, s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_backward":
        rows, cols = s["dy"].shape
        ws = torch.empty(moe.moe_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8,
                         device=DEV)
        moe.moe_layernorm_backward(s["dy"], s["x"], s["x_scales"], s["weight"], s["mean"], s["rstd"],
                                   s["dx"], s["dweight"], s["dbias"], ws)
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if op == "keep":
        moe.moe_ckpt_pack(s["x"], s["q"], s["scales"])
        moe.moe_ckpt_unpack(s["q"], s["scales"], s["back"])
        return {"codes": _value(s["q"], s["x"].shape[1]), "scales": s["scales"], "back": s["back"]}
    if op == "swiglu_backward":
        rows, inter = s["dh"].shape
        moe.moe_swiglu_backward_quant_ckpt(s["dh"], s["ac"], s["ac_scales"], rows, inter, rows, s["q"],
                                           s["q_scales"])
        return {"codes": _value(s["q"], 2 * inter), "scales": s["q_scales"]}
    if op == "ffn_forward":
        moe.moe_ffn_forward(s["x"], s["w13"], s["w2"], s["h"], s["y"])
        return {"y": s["y"]}
    moe.moe_ffn_forward(s["x"], s["w13"], s["w2"], s["h"], s["y"], s["ac"], s["ac_scales"])
    moe.moe_ffn_backward(s["dy"], s["x"], s["w13"], s["w2"], s["ac"], s["ac_scales"], s["dac"], s["h"],
                         s["dx"], s["dw13"], s["dw2"])
    return {"y": s["y"], "dx": s["dx"], "dw13": s["dw13"], "dw2": s["dw2"]}


def run(state):
    return _framework(state) if own else _plain(state)


# -------------------------------------------------------------- the floor
def work(case):
    op, r = case["op"], case["rows"]
    if op == "norm_forward":
        n = r * case["cols"]
        return {"bytes": 2 * n * SIZE[case["type"]] + 8 * r + 8 * case["cols"], "flops": 8 * n}
    if op == "norm_backward":
        n = r * case["cols"]
        b = SIZE[case["type"]]
        kept = b if case["kept"] == "full" else 1 + 4 / TILE
        return {"bytes": int(n * (2 * b + kept)) + 8 * r + 12 * case["cols"], "flops": 14 * n}
    if op == "keep":  # written, and read back
        n = r * case["cols"]
        return {"bytes": int(2 * n * (SIZE[case["type"]] + 1 + 4 / TILE)), "flops": 4 * n}
    if op == "swiglu_backward":
        n = r * case["inter"]
        return {"bytes": int(n * (4 + 2 * (1 + 4 / TILE) + 2 * (1 + 4 / TILE))), "flops": 16 * n}
    d, i, b = case["d"], case["inter"], SIZE[case["type"]]
    if op == "ffn_forward":
        return {"bytes": b * (3 * d * i + 2 * r * d), "flops": 6 * r * d * i}
    # x, dy in; y, dx out; the weights in and their gradients out; the kept values out and in
    return {"bytes": b * (6 * d * i + 4 * r * d) + int(4 * r * i * (1 + 4 / TILE)),
            "flops": 18 * r * d * i}


# ------------------------------------------------- the definition, 64 bits
def _e4m3_64(v):
    """The E4M3 number nearest to v, ties to the even code, |v| up to 448: three mantissa bits
    from 2^-6 up, steps of 2^-9 below."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -40))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _keep_64(v):
    """The codes' numbers [rows, cols], the scales [tiles, rows] and the values kept."""
    rows, cols = v.shape
    wide = torch.nn.functional.pad(v, (0, up(cols, TILE) - cols)).reshape(rows, -1, TILE)
    top = wide.abs().max(2, keepdim=True).values
    scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
    code = _e4m3_64(wide / scale)
    value = (code * scale).reshape(rows, -1)[:, :cols]
    return code.reshape(rows, -1)[:, :cols], scale[:, :, 0].t(), value


def _kept_64(codes, scales):
    n = codes.to(torch.int32)
    sign = 1.0 - 2.0 * (n >> 7).double()
    e, m = (n >> 3) & 15, (n & 7).double()
    mag = torch.where(e > 0, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0), m * 2.0 ** -9)
    return sign * mag * scales.double().t().repeat_interleave(TILE, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, f = case["op"], torch.float64
    if op == "norm_forward":
        x = s["x"].to(f)
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        return {"y": torch.addcmul(s["bias"].to(f), (x - mean[:, None]) * rstd[:, None],
                                   s["weight"].to(f)), "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        cols, dy, r = case["cols"], s["dy"].to(f), s["rstd"].to(f)[:, None]
        x = s["x"].to(f) if case["kept"] == "full" else _kept_64(s["x"], s["x_scales"])[:, :cols]
        xh = (x - s["mean"].to(f)[:, None]) * r
        gr = dy * s["weight"].to(f)
        along = torch.einsum("rc,rc->r", gr, xh)[:, None] / cols
        dx = (gr - gr.sum(1, keepdim=True) / cols - along * xh) * r
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xh), "dbias": dy.sum(0)}
    if op == "keep":
        code, scale, value = _keep_64(s["x"].to(f))
        return {"codes": code, "scales": scale, "back": value}
    if op == "swiglu_backward":
        inter = case["inter"]
        ac, dh = _kept_64(s["ac"], s["ac_scales"]), s["dh"].to(f)
        a, c = ac.split(inter, 1)
        sig = torch.sigmoid(a)
        code, scale, _ = _keep_64(torch.cat([dh * c * (sig + a * sig * (1 - sig)), dh * (a * sig)], 1))
        return {"codes": code, "scales": scale}
    x, w1, w3, w2 = s["x"].to(f), *s["w13"].to(f).split(case["inter"], 0), s["w2"].to(f)
    a, c = torch.einsum("td,id->ti", x, w1), torch.einsum("td,id->ti", x, w3)
    y = torch.einsum("ti,di->td", a * torch.sigmoid(a) * c, w2)
    if op == "ffn_forward":
        return {"y": y}
    a, c = _keep_64(a)[2], _keep_64(c)[2]
    sig, dy = torch.sigmoid(a), s["dy"].to(f)
    dh = torch.einsum("td,di->ti", dy, w2)
    da, dc = dh * c * (sig + a * sig * (1 - sig)), dh * (a * sig)
    return {"y": y, "dx": torch.einsum("ti,id->td", da, w1) + torch.einsum("ti,id->td", dc, w3),
            "dw13": torch.cat([torch.einsum("ti,td->id", da, x), torch.einsum("ti,td->id", dc, x)], 0),
            "dw2": torch.einsum("td,ti->di", dy, a * sig * c)}
