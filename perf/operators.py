"""Workloads of the operators around a block that is fed by hyper-connection
streams: the norm before the block, the norm after it with its gates, its
residual scale and the next norm (both with their gradients), and the 8-bit
integer projections inside it.

``listed()`` names the fixed cases and ``draw(rng)`` gives further ones of the
same ranges; ``prepare`` makes what a program has in hand, ``run`` makes one
pass, ``work`` counts the bytes and operations the pass cannot do without, and
``exact`` evaluates the definition in 64 bits. With ``own`` false ``run``
computes the plain forms, with ``own`` true it calls the library.

Definitions, for one token (HC streams of HS channels, weights w enter as 1 + w):

    norm(v, w)  = v / sqrt(mean(v^2) + eps) * (1 + w)
    residual    z = norm(y, w_post);  iw[s] = 2 sigmoid(inj[s] / HC)
                R2[s] = rho R[s] + iw[s] z;  x = norm(mean_s R2[s], w_pre)
    quantize    scale = max|v| / 127;  q = round_half_even(v / scale)
    linear      out[n] = (sum_k q[k] W[n, k]) * scale * w_scale[n] + bias[n]
"""
import math

import torch

own = False

EPS = 1e-6
RHO = 0.75  # residual scale of the residual cases (0.5 and 1 behave alike)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}

# Limits of drawn cases, under the largest listed ones.
DRAW_BYTES = 4e8
DRAW_FLOPS = 2e11


def listed():
    return [
        # the norm before a block: one decode step of 16 sequences, and a
        # prefill of ragged length in fp16 at a width that is no power of two
        {"name": "norm decode M=16", "op": "norm", "m": 16, "hs": 2560, "dtype": "bf16"},
        {"name": "norm prefill M=4099 hs=1000", "op": "norm", "m": 4099, "hs": 1000, "dtype": "fp16"},
        # its gradient in a training step of 8192 tokens
        {"name": "norm backward M=8192", "op": "norm_bwd", "m": 8192, "hs": 2560, "dtype": "bf16"},
        # the norm after a block, gates, residual and next norm: one decode
        # token (latency), a short ragged prompt over two narrow streams, and
        # a long prefill over four streams
        {"name": "residual decode M=1", "op": "residual", "m": 1, "hc": 4, "hs": 2560, "dtype": "bf16"},
        {"name": "residual M=333 hc=2 hs=1000", "op": "residual", "m": 333, "hc": 2, "hs": 1000, "dtype": "fp16"},
        {"name": "residual prefill M=16384", "op": "residual", "m": 16384, "hc": 4, "hs": 2560, "dtype": "bf16"},
        # its gradient: four streams in bf16, and a single fp32 stream
        {"name": "residual backward M=8192", "op": "residual_bwd", "m": 8192, "hc": 4, "hs": 2560, "dtype": "bf16"},
        {"name": "residual backward M=2047 fp32", "op": "residual_bwd", "m": 2047, "hc": 1, "hs": 2560,
         "dtype": "fp32"},
        # norm + quantised projection of one decode token into a wide layer
        {"name": "norm+linear decode M=1", "op": "norm_linear", "m": 1, "k": 2560, "n": 10240, "dtype": "bf16",
         "bias": False},
        # back from the wide layer for 32 sequences: activations are quantised in the call
        {"name": "quantize+linear decode M=32", "op": "quant_linear", "m": 32, "k": 10240, "n": 2560,
         "dtype": "bf16", "bias": False},
        # a ragged product with a bias and fp32 results
        {"name": "linear M=300 N=777 K=1000", "op": "linear", "m": 300, "k": 1000, "n": 777, "dtype": "fp32",
         "bias": True},
        # a prefill's projection
        {"name": "linear prefill M=8192", "op": "linear", "m": 8192, "k": 2560, "n": 10240, "dtype": "bf16",
         "bias": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "residual", "residual_bwd", "norm_linear", "quant_linear", "linear"))
    while True:
        c = {"op": op, "m": _log_int(rng, 1, 16384)}
        if op.endswith("linear"):
            c["k"] = _log_int(rng, 64, 10240)
            c["n"] = _log_int(rng, 16, 10240)
            if rng.random() < 0.6:  # whole 64-byte pieces, as layers mostly have
                c["k"] = max(64, c["k"] // 64 * 64)
                c["n"] = max(16, c["n"] // 16 * 16)
            # quantised in the call, results are bf16 or fp16; a product of given integers may end in fp32
            c["dtype"] = rng.choice(("bf16", "bf16", "fp16") if op != "linear" else ("bf16", "fp16", "fp32"))
            c["bias"] = rng.random() < 0.5
        else:
            if op.startswith("residual"):
                c["hc"] = rng.choice((1, 2, 4, 8))
            c["hs"] = _log_int(rng, 64, 8192)
            if rng.random() < 0.8:  # whole 16-byte pieces; the rest are odd widths
                c["hs"] = max(64, c["hs"] // 8 * 8)
            c["dtype"] = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        w = work(c)
        if w["bytes"] <= DRAW_BYTES and w["flops"] <= DRAW_FLOPS:
            return c


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, m, n, dtype):
    """Normal values whose channels differ in size, a few of them by far."""
    size = torch.exp(0.4 * _randn(g, n))
    size = torch.where(torch.rand(n, generator=g, device="cuda") < 0.005, 8 * size, size)
    return (_randn(g, m, n) * size).to(dtype)


def _pitched_int8(v):
    """int8 rows at a pitch of whole 16-byte pieces, as the library reads them."""
    m, k = v.shape
    t = torch.zeros((m, (k + 15) // 16 * 16), dtype=torch.int8, device=v.device)
    t[:, :k] = v
    return t[:, :k]


def _rrms(v):
    return (1.0 / torch.sqrt(v.double().square().mean(-1) + EPS)).float()


def prepare(case, seed):
    g, op, m, dt = _gen(seed), case["op"], case["m"], DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op in ("norm", "norm_bwd"):
        hs = case["hs"]
        s["x"] = _activations(g, m, hs, dt)
        s["w"] = (0.1 * _randn(g, hs)).to(dt)
        if op == "norm_bwd":
            s["dxn"] = _randn(g, m, hs).to(dt)
            s["rrms"] = _rrms(s["x"])
    elif op in ("residual", "residual_bwd"):
        hc, hs = case["hc"], case["hs"]
        s["R"] = torch.cat([_activations(g, m, hs, dt) for _ in range(hc)], dim=1)
        s["y"] = _activations(g, m, hs, dt)
        s["inj"] = _randn(g, m, hc).to(dt)
        s["w_post"] = (0.1 * _randn(g, hs)).to(dt)
        s["w_pre"] = (0.1 * _randn(g, hs)).to(dt)
        if op == "residual_bwd":
            s["dR2"] = _randn(g, m, hc * hs).to(dt)
            s["dx"] = _randn(g, m, hs).to(dt)
            # the forward pass saved both reciprocal RMS values of each token
            z = s["y"].double() * _rrms(s["y"]).double()[:, None] * (1 + s["w_post"].double())
            iw = 2 * torch.sigmoid(s["inj"].double() / hc)
            u = RHO * s["R"].double().view(m, hc, hs).mean(1) + iw.mean(1, keepdim=True) * z
            s["rrms"] = torch.stack([_rrms(s["y"]), _rrms(u)], dim=1).contiguous()
    else:
        k, n = case["k"], case["n"]
        w = (_randn(g, n, k) * 30).round().clamp(-127, 127)
        s["wq"] = _pitched_int8(w.to(torch.int8))
        s["w_scale"] = (0.5 + torch.rand(n, generator=g, device="cuda")) / (30 * math.sqrt(k))
        s["bias"] = _randn(g, n).to(dt) if case["bias"] else None
        if op == "linear":
            v = _activations(g, m, k, torch.float32)
            scale = v.abs().amax(1) / 127
            s["q"] = _pitched_int8((v / scale[:, None]).round().clamp(-127, 127).to(torch.int8))
            s["q_scale"] = scale
        else:
            s["x"] = _activations(g, m, k, dt)
            if op == "norm_linear":
                s["w"] = (0.1 * _randn(g, k)).to(dt)
    return s


# ------------------------------------------------------- the library's calls --
def _own(s):
    c = s["case"]
    f = s.get("call")
    if f is None:  # first pass: what a program builds once, handles and output buffers
        import skinny_gemm_hcgr_amd as H
        dt = {"bf16": H.HCGR_BF16, "fp16": H.HCGR_FP16, "fp32": H.HCGR_FP32}[c["dtype"]]
        op, m = c["op"], c["m"]
        if op.endswith("linear"):
            lin = H.Int8Linear(H.LinearConfig(n=c["n"], k=c["k"], dtype=dt), 0)
            out = lin.alloc_output(m)
            args = (s["wq"], s["w_scale"], s["bias"])
            if op == "linear":
                f = lambda: lin.forward(s["q"], s["q_scale"], *args, out=out)  # noqa: E731
            elif op == "quant_linear":
                q = lin.alloc_quantized(m)
                f = lambda: lin.forward(*lin.quantize(s["x"], out=q), *args, out=out)  # noqa: E731
            else:
                blk = H.Block(H.BlockConfig(hc=1, hs=c["k"], dtype=dt, eps=EPS), 0)
                nrm = blk.alloc_norm(m, quantize=True)

                def f():
                    blk.norm(s["x"], s["w"], out=nrm)
                    return lin.forward(nrm["q"], nrm["q_scale"], *args, out=out)
        elif op in ("norm", "norm_bwd"):
            blk = H.Block(H.BlockConfig(hc=1, hs=c["hs"], dtype=dt, eps=EPS), 0)
            if op == "norm":
                out = blk.alloc_norm(m)
                f = lambda: blk.norm(s["x"], s["w"], out=out)  # noqa: E731
            else:
                out = blk.alloc_norm_bwd(m)
                f = lambda: blk.norm_bwd(s["x"], s["w"], s["rrms"], s["dxn"], out=out)  # noqa: E731
        else:
            blk = H.Block(H.BlockConfig(hc=c["hc"], hs=c["hs"], dtype=dt, eps=EPS, res_scale=RHO), 0)
            a = (s["R"], s["y"], s["inj"], s["w_post"], s["w_pre"])
            if op == "residual":
                out = blk.alloc_residual(m)
                f = lambda: blk.residual(*a, out=out)  # noqa: E731
            else:
                out = blk.alloc_residual_bwd(m)
                f = lambda: blk.residual_bwd(*a, s["rrms"], s["dR2"], s["dx"], out=out)  # noqa: E731
        s["call"] = f
    return f()


# ------------------------------------------------------------- plain forms --
def _norm(v, w):
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * r * (1 + w), r


def _norm_grad(v, r, w, d):
    """Gradients of v * r * (1 + w) in v and w, r = 1/sqrt(mean v^2 + eps)."""
    h = v * r
    dh = d * (1 + w)
    return r * (dh - h * (dh * h).mean(-1, keepdim=True)), (d * h).sum(0)


def _quantize(v):
    scale = v.abs().amax(-1, keepdim=True) / 127
    return torch.round(v / scale).clamp(-127, 127), scale


def _project(s, q, scale):
    out = (q @ s["wq"].float().t()) * scale * s["w_scale"]
    return out + s["bias"].float() if s["bias"] is not None else out


def run(state):
    if own:
        return _own(state)
    s, c = state, state["case"]
    op, m, dt = c["op"], c["m"], DTYPES[c["dtype"]]
    if op == "norm":
        x, r = _norm(s["x"].float(), s["w"].float())
        return {"x": x.to(dt), "rrms": r[:, 0]}
    if op == "norm_bwd":
        dx, dw = _norm_grad(s["x"].float(), s["rrms"][:, None], s["w"].float(), s["dxn"].float())
        return {"dx": dx.to(dt), "dw": dw}
    if op == "linear":
        return _project(s, s["q"].float(), s["q_scale"][:, None]).to(dt)
    if op == "quant_linear":
        return _project(s, *_quantize(s["x"].float())).to(dt)
    if op == "norm_linear":
        return _project(s, *_quantize(_norm(s["x"].float(), s["w"].float())[0])).to(dt)
    hc, hs = c["hc"], c["hs"]
    R, y = s["R"].float().view(m, hc, hs), s["y"].float()
    w_post, w_pre = s["w_post"].float(), s["w_pre"].float()
    sig = torch.sigmoid(s["inj"].float() / hc)
    if op == "residual":
        z, ry = _norm(y, w_post)
        R2 = RHO * R + 2 * sig[:, :, None] * z[:, None, :]
        x, ru = _norm(R2.mean(1), w_pre)
        return {"R2": R2.view(m, hc * hs).to(dt), "x": x.to(dt), "rrms": torch.cat([ry, ru], dim=1)}
    ry, ru = s["rrms"][:, :1], s["rrms"][:, 1:]
    z = y * ry * (1 + w_post)
    u = RHO * R.mean(1) + 2 * sig.mean(1, keepdim=True) * z
    du, dw_pre = _norm_grad(u, ru, w_pre, s["dx"].float())
    d = s["dR2"].float().view(m, hc, hs) + du[:, None, :] / hc
    diw = (d * z[:, None, :]).sum(-1)
    dy, dw_post = _norm_grad(y, ry, w_post, (2 * sig[:, :, None] * d).sum(1))
    return {"dR": (RHO * d).view(m, hc * hs).to(dt), "dy": dy.to(dt),
            "dinj": (diw * 2 * sig * (1 - sig) / hc).to(dt), "dw_post": dw_post, "dw_pre": dw_pre}


def work(case):
    """Each input read once and each output written once, in the case's types;
    operations of the sums, products and divisions (two a multiply-add)."""
    op, m, b = case["op"], case["m"], BYTES[case["dtype"]]
    if op.endswith("linear"):
        k, n = case["k"], case["n"]
        x = m * k + 4 * m if op == "linear" else m * k * b + (k * b if op == "norm_linear" else 0)
        return {"bytes": x + n * k + 4 * n + (n * b if case["bias"] else 0) + m * n * b, "flops": 2 * m * n * k}
    hs = case["hs"]
    if op == "norm":
        return {"bytes": 2 * m * hs * b + hs * b + 4 * m, "flops": 4 * m * hs}
    if op == "norm_bwd":
        return {"bytes": 3 * m * hs * b + hs * b + 4 * m + 4 * hs, "flops": 9 * m * hs}
    k = case["hc"] * hs
    if op == "residual":
        return {"bytes": m * (2 * k + 2 * hs + case["hc"]) * b + 2 * hs * b + 8 * m, "flops": m * (4 * k + 8 * hs)}
    return {"bytes": m * (3 * k + 3 * hs + 2 * case["hc"]) * b + 2 * hs * b + 8 * m + 8 * hs,
            "flops": m * (8 * k + 18 * hs)}


# --------------------------------------------------- the definitions, 64 bits --
def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits, written from them
    and not from the plain forms: the gradients go through a product with the
    Jacobian of v/sqrt(mean v^2 + eps) taken apart as (I - v v^T r^2 / n) r."""
    s = prepare(case, seed)
    op, m = case["op"], case["m"]
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}

    def norm(v, w):
        r = (v.pow(2).sum(1) / v.shape[1] + EPS).pow(-0.5)
        return v * r[:, None] * (1 + w)[None, :], r

    def jacobian(v, r, d):
        along = (v * d).sum(1) * r.pow(3) / v.shape[1]
        return d * r[:, None] - v * along[:, None]

    if op == "norm":
        x, r = norm(f["x"], f["w"])
        return {"x": x, "rrms": r}
    if op == "norm_bwd":
        dx = jacobian(f["x"], f["rrms"], f["dxn"] * (1 + f["w"]))
        return {"dx": dx, "dw": (f["dxn"] * f["x"] * f["rrms"][:, None]).sum(0)}
    if op.endswith("linear"):
        if op == "linear":
            q, scale = f["q"], f["q_scale"]
        else:
            v = norm(f["x"], f["w"])[0] if op == "norm_linear" else f["x"]
            scale = v.abs().max(dim=1).values / 127
            q = torch.round(v / scale[:, None])
        out = torch.mm(q, f["wq"].transpose(0, 1).contiguous()) * torch.outer(scale, f["w_scale"])
        return out if s["bias"] is None else out + f["bias"][None, :]
    hc, hs = case["hc"], case["hs"]
    R = f["R"].reshape(m, hc, hs)
    e = torch.exp(-f["inj"] / hc)
    iw = 2 / (1 + e)
    if op == "residual":
        z, ry = norm(f["y"], f["w_post"])
        R2 = R * RHO
        R2 += iw[:, :, None] * z[:, None, :]
        x, ru = norm(R2.sum(1) / hc, f["w_pre"])
        return {"R2": R2.reshape(m, hc * hs), "x": x, "rrms": torch.stack((ry, ru), 1)}
    ry, ru = f["rrms"][:, 0], f["rrms"][:, 1]
    yh = f["y"] * ry[:, None]
    z = yh * (1 + f["w_post"])
    u = (RHO * R.sum(1) + iw.sum(1)[:, None] * z) / hc
    du = jacobian(u, ru, f["dx"] * (1 + f["w_pre"]))
    d = f["dR2"].reshape(m, hc, hs) + (du / hc)[:, None, :]
    dz = (d * iw[:, :, None]).sum(1)
    diw = (d * z[:, None, :]).sum(2)
    return {"dR": (d * RHO).reshape(m, hc * hs), "dy": jacobian(f["y"], ry, dz * (1 + f["w_post"])),
            "dinj": diw * 2 * e / (1 + e).pow(2) / hc, "dw_post": (dz * yh).sum(0),
            "dw_pre": (f["dx"] * u * ru[:, None]).sum(0)}
