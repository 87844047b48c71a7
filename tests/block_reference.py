"""Plain 64-bit evaluation of the block operators (formulas of include/hcgr.h)
and the error bounds that the tests hold the kernels to.

Every output comes with an amplitude: the formula evaluated with the absolute
values of its terms. A kernel computes in 32 bits and rounds once, so its
distance from the 64-bit value is at most

    eps/2 * |value|  +  C * 2^-24 * amplitude  (+ half a subnormal step),

eps that of the output's type. C counts the 32-bit roundings on the longest
path to a value: a row sum takes at most 64 additions in a thread (65536
channels, 1024 threads), 6 across a wave and 16 across waves, and a value
passes two such sums one after the other (their square roots halve the first)
and some ten products: C = 192. Sums over M tokens add at most M more.
"""
from __future__ import annotations

import torch

C_ROW = 192
U32 = 2.0 ** -24


def gate(inj, hc):
    e = torch.exp(-inj.double() / hc)
    return 2 / (1 + e), 2 * e / (1 + e) ** 2 / hc


def rms(v, eps):
    return 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def norm(x, w, eps):
    x, g = x.double(), 1 + w.double()
    r = rms(x, eps)
    v = x * r * g
    return {"x": (v, v.abs()), "rrms": (r[:, 0], r[:, 0])}


def norm_grad(v, r, g, d, amp_d=None, amp_v=None):
    """Gradient in v of v*r*g from d, its amplitude, and the terms of g's."""
    amp_d = d.abs() if amp_d is None else amp_d
    amp_v = v.abs() if amp_v is None else amp_v
    h, ah, e, ae = v * r, amp_v * r, d * g, amp_d * g.abs()
    grad = r * (e - h * (e * h).mean(-1, keepdim=True))
    amp = r * (ae + ah * (ae * ah).mean(-1, keepdim=True))
    return grad, amp, d * h, amp_d * ah


def norm_bwd(x, w, rrms, dxn):
    dx, adx, t, at = norm_grad(x.double(), rrms.double()[:, None], 1 + w.double(), dxn.double())
    return {"dx": (dx, adx), "dw": (t.sum(0), at.sum(0))}


def _streams(R, y, inj, w_post, ry, hc, rho):
    m, hs = y.shape
    R, y = R.double().view(m, hc, hs), y.double()
    g = 1 + w_post.double() if w_post is not None else torch.ones_like(y[0])
    z = y * ry * g
    iw, slope = gate(inj, hc) if inj is not None else (torch.ones((m, hc), device=y.device).double(),) * 2
    R2 = rho * R + iw[:, :, None] * z[:, None, :]
    aR2 = (rho * R).abs() + iw[:, :, None] * z.abs()[:, None, :]
    return y, g, z, iw, slope, R2, aR2


def residual(R, y, inj, w_post, w_pre, *, hc, eps, rho):
    ry = rms(y.double(), eps) if w_post is not None else torch.ones((y.shape[0], 1), device=y.device).double()
    _, _, _, _, _, R2, aR2 = _streams(R, y, inj, w_post, ry, hc, rho)
    out = {"R2": (R2.flatten(1), aR2.flatten(1))}
    cols = [ry[:, 0]]
    if w_pre is not None:
        u, g = R2.mean(1), 1 + w_pre.double()
        ru = rms(u, eps)
        out["x"] = (u * ru * g, aR2.mean(1) * ru * g.abs())
        cols.append(ru[:, 0])
    out["rrms"] = cols
    return out


def residual_bwd(R, y, inj, w_post, w_pre, rrms, dR2, dx, *, hc, rho):
    m, hs = y.shape
    one = torch.ones((m, 1), device=y.device).double()
    ry = rrms.double()[:, :1] if w_post is not None else one
    y, g, z, iw, slope, R2, aR2 = _streams(R, y, inj, w_post, ry, hc, rho)
    d = dR2.double().view(m, hc, hs) if dR2 is not None else torch.zeros_like(R2)
    ad = d.abs()
    out = {}
    if w_pre is not None:
        du, adu, t, at = norm_grad(R2.mean(1), rrms.double()[:, 1:], 1 + w_pre.double(), dx.double(),
                                   amp_v=aR2.mean(1))
        d, ad = d + du[:, None] / hc, ad + adu[:, None] / hc
        out["dw_pre"] = (t.sum(0), at.sum(0))
    out["dR"] = ((rho * d).flatten(1), (abs(rho) * ad).flatten(1))
    if inj is not None:
        out["dinj"] = ((d * z[:, None]).sum(-1) * slope, (ad * z.abs()[:, None]).sum(-1) * slope)
    dz, adz = (iw[:, :, None] * d).sum(1), (iw[:, :, None] * ad).sum(1)
    if w_post is None:
        out["dy"] = (dz, adz)
    else:
        dy, ady, t, at = norm_grad(y, ry, g, dz, amp_d=adz)
        out["dy"] = (dy, ady)
        out["dw_post"] = (t.sum(0), at.sum(0))
    return out


def linear(q, q_scale, w, w_scale, bias):
    acc = torch.mm(q.double(), w.double().t().contiguous())  # exact: below 2^53
    p = acc * q_scale.double()[:, None] * w_scale.double()[None, :]
    b = bias.double() if bias is not None else torch.zeros_like(w_scale).double()
    return p + b, p.abs() + b.abs()


def check(got, ref, what, c=C_ROW):
    """got within the bound of ref = (value, amplitude)."""
    val, amp = ref
    assert got.shape == val.shape, (what, got.shape, val.shape)
    f = torch.finfo(got.dtype)
    err = (got.double() - val).abs()
    pre = c * U32 * amp
    lim = f.eps / 2 * (val.abs() + pre) + pre + f.smallest_normal * f.eps / 2
    bad = ~(err <= lim)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; worst {float((err / lim).nan_to_num(9e9).max()):.3g} times it, "
        f"first at {tuple(bad.nonzero()[0].tolist())}: got {float(got[bad][0])}, want {float(val[bad][0])}")


def check_quantized(q, scale, v, amp, what, c=C_ROW):
    """q, scale against the unrounded values v (64 bits): the scale of the
    largest value, and each q within half a step of v/scale plus what 32 bits
    leave open."""
    s = v.abs().amax(1) / 127
    slack = c * U32 * (amp.amax(1) / 127)
    err = (scale.double() - s).abs()
    assert bool((err <= slack + 2 * U32 * s + 2.0 ** -149).all()), f"{what}: scale off by {float((err / s).max()):.3g}"
    ok = s > 2.0 ** -120
    t = v[ok] / s[ok, None]
    lim = 0.5 + (c + 4) * U32 * 127 * (amp[ok].amax(1) / (127 * s[ok]))[:, None]
    d = (q[ok].double() - t).abs()
    assert bool((d <= lim).all()), f"{what}: q off by {float(d.max()):.6g} steps"
    assert bool((q.abs() <= 127).all()), what
    zero = v.abs().amax(1) == 0
    assert bool((q[zero] == 0).all()) and bool((scale[zero] == 0).all()), what
