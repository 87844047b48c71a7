"""The layer norm's gradient along the two directions of a row in which the norm
does not move: all values together (u = 1), and all deviations in proportion
(u = h = (x - mean)/deviation, up to eps). The derivative of sum_c xn[c] d[c] is
then 0, or of the size of eps; it is the sum of dx = r*(e - mean(e) - h*mean(e*h))
along u, e = d*w, in which a missing mean(e) leaves r*HS*mean(e) for u = 1 and a
missing mean(e*h) r*HS*mean(e*h) for u = h. The rows of d are made so that both
means are near 1."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
STEP = 0.25


def deviations(x):
    d = x.double() - x.double().mean(1, keepdim=True)
    return d / (d * d).mean(1, keepdim=True).sqrt()


def upstream(x, w, noise):
    """d [M, HS] in 32 bits with mean(d*w) and mean(d*w*h) near 1."""
    return ((1 + deviations(x) + 0.3 * noise.double()) / w.double()).float()


def check(forward, dx, x, w, d, amp, dx_amp, c):
    """forward: x [M, HS] float32 -> xn. Its values are off by at most U32 * (|xn|
    + c*amp), those of dx by U32 * (|dx| + c*dx_amp) (amplitudes as in
    block_reference). Each row's slope from dx has to equal the central difference
    with step t = STEP up to what follows from the two: twice the first bound's sum
    over |d|, over 2t, and the second's over |u|.

    The points x +- t*u are rounded to 32 bits; u is taken from the rounded points.
    What is left: their midpoint lies off x by half a step of 32 bits, and along h
    the norm bends by eps (third derivative below 15 eps in units of the deviation,
    t^2/6 of it a value); with |e*h| of order 1 and eps = 1e-6 both are below 1e-6 a
    value."""
    for name, u in (("1", torch.ones_like(x)), ("h", deviations(x).float())):
        hi, lo = x + STEP * u, x - STEP * u
        up, down = forward(hi).double(), forward(lo).double()
        want = ((up - down) * d.double()).sum(1) / (2 * STEP)
        u = (hi.double() - lo.double()) / (2 * STEP)
        got = (dx.double() * u).sum(1)
        lim = (U32 * (up.abs().maximum(down.abs()) + 2 * c * amp) * d.double().abs()).sum(1) / STEP + \
            (U32 * (dx.double().abs() + c * dx_amp) * u.abs()).sum(1) + 1e-6 * x.shape[1]
        bad = ~((got - want).abs() <= lim)
        assert not bool(bad.any()), (name, got[bad][0].item(), want[bad][0].item(), lim[bad][0].item())
