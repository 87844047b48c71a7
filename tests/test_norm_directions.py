"""That the check of the layer norm's gradient along 1 and h takes the right
gradient and none with a term missing or off, in the 64-bit reference."""
import pytest
import torch

import mx_reference as X
import norm_directions as N

EPS = 1e-6
WIDTHS = [33, 67, 1000, 2560, 8192]


def setting(hs, m=4):
    g = torch.Generator().manual_seed(hs)
    x = torch.randn(m, hs, generator=g) + 1.0
    w, b = 1 + 0.2 * torch.randn(hs, generator=g).clamp(-3, 3), torch.randn(hs, generator=g)
    d = N.upstream(x, w, torch.randn(m, hs, generator=g))
    f = X.layer_norm(x, w, b, EPS)
    stats = torch.stack([f["mean"][0], f["r"][0]], 1)
    return x, w, b, d, stats, f["x"][1]


def checked(hs, dx):
    x, w, b, d, stats, amp = setting(hs)
    e, h = d.double() * w.double(), (x.double() - stats[:, :1]) * stats[:, 1:]
    N.check(lambda v: X.layer_norm(v, w, b, EPS)["x"][0], dx(e, h, stats[:, 1:]), x, w, d, amp,
            X.layer_norm_bwd(x, w, stats, d)["dx"][1], 192)


def mean(t):
    return t.mean(1, keepdim=True)


@pytest.mark.parametrize("hs", WIDTHS)
def test_the_gradient_passes(hs):
    checked(hs, lambda e, h, r: r * (e - mean(e) - h * mean(e * h)))


@pytest.mark.parametrize("hs", WIDTHS)
@pytest.mark.parametrize("wrong", [
    lambda e, h, r: r * (e - h * mean(e * h)),                       # no mean of e
    lambda e, h, r: r * (e - mean(e)),                               # no mean of e*h
    lambda e, h, r: r * e,
    lambda e, h, r: r * (e - mean(e) - mean(e * h)),                 # its factor h missing
    lambda e, h, r: r * (e - mean(e) - h * mean(e) * mean(h)),       # a product of means
    lambda e, h, r: r * (e - mean(e) + h * mean(e * h)),             # a sign
    lambda e, h, r: r * (e - 0.99 * mean(e) - h * mean(e * h)),      # a sum that loses values
    lambda e, h, r: r * (e - mean(e) - h * 0.99 * mean(e * h))])
def test_wrong_gradients_are_found(hs, wrong):
    with pytest.raises(AssertionError):
        checked(hs, wrong)
