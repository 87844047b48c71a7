"""The 64-bit reference of the block operators on the CPU: its gradients
against central differences of its forward pass."""
import pytest
import torch

import block_reference as B


def _rand(*shape, g):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def _differences(f, t, h=1e-6):
    """Central differences of the scalar f() in every value of t (in place)."""
    flat, out = t.view(-1), torch.zeros(t.numel(), dtype=torch.float64)
    for i in range(t.numel()):
        x = float(flat[i])
        flat[i] = x + h
        hi = f()
        flat[i] = x - h
        lo = f()
        flat[i] = x
        out[i] = (hi - lo) / (2 * h)
    return out.view(t.shape)


# A central difference is off by h^2 f'''/6 and 2^-53 |f| / h: with h = 1e-6
# and values of order 10, below 1e-7.
TOL = 1e-7


def test_norm_gradient():
    g = torch.Generator().manual_seed(1)
    x, w, d = _rand(3, 5, g=g), 0.3 * _rand(5, g=g), _rand(3, 5, g=g)
    eps = 1e-3
    got = B.norm_bwd(x, w, B.rms(x, eps)[:, 0], d)

    def loss():
        return float((B.norm(x, w, eps)["x"][0] * d).sum())

    for name, t in (("dx", x), ("dw", w)):
        assert torch.allclose(got[name][0], _differences(loss, t), atol=TOL, rtol=TOL), name


@pytest.mark.parametrize("hc", [1, 2, 4])
@pytest.mark.parametrize("gates,post,pre,from_R2", [(1, 1, 1, 1), (0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0)])
def test_residual_gradient(hc, gates, post, pre, from_R2):
    g = torch.Generator().manual_seed(hc)
    m, hs, rho, eps = 2, 5, 0.6, 1e-3
    R, y, inj = _rand(m, hc * hs, g=g), _rand(m, hs, g=g), _rand(m, hc, g=g) if gates else None
    w_post = 0.3 * _rand(hs, g=g) if post else None
    w_pre = 0.3 * _rand(hs, g=g) if pre else None
    dR2 = _rand(m, hc * hs, g=g) if from_R2 else None
    dx = _rand(m, hs, g=g) if pre else None

    def out():
        return B.residual(R, y, inj, w_post, w_pre, hc=hc, eps=eps, rho=rho)

    def loss():
        o = out()
        v = (o["R2"][0] * dR2).sum() if from_R2 else torch.zeros(())
        return float(v + ((o["x"][0] * dx).sum() if pre else 0.0))

    rr = out()["rrms"]
    rrms = torch.stack([rr[0], rr[1] if pre else rr[0]], 1)
    got = B.residual_bwd(R, y, inj, w_post, w_pre, rrms, dR2, dx, hc=hc, rho=rho)
    wrt = {"dR": R, "dy": y, "dinj": inj, "dw_post": w_post, "dw_pre": w_pre}
    assert set(got) == {k for k, t in wrt.items() if t is not None}
    for name, t in wrt.items():
        if t is not None:
            assert torch.allclose(got[name][0], _differences(loss, t), atol=TOL, rtol=TOL), name
