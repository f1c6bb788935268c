"""The gradient of the decays where these are strong, in 64 bits on the CPU: the sum of all that
crosses a token, which the kernels compute, against the recurrence's chain rule, and that
against differences."""
import pytest
import torch

from tests import delta_ref as delta


def make(T, H, dk, dv, low, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    return dict(q=unit(r(T, H, dk)), k=unit(r(T, H, dk)), v=r(T, H, dv), g=low * (1 / 3 + 2 / 3 * u(T, H)), beta=u(T, H),
                s0=r(1, H, dk, dv), ds=r(1, H, dk, dv), dy=r(T, H, dv))


def crossing(x, scale):
    """dg of one chunk from its pairs, the state that enters, and the gradient of the state behind it."""
    T, H, _ = x["v"].shape
    cu = [0, T]
    seen = delta.steps(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, x["s0"], scale)[2]
    dvv = delta.grad(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, x["dy"], x["s0"], x["ds"], scale)[2]
    e = torch.stack([s[2] for s in seen])
    out = torch.zeros(T, H, dtype=torch.float64)
    for h in range(H):
        q, k, b, dy, dv, E = x["q"][:, h], x["k"][:, h], x["beta"][:, h], x["dy"][:, h], dvv[:, h], e[:, h]
        S, R, G = x["s0"][0, h], x["ds"][0, h], x["g"][:, h].cumsum(0)
        D = torch.exp(G[:, None] - G[None]).tril(-1)
        N = ((scale * (dy @ E.t()) * (q @ k.t()) - (dv @ E.t()) * (k @ k.t())) * D).nan_to_num(0) * b[None]
        a = torch.exp(G) * (scale * (q * (dy @ S.t())).sum(-1) - (k * (dv @ S.t())).sum(-1))
        c = torch.exp(G[-1] - G) * b * (k * (E @ R.t())).sum(-1)
        for t in range(T):
            out[t, h] = N[t:, :t].sum() + a[t:].sum() + c[:t].sum() + torch.exp(G[-1]) * (S * R).sum()
    return out


@pytest.mark.parametrize("low", [-0.3, -6.0, -12.0, -40.0])
def test_what_crosses_a_token(low):
    x = make(20, 2, 5, 7, low, 3)
    want = delta.grad(x["q"], x["k"], x["v"], x["g"], x["beta"], [0, 20], x["dy"], x["s0"], x["ds"], 0.7)[3]
    got = crossing(x, 0.7)
    # 64 bits: some hundred terms of a few 1e-16 each
    assert bool(((got - want).norm(dim=0) <= 1e-13 * want.norm(dim=0)).all())


@pytest.mark.parametrize("low", [-6.0, -12.0])
def test_strong_decays_against_differences(low):
    x, cu, T = make(6, 2, 3, 4, low, 4), [0, 6], 6

    def loss(g):
        y, S, _ = delta.steps(x["q"], x["k"], x["v"], g, x["beta"], cu, x["s0"], 0.7)
        return float((y * x["dy"]).sum() + (S * x["ds"]).sum())
    want = delta.grad(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, x["dy"], x["s0"], x["ds"], 0.7)[3]
    h = 1e-3
    for t in range(T):
        for i in range(2):
            up, down = x["g"].clone(), x["g"].clone()
            up[t, i] += h
            down[t, i] -= h
            # in exp(g) the loss is linear: sinh(h) / h is 1 + h^2 / 6; the loss itself is off by some 1e-15 of about 10
            assert abs((loss(up) - loss(down)) / (2 * h) - float(want[t, i])) <= h * h / 5 * abs(float(want[t, i])) + 1e-11
