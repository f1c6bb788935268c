"""Plain 64-bit forms of the layer operators on the CPU, token by token, for
the tests: no code shared with the library."""
import math

import torch


def expand(x, H):
    """[T, Hk, d] to [T, H, d]: the value heads that share a key head are neighbours."""
    return x.double().repeat_interleave(H // x.shape[1], 1)


def decays(g, T, H):
    return torch.exp(g.double()).expand(T, H)


def linattn(q, k, v, g, cu, s0=None, scale=1.0):
    T, H, dv = v.shape
    dk = q.shape[-1]
    q, k, v, a = expand(q, H), expand(k, H), v.double(), decays(g, T, H)
    N = len(cu) - 1
    y = torch.zeros(T, H, dv, dtype=torch.float64)
    S = torch.zeros(N, H, dk, dv, dtype=torch.float64) if s0 is None else s0.double().clone()
    before = torch.zeros(T, H, dk, dv, dtype=torch.float64)   # S_{t-1}
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            before[t] = S[n]
            # a decay of 0 clears the state whatever it holds
            S[n] = a[t][:, None, None] * S[n] + k[t][:, :, None] * v[t][:, None, :]
            y[t] = scale * (q[t][:, :, None] * S[n]).sum(1)
    return y, S, before


def linattn_grad(q, k, v, g, cu, dy, s0=None, ds=None, scale=1.0):
    T, H, dv = v.shape
    Hk, dk = q.shape[1], q.shape[2]
    _, _, before = linattn(q, k, v, g, cu, s0, scale)
    q, k, v, a, dy = expand(q, H), expand(k, H), v.double(), decays(g, T, H), scale * dy.double()
    N = len(cu) - 1
    R = torch.zeros(N, H, dk, dv, dtype=torch.float64) if ds is None else ds.double().clone()
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg = torch.zeros(T, H, dtype=torch.float64)
    for n in range(N):
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            S = a[t][:, None, None] * before[t] + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = (S * dy[t][:, None, :]).sum(-1)
            R[n] += q[t][:, :, None] * dy[t][:, None, :]
            dkk[t] = (R[n] * v[t][:, None, :]).sum(-1)
            dvv[t] = (R[n] * k[t][:, :, None]).sum(-2)
            dg[t] = a[t] * (R[n] * before[t]).sum((-1, -2))
            R[n] = a[t][:, None, None] * R[n]
    fold = lambda x: x.view(T, Hk, H // Hk, dk).sum(2)  # noqa: E731
    if g.dim() == 1:
        dg = dg.sum(0)
    return fold(dq), fold(dkk), dvv, dg, R


def rope(x, pos, freq, layout, inverse, m):
    """Pair by pair, from the definition."""
    x = x.double().clone()
    rot = 2 * freq.numel()
    ang = pos.double()[:, None] * freq.double()
    if inverse:
        ang = -ang
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = m * torch.cos(ang[:, i])[:, None], m * torch.sin(ang[:, i])[:, None]
        u, w = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    return x


def norm(x, w, b, z, eps, kind):
    x = x.double()
    m = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    r = 1 / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - m) * r * w.double()
    if b is not None:
        y = y + b.double()
    if z is not None:
        y = y / (1 + torch.exp(-z.double()))
    return y, m[..., 0], r[..., 0]


def norm_grad(x, w, b, z, eps, kind, dy):
    x, dy, w = x.double(), dy.double(), w.double()
    m = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    r = 1 / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    h = (x - m) * r
    dz = None
    if z is not None:
        s = 1 / (1 + torch.exp(-z.double()))
        n = h * w + (0 if b is None else b.double())
        dz = dy * n * s * (1 - s)
        dy = dy * s
    e = dy * w
    dx = r * (e - h * (e * h).mean(-1, keepdim=True) - (e.mean(-1, keepdim=True) if kind == "layer" else 0))
    return dx, (dy * h).sum(0), None if b is None else dy.sum(0), dz


# Largest relative 2-norm of an error, derived from the roundings on the way.
# fp32 in and out: sums of up to a few hundred terms in fp32, each rounding off
#   by 2^-24 at most; of random sign, sqrt(256) 2^-24 = 1e-6 of the terms' size,
#   and the terms' size is up to about 8 times that of their sum: 1e-5.
# bf16 out of fp32 sums: the output's rounding (2^-8 at most, 2^-8 / sqrt(3) in
#   the mean square) and one of an operand inside: sqrt(2 / 3) 2^-8 = 3.2e-3;
#   2^-8 leaves a margin of a fifth.
# fp32 out of bf16 inputs (states, statistics, weight gradients): the operands
#   enter with 24 bits, so as fp32.
# dg: differences of sums over up to 1024 tokens, each with fp32's error of
#   about 2^-22, of random sign: sqrt(1024) 2^-22 = 8e-6 of a token's term: 2e-5.
TOL = {"f32": 1e-5, "bf16": 2.0 ** -8}
TOL_STATE, TOL_DG = 1e-5, 2e-5


def rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), "not finite"
    n = float(ref.norm())
    return float((got - ref).norm()) / n if n > 0 else float(got.norm())


def worst(got, ref):
    """Largest error of one value against its size or the mean size of all."""
    got, ref = got.detach().double().cpu(), ref.double()
    rms = float(ref.square().mean().sqrt())
    if rms == 0 or not math.isfinite(rms):
        return float(got.abs().max()) if got.numel() else 0.0
    return float(((got - ref).abs() / ref.abs().clamp_min(rms)).max()) if got.numel() else 0.0


def check(name, got, ref, tol):
    e, w = rel(got, ref), worst(got, ref)
    print(f"[layer] {name}: rel {e:.2e} worst {w:.2e} (tol {tol:.1e})", flush=True)
    assert e <= tol, f"{name}: rel {e:.3e} > {tol:.3e}"
    # one value: an error of random parts is within 8 times its mean square
    # over the sizes here (up to a few million values), and values have up to
    # that many times the mean size in their terms
    assert w <= 16 * tol, f"{name}: worst value {w:.3e} > {16 * tol:.3e}"
