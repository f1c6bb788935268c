"""The gated delta rule token by token in 64 bits on the CPU, and its gradient
by the chain rule of each step, for the tests: no code shared with the library."""
import torch

from tests.layer_ref import expand

# Largest relative 2-norm of an error, beside layer_ref's for outputs.
# fp32 outputs (states, dbeta): what is computed inside a chunk enters products
#   with 24 bits at best and 16 at least, off by 2^-18 at most; a chunk rounds a
#   state, an error of prediction, a row of the inverse and an update, sqrt(4 / 3)
#   2^-18 = 4.4e-6 of the terms' size, which is up to about twice that of their sum:
#   1e-5.
# dg: differences of two sums over tokens and of the states' product, each term
#   with that error, of random sign: twice as much, 2e-5.
TOL_STATE, TOL_DG = 1e-5, 2e-5


def steps(q, k, v, g, beta, cu, s0, scale):
    """y, final states, and what each token saw: (state before it, decayed state, error)."""
    T, H, dv = v.shape
    q, k, v, beta = expand(q, H), expand(k, H), v.double(), beta.double()
    a = torch.ones(T, H, dtype=torch.float64) if g is None else torch.exp(g.double())
    N = len(cu) - 1
    S = torch.zeros(N, H, q.shape[-1], dv, dtype=torch.float64) if s0 is None else s0.double().clone()
    y, seen = torch.zeros(T, H, dv, dtype=torch.float64), [None] * T
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            u = torch.where(a[t][:, None, None] == 0, torch.zeros_like(S[n]), a[t][:, None, None] * S[n])
            e = v[t] - (u * k[t][:, :, None]).sum(1)
            seen[t] = (S[n].clone(), u, e)
            S[n] = u + beta[t][:, None, None] * k[t][:, :, None] * e[:, None, :]
            y[t] = scale * (S[n] * q[t][:, :, None]).sum(1)
    return y, S, seen


def grad(q, k, v, g, beta, cu, dy, s0=None, ds=None, scale=1.0):
    T, H, dv = v.shape
    Hk, dk = q.shape[1], q.shape[2]
    seen = steps(q, k, v, g, beta, cu, s0, scale)[2]
    q, k, dy, beta = expand(q, H), expand(k, H), scale * dy.double(), beta.double()
    a = torch.ones(T, H, dtype=torch.float64) if g is None else torch.exp(g.double())
    R = torch.zeros(len(cu) - 1, H, dk, dv, dtype=torch.float64) if ds is None else ds.double().clone()
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros(T, H, dv, dtype=torch.float64)
    dg, db = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for n in range(len(cu) - 1):
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            before, u, e = seen[t]
            b = beta[t][:, None]
            S = u + b[:, :, None] * k[t][:, :, None] * e[:, None, :]
            dq[t] = (S * dy[t][:, None, :]).sum(-1)
            D = R[n] + q[t][:, :, None] * dy[t][:, None, :]
            db[t] = (D * k[t][:, :, None] * e[:, None, :]).sum((-1, -2))
            de = b * (D * k[t][:, :, None]).sum(1)
            dvv[t] = de
            dkk[t] = b * (D * e[:, None, :]).sum(-1) - (u * de[:, None, :]).sum(-1)
            U = D - k[t][:, :, None] * de[:, None, :]
            dg[t] = (U * u).sum((-1, -2))
            R[n] = U * a[t][:, None, None]
    fold = lambda x: x.view(T, Hk, H // Hk, dk).sum(2)  # noqa: E731
    return fold(dq), fold(dkk), dvv, None if g is None else dg, db, R
