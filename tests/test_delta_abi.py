"""The gated delta rule, rotary axes and the kept norm without a GPU: arguments are
refused before anything is launched, sizes of workspaces, the axes of pairs; and
the gradient that the GPU tests hold the kernels to, against differences."""
import pytest
import torch

import gated_delta_rule_75_amd as kda
from tests import delta_ref as delta

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
BF16, F32 = kda.KDA_BF16, kda.KDA_F32
A = 1 << 20                                # a fake, aligned, never dereferenced address


def fwd(name="kda_gdr_fwd", dt=BF16, H=4, Hk=2, dk=128, dv=64, N=1, T=1000, cu=None, q=A, qs=256, k=A, ks=256, v=A, vs=256,
        g=A, beta=A, s0=None, sf=None, y=A, ws=A, wsb=1 << 40):
    return getattr(kda.lib(), name)(dt, H, Hk, dk, dv, 1.0, N, T, cu, q, qs, k, ks, v, vs, g, beta, s0, sf, y, ws, wsb, None)


def bwd(name="kda_gdr_bwd", dt=BF16, H=4, Hk=2, dk=128, dv=64, N=1, T=1000, cu=None, q=A, qs=256, k=A, ks=256, v=A, vs=256,
        g=A, beta=A, s0=None, dy=A, ds=None, dq=A, dko=A, dvo=A, dg=A, db=A, ds0=None, ws=A, wsb=1 << 40):
    return getattr(kda.lib(), name)(dt, H, Hk, dk, dv, 1.0, N, T, cu, q, qs, k, ks, v, vs, g, beta, s0, dy, ds, dq, dko, dvo,
                                    dg, db, ds0, ws, wsb, None)


@pytest.mark.parametrize("call,name", [(fwd, "kda_gdr_fwd"), (fwd, "kda_gdr_fwd_padded"), (bwd, "kda_gdr_bwd"),
                                       (bwd, "kda_gdr_bwd_padded")])
def test_gdr_refuses(call, name):
    for bad in (dict(dt=3), dict(H=0), dict(Hk=0), dict(Hk=3), dict(N=0), dict(T=-1), dict(N=2), dict(q=None),
                dict(k=None), dict(v=None), dict(beta=None), dict(q=A + 8), dict(v=A + 2), dict(qs=255), dict(qs=260),
                dict(ks=128), dict(vs=0), dict(s0=A + 8), dict(ws=None), dict(ws=A + 128), dict(T=1 << 31),
                dict(N=1 << 21, cu=A), dict(T=1 << 28), dict(cu=A + 2), dict(g=A + 2), dict(beta=A + 1),
                dict(qs=1 << 24)):
        assert call(name, **bad) == INVALID, bad
    for bad in (dict(dk=96), dict(dv=256), dict(dk=0)):
        assert call(name, **bad) == UNSUPPORTED, bad
    assert call(name, wsb=1000) == WS_SMALL


def test_gdr_refuses_outputs():
    for bad in (dict(y=None), dict(y=A + 2), dict(sf=A + 4)):
        assert fwd(**bad) == INVALID, bad
    for bad in (dict(dy=None), dict(dq=None), dict(dko=None), dict(dvo=None), dict(dg=None), dict(g=None), dict(db=None),
                dict(dy=A + 8), dict(ds=A + 4), dict(ds0=A + 4), dict(db=A + 2)):
        assert bwd(**bad) == INVALID, bad        # dg is given exactly where g is


def test_gdr_decode_refuses():
    def dec(dt=BF16, N=4, H=4, Hk=2, dk=128, dv=64, q=A, qs=256, k=A, v=A, g=A, beta=A, state=A, y=A):
        return kda.lib().kda_gdr_decode_step(dt, N, H, Hk, dk, dv, 1.0, q, qs, k, 256, v, 256, g, beta, state, y, None)
    for bad in (dict(dt=9), dict(N=-1), dict(H=0), dict(Hk=3), dict(q=None), dict(k=None), dict(v=None), dict(beta=None),
                dict(state=None), dict(y=None), dict(qs=200), dict(q=A + 8), dict(state=A + 8), dict(y=A + 2),
                dict(N=1 << 22)):
        assert dec(**bad) == INVALID, bad
    assert dec(dk=32) == UNSUPPORTED
    assert dec(N=0) == OK                       # nothing launched


def test_gdr_workspaces():
    f, b = kda.gdr_fwd_workspace_size, kda.gdr_bwd_workspace_size
    assert f(BF16, 4, 4, 128, 128, 1, 0) == b(BF16, 4, 4, 128, 128, 1, 0) == 256
    assert f(BF16, 4, 3, 128, 128, 1, 8192) == f(7, 4, 4, 128, 128, 1, 8192) == f(BF16, 4, 4, 96, 128, 1, 8192) == 0
    assert b(F32, 0, 1, 64, 64, 1, 10) == b(BF16, 96, 96, 128, 128, 1, 1 << 30) == 0
    # every chunk of a head: two 64 x 64 matrices; backwards two states, two blocks of rows
    chunks = 8192 // 64 + 1
    assert f(BF16, 4, 2, 128, 64, 1, 8192) >= chunks * 4 * 2 * 64 * 64 * 4 // 2
    assert b(BF16, 4, 2, 128, 64, 1, 8192) >= chunks * 4 * (2 * 128 * 64 + 2 * 64 * 64) * 4
    # from 257 sequences on, a table of their first chunks (so few are not cut into segments)
    at = [f(BF16, 1, 1, 64, 64, n, 1900) for n in (255, 256, 257)]
    assert at[2] - at[1] - (at[1] - at[0]) == (258 * 4 + 255) // 256 * 256
    # segments: their transitions and states beside that, up to 256 sequences
    m = [f(BF16, 1, 1, 64, 64, n, 100000) for n in (255, 256, 257)]
    assert m[1] - m[2] > 256 * 2 * 64 * 64 * 4 and m[1] > m[0]


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_gdr_binding_refuses():
    q, v, g = z(8, 2, 64), z(8, 4, 128), z(8, 4, dtype=torch.float32)
    for exc, args, kw in (
            (ValueError, (q, q, v, g, g), {}),                                     # not on the GPU
            (TypeError, (q, q.float(), v, g, g), {}), (TypeError, (q, q, v, g.double(), g), {}),
            (TypeError, (q, q, v, g, g.bfloat16()), {}), (TypeError, (q, q, v, None, g.bfloat16()), {}),
            (TypeError, (q.half(), q.half(), v.half(), g, g), {}), (ValueError, (q, q, v, g, None), {}),
            (ValueError, (q, z(8, 1, 64), v, g, g), {}), (ValueError, (q, q, z(7, 4, 128), g, g), {}),
            (ValueError, (q, q, z(8, 3, 128), g, g), {}), (ValueError, (q, q, v, g[:, :2], g), {}),
            (ValueError, (q, q, v, g[0], g), {}), (ValueError, (q, q, v, g, g[0]), {}),
            (ValueError, (q, q, v, g, z(4, 8, dtype=torch.float32).t()), {}),
            (ValueError, (q, q, v, g, g), dict(initial_state=z(2, 4, 64, 128, dtype=torch.float32))),
            (TypeError, (q, q, v, g, g), dict(y=z(8, 4, 128, dtype=torch.float32))),
            (ValueError, (q, q, v, g, g), dict(y=z(8, 4, 64))),
            (TypeError, (q, q, v, g, g), dict(cu_seqlens=torch.tensor([0, 8]))),
            (TypeError, (q, q, v, g, g), dict(workspace=z(100))),
            (ValueError, (z(8, 64, 2).transpose(1, 2), q, v, g, g), {})):          # heads not contiguous
        with pytest.raises(exc):
            kda.gdr_fwd(*args, **kw)
    with pytest.raises(ValueError):
        kda.gdr_bwd(q, q, v, g, g, z(8, 4, 64))
    with pytest.raises(ValueError):
        kda.gdr_decode_step(q, q, v, g, g, None)
    with pytest.raises(ValueError):
        kda.gdr_decode_step(q, q, v, g, g, z(8, 4, 128, 64, dtype=torch.float32))


def test_axes_refuse():
    def call(dt=BF16, T=4, Hq=2, Hk=1, d=64, rot=32, layout=0, axes=3, pos=A, ax=A, f=A, q=A, qs=128, k=A, ks=64,
             qo=A + 4096, qos=128, ko=A + 8192, kos=64):
        return kda.lib().kda_rope_axes(dt, T, Hq, Hk, d, rot, layout, 0, 1.0, axes, pos, ax, f, q, qs, k, ks, qo, qos, ko,
                                       kos, None)
    for bad in (dict(dt=4), dict(T=-1), dict(Hq=0), dict(rot=0), dict(rot=66), dict(layout=2), dict(pos=None),
                dict(ax=None), dict(axes=0), dict(axes=256), dict(f=None), dict(q=None), dict(ko=None), dict(qs=127),
                dict(q=A + 1), dict(pos=A + 2), dict(qo=A, qos=256)):
        assert call(**bad) == INVALID, bad
    assert call(T=0) == OK
    q, pos, fr = z(8, 2, 64), torch.zeros(2, 8, dtype=torch.int32), torch.zeros(16, dtype=torch.float64)
    ax = torch.zeros(16, dtype=torch.uint8)
    for exc, args in ((ValueError, (q, q, pos, ax, fr)), (ValueError, (q, q, pos[0], ax, fr)),
                      (ValueError, (q, q, pos, None, fr)), (TypeError, (q, q, pos, ax.int(), fr)),
                      (ValueError, (q, q, pos, ax[:15], fr)), (ValueError, (q, q, pos[:, :7], ax, fr)),
                      (TypeError, (q, q, pos.long(), ax, fr))):
        with pytest.raises(exc):
            kda.rope_axes(*args)


def test_pair_axes():
    assert kda.rope_pair_axes((2, 3, 1)).tolist() == [0, 0, 1, 1, 1, 2]
    assert kda.rope_pair_axes((2, 3, 1), "turns").tolist() == [0, 1, 2, 0, 1, 1]
    assert kda.rope_pair_axes((0, 2), "turns").tolist() == [1, 1]
    for bad in ((), (0, 0), (-1, 4), (513,), (300, 300)):
        with pytest.raises(kda.KDAError):
            kda.rope_pair_axes(bad)
    with pytest.raises(ValueError):
        kda.rope_pair_axes((1, 1), "mixed")


def test_kept_norm_refuses():
    L = kda.lib()

    def f(dt=BF16, kind=0, T=4, H=2, D=64, eps=1e-5, x=A, w=A, b=None, z=None, y=A, mean=A, rstd=A, x8=A, xe=A, z8=None,
          ze=None):
        return L.kda_norm_fwd_kept(dt, kind, T, H, D, eps, x, w, b, z, y, mean, rstd, x8, xe, z8, ze, None)

    def g(dt=BF16, kind=0, T=4, H=2, D=64, x8=A, xe=A, w=A, b=None, z8=None, ze=None, mean=A, rstd=A, dy=A, dx=A, dw=A,
          db=None, dz=None, ws=A, wsb=1 << 30):
        return L.kda_norm_bwd_kept(dt, kind, T, H, D, x8, xe, w, b, z8, ze, mean, rstd, dy, dx, dw, db, dz, ws, wsb, None)
    for bad in (dict(dt=5), dict(kind=2), dict(T=-1), dict(H=0), dict(D=0), dict(eps=-1.0), dict(x=None), dict(w=None),
                dict(y=None), dict(kind=1), dict(x=A + 1), dict(x8=None), dict(xe=None), dict(z=A), dict(z8=A),
                dict(ze=A), dict(z=A, z8=A), dict(z8=A, ze=A)):
        assert f(**bad) == INVALID, bad
    assert f(D=16385) == UNSUPPORTED
    assert f(T=0, x8=None, xe=None) == OK
    for bad in (dict(dt=5), dict(kind=3), dict(x8=None), dict(xe=None), dict(w=None), dict(mean=None), dict(rstd=None),
                dict(dy=None), dict(dx=None), dict(dw=None), dict(z8=A, dz=A), dict(z8=A, ze=A), dict(dz=A), dict(kind=1),
                dict(ws=None), dict(ws=A + 16)):
        assert g(**bad) == INVALID, bad
    assert g(D=20000) == UNSUPPORTED
    assert g(wsb=100) == WS_SMALL
    x, w, m = z(8, 2, 200), z(2, 200, dtype=torch.float32), z(8, 2, dtype=torch.float32)
    with pytest.raises(ValueError):
        kda.norm_fwd_kept(x, w)                                                    # not on the GPU
    x8, e = torch.zeros(8, 2, 200, dtype=torch.float8_e4m3fn), torch.zeros(8, 2, 2, dtype=torch.uint8)
    for exc, kept in ((ValueError, (x8, e, None, None)), (ValueError, (x8, None, None, None)),
                      (ValueError, (x8, e, x8, None)), (ValueError, (x8, e[..., :1], None, None)),
                      (TypeError, (x8.view(torch.uint8), e, None, None)), (TypeError, (x8, e.int(), None, None)),
                      (ValueError, (x8[..., :100], e, None, None))):
        with pytest.raises(exc):
            kda.norm_bwd_kept(x, kept, w, m, m)
    with pytest.raises(ValueError):
        kda.norm_bwd_kept(x, (x8, e, None, None), w, None, m)


def test_the_reference_gradient_by_differences():
    gen = torch.Generator().manual_seed(2)
    T, Hk, H, dk, dv, cu = 9, 1, 2, 3, 4, [0, 4, 4, 9]
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x = dict(q=r(T, Hk, dk), k=0.5 * r(T, Hk, dk), v=r(T, H, dv), g=-torch.rand(T, H, generator=gen, dtype=torch.float64),
             beta=torch.rand(T, H, generator=gen, dtype=torch.float64), s0=r(3, H, dk, dv))
    dy, ds = r(T, H, dv), r(3, H, dk, dv)

    def loss(x):
        y, S, _ = delta.steps(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, x["s0"], 0.7)
        return float((y * dy).sum() + (S * ds).sum())
    got = delta.grad(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, dy, x["s0"], ds, 0.7)
    h = 1e-5
    for name, d in zip(("q", "k", "v", "g", "beta", "s0"), got):
        for _ in range(4):
            way = r(*x[name].shape)
            up, down = (loss({**x, name: x[name] + s * h * way}) for s in (1, -1))
            want = float((d * way).sum())
            # central differences: an error of h^2 times the third derivative, and 1e-16 / h of the loss
            assert abs((up - down) / (2 * h) - want) <= 1e-7 * (1 + abs(want)), name
