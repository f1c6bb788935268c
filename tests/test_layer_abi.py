"""The layer operators without a GPU: arguments are refused before anything is
launched, sizes of workspaces, and the rotary frequencies (host only)."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_75_amd as kda

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
BF16, F32 = kda.KDA_BF16, kda.KDA_F32
A = 1 << 20                                # a fake, aligned, never dereferenced address


@pytest.fixture(scope="module")
def L():
    return kda.lib()


def _fwd(L, dt=BF16, H=4, Hk=2, dk=128, dv=64, N=1, T=1000, cu=None, q=A, qs=256, k=A, ks=256, v=A, vs=256, g=A,
         s0=None, sf=None, y=A, ws=A, wsb=1 << 40):
    return L.kda_linattn_fwd(dt, H, Hk, dk, dv, 1.0, N, T, cu, q, qs, k, ks, v, vs, g, 1, s0, sf, y, ws, wsb, None)


def _bwd(L, dt=BF16, H=4, Hk=2, dk=128, dv=64, N=1, T=1000, cu=None, q=A, qs=256, k=A, ks=256, v=A, vs=256, g=A,
         s0=None, dy=A, ds=None, dq=A, dko=A, dvo=A, dg=A, ds0=None, ws=A, wsb=1 << 40):
    return L.kda_linattn_bwd(dt, H, Hk, dk, dv, 1.0, N, T, cu, q, qs, k, ks, v, vs, g, 1, s0, dy, ds, dq, dko, dvo,
                             dg, ds0, ws, wsb, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_linattn_refuses(L, call):
    for bad in (dict(dt=3), dict(H=0), dict(Hk=0), dict(Hk=3), dict(N=0), dict(T=-1), dict(N=2), dict(q=None),
                dict(k=None), dict(v=None), dict(g=None), dict(q=A + 8), dict(v=A + 2), dict(qs=255), dict(qs=260),
                dict(ks=128), dict(vs=0), dict(s0=A + 8), dict(ws=None), dict(ws=A + 128), dict(T=1 << 31),
                dict(N=1 << 21, cu=A), dict(cu=A + 2), dict(g=A + 2)):
        assert call(L, **bad) == INVALID, bad
    for bad in (dict(dk=96), dict(dv=256), dict(dk=0)):
        assert call(L, **bad) == UNSUPPORTED, bad
    assert call(L, wsb=1000) == WS_SMALL


def test_linattn_refuses_outputs(L):
    for bad in (dict(y=None), dict(y=A + 2), dict(sf=A + 4)):
        assert _fwd(L, **bad) == INVALID, bad
    for bad in (dict(dy=None), dict(dq=None), dict(dko=None), dict(dvo=None), dict(dg=None), dict(dy=A + 8),
                dict(ds=A + 4), dict(ds0=A + 4)):
        assert _bwd(L, **bad) == INVALID, bad


def test_linattn_decode_refuses(L):
    def dec(dt=BF16, N=4, H=4, Hk=2, dk=128, dv=64, q=A, qs=256, k=A, v=A, g=A, state=A, y=A):
        return L.kda_linattn_decode_step(dt, N, H, Hk, dk, dv, 1.0, q, qs, k, 256, v, 256, g, 1, state, y, None)
    for bad in (dict(dt=9), dict(N=-1), dict(H=0), dict(Hk=3), dict(q=None), dict(k=None), dict(v=None), dict(g=None),
                dict(state=None), dict(y=None), dict(qs=200), dict(q=A + 8), dict(state=A + 8), dict(y=A + 2)):
        assert dec(**bad) == INVALID, bad
    assert dec(dk=32) == UNSUPPORTED
    assert dec(N=0) == OK                       # nothing launched


def test_linattn_workspaces(L):
    size = kda.linattn_fwd_workspace_size
    assert size(BF16, 4, 4, 128, 128, 1, 64) == 256             # one block a sequence: nothing kept
    # 8192 tokens of 4 heads: blocks of 64 tokens, a state and a decay for each and head
    blocks = 8192 // 64 + 1
    assert size(BF16, 4, 4, 128, 128, 1, 8192) == blocks * 4 * 128 * 128 * 4 + (blocks * 4 * 4 + 255) // 256 * 256
    assert size(BF16, 4, 3, 128, 128, 1, 8192) == 0
    assert size(7, 4, 4, 128, 128, 1, 8192) == 0
    assert size(BF16, 4, 4, 96, 128, 1, 8192) == 0
    back = kda.linattn_bwd_workspace_size
    assert back(BF16, 4, 2, 64, 64, 1, 8192) >= 2 * blocks * 4 * 64 * 64 * 4 + 8192 * 4 * 64 * 4
    assert back(F32, 0, 1, 64, 64, 1, 10) == 0


def _rope(L, dt=BF16, T=4, Hq=2, Hk=1, d=64, rot=32, layout=0, pos=A, f=A, q=A, qs=128, k=A, ks=64, qo=A + 4096,
          qos=128, ko=A + 8192, kos=64):
    return L.kda_rope(dt, T, Hq, Hk, d, rot, layout, 0, 1.0, pos, f, q, qs, k, ks, qo, qos, ko, kos, None)


def test_rope_refuses(L):
    for bad in (dict(dt=4), dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(d=0), dict(rot=0), dict(rot=31), dict(rot=66),
                dict(layout=2), dict(pos=None), dict(f=None), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None),
                dict(qs=127), dict(kos=10), dict(q=A + 1), dict(f=A + 4), dict(pos=A + 2),
                dict(qo=A, qos=256)):           # in place at another stride
        assert _rope(L, **bad) == INVALID, bad
    assert _rope(L, d=2048, qs=4096, qos=4096, ks=2048, kos=2048) == UNSUPPORTED
    assert _rope(L, T=0) == OK


def test_norm_refuses(L):
    def fwd(dt=BF16, kind=0, T=4, H=2, D=64, eps=1e-5, x=A, w=A, b=None, z=None, y=A, mean=A, rstd=A):
        return L.kda_norm_fwd(dt, kind, T, H, D, eps, x, w, b, z, y, mean, rstd, None)

    def bwd(dt=BF16, kind=0, T=4, H=2, D=64, x=A, w=A, b=None, z=None, mean=A, rstd=A, dy=A, dx=A, dw=A, db=None,
            dz=None, ws=A, wsb=1 << 30):
        return L.kda_norm_bwd(dt, kind, T, H, D, x, w, b, z, mean, rstd, dy, dx, dw, db, dz, ws, wsb, None)
    for bad in (dict(dt=5), dict(kind=2), dict(T=-1), dict(H=0), dict(D=0), dict(eps=-1.0), dict(eps=math.nan),
                dict(x=None), dict(w=None), dict(y=None), dict(kind=1), dict(x=A + 1), dict(w=A + 2)):
        assert fwd(**bad) == INVALID, bad        # kind 1 (rms) takes no mean
    assert fwd(D=16385) == UNSUPPORTED
    assert fwd(T=0) == OK
    for bad in (dict(dt=5), dict(kind=3), dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(dy=None),
                dict(dx=None), dict(dw=None), dict(z=A), dict(dz=A), dict(kind=1), dict(ws=None), dict(ws=A + 16)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(D=20000) == UNSUPPORTED
    assert bwd(wsb=100) == WS_SMALL
    assert kda.norm_bwd_workspace_size(BF16, 4, 2, 64) >= 2 * 8 * 64 * 4
    assert kda.norm_bwd_workspace_size(BF16, 4, 2, 20000) == 0


def test_frequencies():
    """The published formulas, written apart from the library's."""
    f, m = kda.rope_frequencies(64, base=1e4)
    assert m == 1.0 and f.dtype == torch.float64
    for i in range(32):
        assert f[i] == pytest.approx(1e4 ** (-i / 32), rel=1e-14)
    lin, m = kda.rope_frequencies(64, scaling="linear", factor=8.0)
    assert m == 1.0 and torch.allclose(lin * 8, f, rtol=1e-14, atol=0)
    # the base is stretched so that the slowest pair turns 1 / factor as fast, the fastest as before
    ntk, m = kda.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert m == 1.0 and ntk[0] == 1.0 and float(ntk[31]) == pytest.approx(float(f[31]) / 8, rel=1e-12)
    yarn, m = kda.rope_frequencies(64, scaling="yarn", factor=8.0, trained_len=4096)
    assert m == pytest.approx(0.1 * math.log(8) + 1, rel=1e-6)
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(yarn[turns > 40], f[turns > 40])
    assert torch.allclose(yarn[turns < 0.7] * 8, f[turns < 0.7], rtol=1e-13, atol=0)
    assert bool((yarn <= f).all()) and bool((yarn * 8 >= f * (1 - 1e-12)).all())


def test_frequencies_refuse():
    for bad in (dict(rot=0), dict(rot=7), dict(rot=64, base=1.0), dict(rot=64, base=math.inf),
                dict(rot=64, scaling="linear", factor=0.5), dict(rot=2, scaling="ntk", factor=2.0),
                dict(rot=64, scaling="yarn", factor=2.0, trained_len=0)):
        with pytest.raises(kda.KDAError):
            kda.rope_frequencies(**bad)
    with pytest.raises(ValueError):
        kda.rope_frequencies(64, scaling="other")


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses():
    q, v, g = z(8, 2, 64), z(8, 4, 128), z(8, 4, dtype=torch.float32)
    f = kda.linattn_fwd
    for exc, args, kw in (
            (ValueError, (q, q, v, g), {}),                                     # not on the GPU
            (TypeError, (q, q.float(), v, g), {}), (TypeError, (q, q, v, g.double()), {}),
            (TypeError, (q.half(), q.half(), v.half(), g), {}),
            (ValueError, (q, z(8, 1, 64), v, g), {}), (ValueError, (q, q, z(7, 4, 128), g), {}),
            (ValueError, (q, q, z(8, 3, 128), g), {}), (ValueError, (q, q, v, g[:, :2]), {}),
            (ValueError, (q, q, v, g), dict(initial_state=z(2, 4, 64, 128, dtype=torch.float32))),
            (TypeError, (q, q, v, g), dict(y=z(8, 4, 128, dtype=torch.float32))),
            (ValueError, (q, q, v, g), dict(y=z(8, 4, 64))),
            (TypeError, (q, q, v, g), dict(cu_seqlens=torch.tensor([0, 8]))),
            (ValueError, (q, q, v, g), dict(cu_seqlens=torch.tensor([0], dtype=torch.int32))),
            (TypeError, (q, q, v, g), dict(workspace=z(100))),
            (ValueError, (z(8, 64, 2).transpose(1, 2), q, v, g), {}),           # heads not contiguous
            (ValueError, (z(1, 2, 64).expand(8, 2, 64), q, v, g), {})):         # tokens overlap
        with pytest.raises(exc):
            f(*args, **kw)
    with pytest.raises(ValueError):
        kda.linattn_bwd(q, q, v, g, z(8, 4, 64))
    with pytest.raises(ValueError):
        kda.linattn_decode_step(q, q, v, g, None)
    with pytest.raises(ValueError):
        kda.linattn_decode_step(q, q, v, g, z(8, 4, 128, 64, dtype=torch.float32))
    pos, fr = torch.zeros(8, dtype=torch.int32), torch.zeros(16, dtype=torch.float64)
    for exc, args, kw in (
            (ValueError, (q, q, pos, fr), {}), (TypeError, (q, q, pos.long(), fr), {}),
            (TypeError, (q, q, pos, fr.float()), {}), (ValueError, (q, q, pos[:7], fr), {}),
            (ValueError, (q, z(8, 2, 32), pos, fr), {}), (ValueError, (q, q, pos, fr), dict(layout="full")),
            (ValueError, (q, None, pos, fr), dict(k_out=q))):
        with pytest.raises(exc):
            kda.rope(*args, **kw)
    x, w, m = z(8, 2, 64), z(2, 64, dtype=torch.float32), z(8, 2, dtype=torch.float32)
    for exc, args, kw in (
            (ValueError, (x, w), {}), (TypeError, (x, w.bfloat16()), {}), (ValueError, (x, w[:1]), {}),
            (ValueError, (x, None), {}), (ValueError, (x, w), dict(kind="group")),
            (ValueError, (x, w), dict(z=z(8, 2, 63))), (TypeError, (x, w), dict(y=x.float())),
            (ValueError, (x[:, :, ::2], w[:, ::2]), {})):
        with pytest.raises(exc):
            kda.norm_fwd(*args, **kw)
    for args, kw in (((x, x, w, None, m), {}), ((x, x, w, m, m), dict(kind="rms")), ((x, x, w, m, None), {}),
                     ((x, x, w, m, m), {})):
        with pytest.raises(ValueError):
            kda.norm_bwd(*args, **kw)
