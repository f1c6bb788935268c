"""Rotary positions with several axes, and the norm that keeps its inputs in 8 bits
with the gradient that reads them, on the GPU against plain forms in 64 bits; and
a mixer made of these and the gated delta rule, forwards and backwards."""
import math

import pytest
import torch

from tests import delta_ref as delta
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import gated_delta_rule_75_amd as m
    m.lib()
    return m


# ------------------------------------------------------------------ rotary positions
def rope_axes(x, pos, axis, freq, layout, inverse, m):
    """Pair by pair, from the definition."""
    x = x.double().clone()
    n = freq.numel()
    for i in range(n):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        ang = pos[int(axis[i])].double() * freq[i] * (-1 if inverse else 1)
        c, s = m * torch.cos(ang)[:, None], m * torch.sin(ang)[:, None]
        u, w = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,d,sections,order", [
    (1, 2, 1, 64, (8, 12, 12), "runs"), (65, 6, 2, 128, (16, 24, 24), "turns"), (333, 3, 0, 96, (5, 3), "turns"),
    (40, 1, 1, 66, (4, 0, 7, 1), "runs"), (2100, 2, 2, 64, (16, 16), "turns")], ids=str)
def test_axes(kda, T, Hq, Hk, d, sections, order, layout, dtype):
    gen = torch.Generator().manual_seed(T + d)
    n = sum(sections)
    q, k = (torch.randn(T, h, d, generator=gen).to(DT[dtype]) if h else None for h in (Hq, Hk))
    pos = torch.randint(-50, 1 << 20, (len(sections), T), generator=gen, dtype=torch.int32)
    axis = kda.rope_pair_axes(sections, order)
    freq, _ = kda.rope_frequencies(2 * n)
    for inverse, m in ((False, 1.0), (True, 1.25)):
        got = kda.rope_axes(q.cuda(), None if k is None else k.cuda(), pos.cuda(), axis.cuda(), freq.cuda(), layout=layout,
                            inverse=inverse, mscale=m)
        for name, x, y in (("q", q, got[0]), ("k", k, got[1])):
            if x is None:
                assert y is None
                continue
            ref.check(f"axes {dtype} {layout} {T} {sections} {order} {inverse} {name}", y,
                      rope_axes(x, pos, axis, freq, layout, inverse, m), ref.TOL[dtype])


def test_one_axis_is_rope(kda):
    """Axes that all have the same positions are rope, bit for bit; in place and at a stride too."""
    T, d = 70, 128
    x = torch.randn(T, 5, d, device="cuda").bfloat16()
    q, k = x[:, :4], x[:, 4:]
    pos = (torch.arange(T, device="cuda", dtype=torch.int32) * 1999)
    freq = kda.rope_frequencies(d)[0].cuda()
    axis = kda.rope_pair_axes((20, 30, 14), "turns").cuda()
    want = kda.rope(q, k, pos, freq)
    three = pos.expand(3, T).contiguous()
    got = kda.rope_axes(q, k, three, axis, freq)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    kda.rope_axes(q, k, three, axis, freq, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_axes_behind_the_last(kda):
    """A pair whose axis does not exist takes the last one."""
    q = torch.randn(9, 2, 64, device="cuda")
    pos = torch.randint(0, 1000, (2, 9), device="cuda", dtype=torch.int32)
    freq = kda.rope_frequencies(64)[0].cuda()
    axis = torch.tensor([0, 1, 2, 255] * 8, dtype=torch.uint8, device="cuda")
    a, _ = kda.rope_axes(q, None, pos, axis, freq)
    b, _ = kda.rope_axes(q, None, pos, axis.clamp(max=1), freq)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ 8 bits
def e4m3():
    """The 127 values from 0 to 448 by their codes."""
    v = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64)


def keep(x):
    """Codes and exponent bytes from the definition: blocks of 128, a power of two by trying them
    from above, each value to the nearest code, the even one at a tie."""
    x, table = x.double(), e4m3()
    D = x.shape[-1]
    codes, exps = torch.zeros(x.shape, dtype=torch.uint8), torch.zeros(*x.shape[:-1], -(-D // 128), dtype=torch.uint8)
    for b in range(exps.shape[-1]):
        u = x[..., 128 * b:128 * b + 128]
        top = torch.where(u.isnan(), torch.zeros_like(u), u.abs()).amax(-1)
        e = torch.full(top.shape, 121, dtype=torch.float64)
        for t in range(120, -127, -1):
            e = torch.where(top <= 448 * 2.0 ** t, torch.full_like(e, t), e)
        e = torch.where(top.isinf(), torch.full_like(e, 120), e)
        exps[..., b] = (e + 127).to(torch.uint8)
        a = u.abs() / torch.exp2(e)[..., None]
        hi = torch.searchsorted(table, a.nan_to_num(0, 0)).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        dl, dh = a - table[lo], table[hi] - a
        c = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        c = torch.where(a.isnan() | a.isinf(), torch.full_like(c, 127), c)
        codes[..., 128 * b:128 * b + 128] = (c + 128 * torch.signbit(u)).to(torch.uint8)
    return codes, exps


def stands_for(codes, exps):
    """The values of codes and exponent bytes."""
    c = codes.long()
    v = torch.cat([e4m3(), torch.tensor([math.nan], dtype=torch.float64)])[c % 128] * torch.where(c >= 128, -1.0, 1.0)
    e = exps.double().repeat_interleave(128, -1)[..., :codes.shape[-1]] - 127
    return v * torch.exp2(e)


def rows(T, H, D, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=gen) * torch.exp(2 * torch.randn(T, H, 1, generator=gen)) + 0.3
    return x.to(DT[dtype]), gen


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D", [(3, 2, 64), (5, 3, 128), (4, 1, 1), (3, 1, 129), (2, 2, 300), (3, 1, 1000), (2, 1, 2047),
                                   (2, 1, 5000), (1, 1, 16384), (33, 4, 80)], ids=str)
def test_kept_norm(kda, T, H, D, dtype):
    for kind, gated, biased in (("layer", True, True), ("rms", False, False), ("rms", True, False)):
        x, gen = rows(T, H, D, dtype, D)
        w, b = 1 + 0.2 * torch.randn(H, D, generator=gen), 0.2 * torch.randn(H, D, generator=gen) if biased else None
        z = torch.randn(T, H, D, generator=gen).to(DT[dtype]) if gated else None
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        y, mean, rstd, kept = kda.norm_fwd_kept(c(x), c(w), bias=c(b), z=c(z), kind=kind)
        plain = kda.norm_fwd(c(x), c(w), bias=c(b), z=c(z), kind=kind)
        name = f"kept {dtype} {kind} {T}x{H}x{D}"
        # the norm itself is the other call's, bit for bit
        assert torch.equal(y, plain[0]) and torch.equal(rstd, plain[2]) and (mean is None or torch.equal(mean, plain[1]))
        for t, v8, e8 in ((x, kept[0], kept[1]), (z, kept[2], kept[3])):
            if t is None:
                assert v8 is None and e8 is None
                continue
            codes, exps = keep(t)
            assert torch.equal(e8.cpu(), exps), name
            assert torch.equal(v8.view(torch.uint8).cpu(), codes), name
        # the gradient at the kept values, with the statistics of the full ones
        dy = torch.randn(T, H, D, generator=gen).to(DT[dtype])
        got = kda.norm_bwd_kept(c(dy), kept, c(w), mean, rstd, bias=c(b), kind=kind)
        xv = stands_for(kept[0].view(torch.uint8).cpu(), kept[1].cpu())
        r = rstd.double().cpu()[..., None]
        h = (xv - (mean.double().cpu()[..., None] if mean is not None else 0)) * r
        g, dz = dy.double(), None
        if gated:
            s = 1 / (1 + torch.exp(-stands_for(kept[2].view(torch.uint8).cpu(), kept[3].cpu())))
            dz = g * (h * w.double() + (0 if b is None else b.double())) * s * (1 - s)
            g = g * s
        e = g * w.double()
        dx = r * (e - h * (e * h).mean(-1, keepdim=True) - (e.mean(-1, keepdim=True) if kind == "layer" else 0))
        tol = 2 * ref.TOL[dtype] if dtype == "f32" else ref.TOL[dtype]
        if D > 1:            # of one element the layer norm's gradient is a difference of equal terms
            ref.check(name + " dx", got[0], dx, tol)
        ref.check(name + " dw", got[1], (g * h).sum(0), ref.TOL["f32"])
        if biased:
            ref.check(name + " db", got[2], g.sum(0), ref.TOL["f32"])
        if gated:
            ref.check(name + " dz", got[3], dz, ref.TOL[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_kept_extremes(kda, dtype):
    """Blocks of zeros, of the smallest and largest values, borders of a power of two, ties, NaN and infinities."""
    x = torch.zeros(12, 1, 256)
    x[1] = 1e-45
    x[2] = torch.linspace(-3e38, 3e38, 256)
    x[3, :, 0], x[3, :, 1] = 448, 447
    x[4, :, 0], x[4, :, 130] = 450, 224
    x[5] = e4m3().float().repeat(3)[:256] * 2.0 ** -30
    x[6] = torch.arange(256) * 0.5 + 16.5
    x[7, :, 3], x[7, :, 4] = math.nan, 5.0
    x[8, :, 200], x[8, :, 201] = math.inf, 7.0
    x[9, :, 5] = -math.inf
    x[10] = -0.0
    x[11] = torch.linspace(1e-41, 1e-37, 256)
    x = x.to(DT[dtype])
    _, _, _, (v8, e8, _, _) = kda.norm_fwd_kept(x.cuda(), torch.ones(1, 256, device="cuda"), kind="rms")
    codes, exps = keep(x)
    assert torch.equal(e8.cpu(), exps)
    got, nan = v8.view(torch.uint8).cpu(), (codes % 128) == 127
    assert torch.equal(got % 128 == 127, nan)
    assert torch.equal(got[~nan], codes[~nan])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_8_bits_hold(kda, dtype):
    """Where keeping loses nothing the gradient is norm_bwd's, bit for bit, and so is one over rows in
    other places: recorded in a graph, and on another stream."""
    gen = torch.Generator().manual_seed(4)
    v = e4m3()[torch.randint(60, 120, (50, 3, 200), generator=gen)]
    x = (v * (torch.randint(0, 2, v.shape, generator=gen) * 2 - 1)).to(DT[dtype]).cuda()
    z = torch.randint(-15, 16, v.shape, generator=gen).to(DT[dtype]).cuda()
    dy, w = torch.randn(v.shape, generator=gen).to(DT[dtype]).cuda(), torch.randn(3, 200, generator=gen).cuda()
    y, mean, rstd, kept = kda.norm_fwd_kept(x, w, z=z)
    want = kda.norm_bwd(dy, x, w, mean, rstd, z=z)
    got = kda.norm_bwd_kept(dy, kept, w, mean, rstd)
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = kda.norm_bwd_kept(dy, kda.norm_fwd_kept(x, w, z=z)[3], w, mean, rstd)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(again, want):
        assert a is None or torch.equal(a, b)


# ------------------------------------------------------------------ together
def test_a_mixer(kda):
    """Rotary positions of an image's tokens, the gated delta rule over two packed sequences, the gated norm
    that keeps its inputs; then back through all three, against the same chain in 64 bits."""
    gen = torch.Generator().manual_seed(12)
    lens, H, Hk, d = [70, 150], 4, 2, 64
    T, cu = sum(lens), [0, 70, 220]
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(T, Hk, d), dim=-1) for _ in range(2))
    v, z, dout = r(T, H, d), r(T, H, d), r(T, H, d)
    g, beta = -torch.rand(T, H, generator=gen) * 0.2, torch.rand(T, H, generator=gen)
    w = 1 + 0.2 * r(H, d)
    pos = torch.stack([torch.arange(T) // 16, torch.arange(T) % 16]).int()
    axis, freq = kda.rope_pair_axes((16, 16), "turns"), kda.rope_frequencies(d)[0]
    c = lambda t: t.cuda()  # noqa: E731
    cu_t = torch.tensor(cu, dtype=torch.int32).cuda()

    qr, kr = kda.rope_axes(c(q), c(k), c(pos), c(axis), c(freq))
    y, _ = kda.gdr_fwd(qr, kr, c(v), c(g), c(beta), cu_seqlens=cu_t)
    out, mean, rstd, kept = kda.norm_fwd_kept(y, c(w), z=c(z), kind="rms")
    dy, dw, _, dz = kda.norm_bwd_kept(c(dout), kept, c(w), mean, rstd, kind="rms")
    dqr, dkr, dv, dg, db, _ = kda.gdr_bwd(qr, kr, c(v), c(g), c(beta), dy, cu_seqlens=cu_t)
    dq, dk = kda.rope_axes(dqr, dkr, c(pos), c(axis), c(freq), inverse=True)

    qw, kw = (rope_axes(x, pos, axis, freq, "half", False, 1.0) for x in (q, k))
    yw, _, _ = delta.steps(qw, kw, v, g, beta, cu, None, 1.0)
    ow, _, rw = ref.norm(yw, w, None, z, 1e-5, "rms")
    ref.check("mixer out", out, ow, ref.TOL["f32"])
    h = stands_for(kept[0].view(torch.uint8).cpu(), kept[1].cpu()) * rw[..., None]
    s = 1 / (1 + torch.exp(-stands_for(kept[2].view(torch.uint8).cpu(), kept[3].cpu())))
    e = dout.double() * s * w.double()
    dyw = rw[..., None] * (e - h * (e * h).mean(-1, keepdim=True))
    ref.check("mixer dz", dz, dout.double() * h * w.double() * s * (1 - s), ref.TOL["f32"])
    ref.check("mixer dw", dw, (dout.double() * s * h).sum(0), ref.TOL["f32"])
    want = delta.grad(qw, kw, v, g, beta, cu, dyw)
    # errors of the two operators before add to the gradient's own
    for name, a, b in zip(("dv", "dg", "dbeta"), (dv, dg, db), want[2:]):
        ref.check("mixer " + name, a, b, 2 * delta.TOL_DG)
    for name, a, b in zip(("dq", "dk"), (dq, dk), want):
        ref.check("mixer " + name, a, rope_axes(b, pos, axis, freq, "half", True, 1.0), 2 * delta.TOL_DG)
