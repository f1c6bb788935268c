"""Rotary positions and the gated norm with its gradient on the GPU, against
their 64-bit definitions, and a layer of them around linear attention."""
import pytest
import torch

from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import gated_delta_rule_75_amd as m
    m.lib()
    return m


def randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen).to(dtype)


# elementwise: one rounding of an fp32 value with an error of a few 2^-24
EXACT = {"bf16": 2.0 ** -8, "f32": 1e-6}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(1, 1, 1, 64, 64), (129, 12, 4, 64, 64), (77, 4, 2, 128, 64),
                                           (5, 3, 1, 96, 48), (33, 2, 2, 80, 6), (17, 3, 2, 33, 10), (9, 5, 0, 64, 32),
                                           (5000, 2, 1, 64, 32)])
def test_rope(kda, T, Hq, Hk, d, rot, layout, dtype):
    gen = torch.Generator().manual_seed(T + d)
    q = randn(gen, T, Hq, d, dtype=DT[dtype])
    k = randn(gen, T, Hk, d, dtype=DT[dtype]) if Hk else None
    pos = torch.randint(-5, 1 << 21, (T,), generator=gen, dtype=torch.int32)
    freq, m = kda.rope_frequencies(rot, scaling="yarn", factor=8.0)
    f = freq.cuda()
    for inverse in (False, True):
        qo, ko = kda.rope(q.cuda(), None if k is None else k.cuda(), pos.cuda(), f, layout=layout, inverse=inverse,
                          mscale=m)
        for name, a, b in (("q", qo, q), ("k", ko, k)):
            if b is None:
                assert a is None
                continue
            ref.check(f"rope {dtype} {layout} {T}x{d}/{rot} {name}", a, ref.rope(b, pos, freq, layout, inverse, m),
                      EXACT[dtype])
            assert torch.equal(a[..., rot:].cpu(), b[..., rot:])


def test_rope_in_place_on_slices_and_back(kda):
    """In place on slices of a projection; the channels around stay, and turning
    back (m = 1) restores q and k."""
    T, H, Hk, d = 65, 4, 2, 64
    gen = torch.Generator().manual_seed(3)
    buf = randn(gen, T, (H + 2 * Hk) * d).cuda()
    old = buf.clone()
    q, k = buf[:, :H * d].unflatten(1, (H, d)), buf[:, H * d:(H + Hk) * d].unflatten(1, (Hk, d))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 7
    f = kda.rope_frequencies(32)[0].cuda()
    want = kda.rope(q, k, pos, f)
    got = kda.rope(q, k, pos, f, q_out=q, k_out=k)
    assert got[0] is q
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, (H + Hk) * d:], old[:, (H + Hk) * d:])
    kda.rope(q, k, pos, f, inverse=True, q_out=q, k_out=k)
    # two turns of an fp32 value: four products and sums, each within 2^-24
    assert float((buf - old).abs().max()) <= 8 * 2.0 ** -24 * float(old.abs().max()) * 2


def test_rope_no_tokens(kda):
    q = torch.zeros(0, 2, 64, device="cuda")
    out, _ = kda.rope(q, None, torch.zeros(0, dtype=torch.int32, device="cuda"), kda.rope_frequencies(64)[0].cuda())
    assert out.shape == (0, 2, 64)


NORM_SHAPES = [(1, 1, 1), (3, 1, 33), (7, 4, 64), (130, 12, 128), (65, 3, 80), (5, 1, 515), (9, 2, 1000), (4, 1, 2047),
               (300, 1, 2048), (3, 1, 4099), (6, 1, 7168), (2, 1, 8191), (3, 1, 16384), (2, 1, 16383), (700, 2, 192)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D", NORM_SHAPES)
def test_norm_and_gradient(kda, T, H, D, dtype):
    gen = torch.Generator().manual_seed(D)
    for kind, gated, biased in (("layer", False, True), ("rms", True, False), ("layer", True, True), ("rms", False, True)):
        x = (randn(gen, T, H, D) + 0.7).to(DT[dtype])
        dy, z = randn(gen, T, H, D, dtype=DT[dtype]), randn(gen, T, H, D, dtype=DT[dtype]) if gated else None
        w = 1 + 0.3 * randn(gen, H, D)
        b = 0.3 * randn(gen, H, D) if biased else None
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        name = f"norm {dtype} {T}x{H}x{D} {kind}{' gated' if gated else ''}"
        eps = 1e-5
        y, mean, rstd = kda.norm_fwd(c(x), c(w), bias=c(b), z=c(z), eps=eps, kind=kind)
        yr, mr, rr = ref.norm(x, w, b, z, eps, kind)
        if D > 1 or kind == "rms":
            ref.check(name + " y", y, yr, EXACT[dtype])
            ref.check(name + " rstd", rstd, rr, 1e-6)
        if kind == "layer":
            ref.check(name + " mean", mean, mr, 1e-6)
        else:
            assert mean is None
        dx, dw, db, dz = kda.norm_bwd(c(dy), c(x), c(w), mean, rstd, bias=c(b), z=c(z), kind=kind)
        xr, wr, br, zr = ref.norm_grad(x, w, b, z, eps, kind, dy)
        if D > 1:
            # dx subtracts two means from its terms: a few roundings more, 2^-8 for bf16 all the same
            ref.check(name + " dx", dx, xr, max(EXACT[dtype], 2e-6))
            ref.check(name + " dw", dw, wr, 2e-6)
        if b is not None:
            ref.check(name + " db", db, br, 2e-6)
        if z is not None and D > 1:
            ref.check(name + " dz", dz, zr, max(EXACT[dtype], 2e-6))


def test_norm_unaligned_rows(kda):
    """A vectorisable width at an address that allows single elements only."""
    gen = torch.Generator().manual_seed(2)
    base = randn(gen, 4 * 128 + 1, dtype=torch.bfloat16).cuda()
    x = base[1:].view(2, 2, 128)
    w = torch.ones(2, 128, device="cuda")
    y, _, _ = kda.norm_fwd(x, w)
    yr, _, _ = ref.norm(x.cpu(), w.cpu(), None, None, 1e-5, "layer")
    ref.check("unaligned", y, yr, EXACT["bf16"])


# more workgroups than one axis of a launch holds (2^32 threads)
def test_norm_of_very_many_rows(kda):
    T, D = 2 ** 28 + 5, 2
    x = torch.randn(T, 1, D, device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(1))
    w = torch.tensor([[0.5, -2.0]], device="cuda")
    y, _, _ = kda.norm_fwd(x, w, eps=1e-3, kind="rms", stats=False)
    for at in (0, T // 2, T - 4096):
        r = x[at:at + 4096].double()
        want = r / (r.square().mean(-1, keepdim=True) + 1e-3).sqrt() * w.double()
        ref.check(f"row {at}", y[at:at + 4096], want.cpu(), EXACT["bf16"])
    assert torch.equal(torch.signbit(y[..., 0]), torch.signbit(x[..., 0])), "a row was left out"
    assert torch.equal(torch.signbit(y[..., 1]), ~torch.signbit(x[..., 1])), "a row was left out"


def test_rope_of_very_many_tokens(kda):
    T = 2 ** 28 + 5
    q = torch.randn(T, 1, 2, device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(2))
    pos = (torch.arange(T, device="cuda", dtype=torch.int32) % 4) * 2   # turns by 0, 1/4, 1/2, 3/4 of a circle
    freq = torch.tensor([torch.pi / 4], dtype=torch.float64, device="cuda")
    out, _ = kda.rope(q, None, pos, freq)
    for n in range(4):
        a, b = q[n::4, 0, 0], q[n::4, 0, 1]
        want = ((a, b), (-b, a), (-a, -b), (b, -a))[n]
        # sine and cosine of a quarter turn: exact up to their rounding in fp32
        assert torch.allclose(out[n::4, 0, 0].float(), want[0].float(), rtol=2.0 ** -8, atol=1e-5)
        assert torch.allclose(out[n::4, 0, 1].float(), want[1].float(), rtol=2.0 ** -8, atol=1e-5)


def test_norm_constant_and_large_rows(kda):
    """A constant row has variance 0 exactly; a large mean costs no digits."""
    x = torch.full((2, 1, 1024), 3.0).cuda()
    w, b = torch.ones(1, 1024).cuda(), torch.full((1, 1024), 0.25).cuda()
    y, mean, rstd = kda.norm_fwd(x, w, bias=b, eps=1e-5)
    assert bool((y == 0.25).all()) and bool((mean == 3).all())
    gen = torch.Generator().manual_seed(8)
    big = (randn(gen, 3, 1, 1000) + 4096.0)
    y, _, _ = kda.norm_fwd(big.cuda(), torch.ones(1, 1000).cuda())
    yr, _, _ = ref.norm(big, torch.ones(1, 1000), None, None, 1e-5, "layer")
    # the mean of values near 4096 is off by a few 2^-24 of it: 4096 * 4 * 2^-24 = 1e-3 of the row's spread
    ref.check("large mean", y, yr, 1e-3)


@pytest.mark.parametrize("D", [128, 257, 5000])
def test_norm_over_its_input_or_gate(kda, D):
    gen = torch.Generator().manual_seed(D)
    x, z = (randn(gen, 33, 2, D, dtype=torch.bfloat16).cuda() for _ in range(2))
    w, b = (randn(gen, 2, D).cuda() for _ in range(2))
    want, mean, rstd = kda.norm_fwd(x, w, b, z)
    for k in range(2):
        t = [x.clone(), z.clone()]
        y, m, r = kda.norm_fwd(t[0], w, b, t[1], y=t[k])
        assert y is t[k] and torch.equal(y, want) and torch.equal(m, mean) and torch.equal(r, rstd)
        assert torch.equal(t[1 - k], (x, z)[1 - k])


def test_norm_no_tokens(kda):
    x = torch.zeros(0, 2, 64, device="cuda")
    w = torch.ones(2, 64, device="cuda")
    y, mean, rstd = kda.norm_fwd(x, w, bias=w)
    dx, dw, db, dz = kda.norm_bwd(x, x, w, mean, rstd, bias=w)
    assert y.shape == dx.shape == x.shape and bool((dw == 0).all()) and bool((db == 0).all())


def test_norm_gradient_same_bits(kda):
    gen = torch.Generator().manual_seed(5)
    x, dy, z = (randn(gen, 3000, 4, 128, dtype=torch.bfloat16).cuda() for _ in range(3))
    w = torch.ones(4, 128, device="cuda")
    _, _, rstd = kda.norm_fwd(x, w, z=z, kind="rms")
    a, b = (kda.norm_bwd(dy, x, w, None, rstd, z=z, kind="rms") for _ in range(2))
    for u, v in zip(a, b):
        assert u is v or torch.equal(u, v)


def test_a_layer_and_its_gradient(kda):
    """Positions, linear attention, gated norm, as a layer runs them, and the
    gradients back to q, k, v, g, z, the weight and the first state, against
    the 64-bit chain and in one HIP graph."""
    T, H, d = 200, 2, 64
    gen = torch.Generator().manual_seed(40)
    q, k, v, z, dy = (randn(gen, T, H, d) for _ in range(5))
    g = -torch.rand(T, H, generator=gen) * 0.2
    w, s0 = 1 + 0.2 * randn(gen, H, d), randn(gen, 2, H, d, d)
    cu = [0, 120, T]
    pos = torch.cat([torch.arange(120), torch.arange(80)]).to(torch.int32)
    freq, m = kda.rope_frequencies(32, scaling="linear", factor=4.0)
    t = {n: x.cuda() for n, x in dict(q=q, k=k, v=v, z=z, dy=dy, g=g, w=w, s0=s0, pos=pos, f=freq).items()}
    cud = torch.tensor(cu, dtype=torch.int32).cuda()
    scale = d ** -0.5

    def layer():
        qr, kr = kda.rope(t["q"], t["k"], t["pos"], t["f"], mscale=m)
        o, s = kda.linattn_fwd(qr, kr, t["v"], t["g"], cu_seqlens=cud, initial_state=t["s0"], scale=scale)
        y, _, rstd = kda.norm_fwd(o, t["w"], z=t["z"], kind="rms")
        do, dw, _, dz = kda.norm_bwd(t["dy"], o, t["w"], None, rstd, z=t["z"], kind="rms")
        dq, dk, dv, dg, ds = kda.linattn_bwd(qr, kr, t["v"], t["g"], do, cu_seqlens=cud, initial_state=t["s0"],
                                             scale=scale)
        dq, dk = kda.rope(dq, dk, t["pos"], t["f"], inverse=True, mscale=m, q_out=dq, k_out=dk)
        return y, s, dq, dk, dv, dg, ds, dz, dw

    got = layer()
    qr, kr = (ref.rope(x, pos, freq, "half", False, m) for x in (q, k))
    o, s, _ = ref.linattn(qr, kr, v, g, cu, s0, scale)
    y, _, _ = ref.norm(o, w, None, z, 1e-5, "rms")
    do, dw, _, dz = ref.norm_grad(o, w, None, z, 1e-5, "rms", dy)
    dq, dk, dv, dg, ds = ref.linattn_grad(qr, kr, v, g, cu, do, s0, None, scale)
    dq, dk = (ref.rope(x, pos, freq, "half", True, m) for x in (dq, dk))
    names = ("y", "state", "dq", "dk", "dv", "dg", "ds0", "dz", "dw")
    # each step adds fp32's error to the one before it: three times one operator's
    for n, a, b in zip(names, got, (y, s, dq, dk, dv, dg, ds, dz, dw)):
        ref.check(f"layer {n}", a, b, 3 * (ref.TOL_DG if n == "dg" else ref.TOL["f32"]))

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    noise = torch.zeros(1 << 20, device="cuda")
    for r in range(4):
        for x in out:
            x.zero_()
        noise.mul_(1.0001).add_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, a, b in zip(names, out, got):
            assert torch.equal(a, b), f"replay {r}: {n}"
