"""Linear attention with a decay for each head, on the GPU: prompt, single token
and gradient against the 64-bit recurrence, at lengths around the chunk (64) and
block (256 and more) sizes, empty sequences, shared heads, strides, both forms
of the decay, and decays that clear the state."""
import itertools

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


def make(dtype, lens, H, Hk, dk, dv, seed, decay="token", state=True):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = dict(q=r(T, Hk, dk).to(DT[dtype]), k=r(T, Hk, dk).to(DT[dtype]), v=r(T, H, dv).to(DT[dtype]),
             dy=r(T, H, dv).to(DT[dtype]), s0=r(N, H, dk, dv) if state else None, ds=r(N, H, dk, dv) if state else None)
    if decay == "head":
        x["g"] = -torch.rand(H, generator=gen) * 0.3
    else:
        x["g"] = -torch.rand(T, H, generator=gen) * torch.logspace(-3, 0, H)[None]
    if decay == "reset":          # clears the state now and then, strongly or wholly
        hit = torch.rand(T, H, generator=gen)
        x["g"][hit < 0.02] = -float("inf")
        x["g"][(hit >= 0.02) & (hit < 0.05)] = -90.0
        x["g"][(hit >= 0.05) & (hit < 0.2)] = 0.0
    x["cu"] = [sum(lens[:i]) for i in range(N + 1)]
    x["scale"] = dk ** -0.5
    return x


def cuda(x):
    return {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in x.items()}


def cu_of(x):
    return torch.tensor(x["cu"], dtype=torch.int32).cuda()


def fwd(kda, x, **kw):
    c = cuda(x)
    return kda.linattn_fwd(c["q"], c["k"], c["v"], c["g"], cu_seqlens=cu_of(x), initial_state=c["s0"],
                           scale=x["scale"], **kw)


def bwd(kda, x, **kw):
    c = cuda(x)
    return kda.linattn_bwd(c["q"], c["k"], c["v"], c["g"], c["dy"], cu_seqlens=cu_of(x), initial_state=c["s0"],
                           d_final_state=c["ds"], scale=x["scale"], **kw)


LENS = [[1], [63], [64], [65], [300], [0, 1, 130, 0, 700, 64], [2, 1, 1, 0, 5], [513, 255, 257]]
SHAPES = [(4, 4, 128, 128), (6, 2, 64, 128), (3, 1, 128, 64), (2, 2, 64, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_prompt(kda, lens, dtype):
    for i, (shape, decay) in enumerate(zip(SHAPES, itertools.cycle(["token", "head", "reset"]))):
        x = make(dtype, lens, *shape, seed=10 + i, decay=decay, state=i % 2 == 0)
        y, s = fwd(kda, x)
        yr, sr, _ = ref.linattn(x["q"], x["k"], x["v"], x["g"], x["cu"], x["s0"], x["scale"])
        name = f"prompt {dtype} {lens} {shape} {decay}"
        ref.check(name + " y", y, yr, ref.TOL[dtype])
        ref.check(name + " state", s, sr, ref.TOL_STATE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_gradient(kda, lens, dtype):
    for i, (shape, decay) in enumerate(zip(SHAPES, itertools.cycle(["token", "head", "reset"]))):
        x = make(dtype, lens, *shape, seed=50 + i, decay=decay, state=i % 2 == 0)
        got = bwd(kda, x)
        want = ref.linattn_grad(x["q"], x["k"], x["v"], x["g"], x["cu"], x["dy"], x["s0"], x["ds"], x["scale"])
        name = f"gradient {dtype} {lens} {shape} {decay}"
        for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), got, want):
            ref.check(f"{name} {n}", a, b, ref.TOL_DG if n == "dg" else ref.TOL_STATE if n == "ds0" else ref.TOL[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_sequence_many_blocks(kda, dtype):
    """Cut into blocks (one head, 3001 tokens), against the recurrence; the
    states pass from block to block in both directions."""
    x = make(dtype, [3001], 1, 1, 64, 64, seed=5)
    x["g"] = x["g"] * 0.3
    y, s = fwd(kda, x)
    yr, sr, _ = ref.linattn(x["q"], x["k"], x["v"], x["g"], x["cu"], x["s0"], x["scale"])
    ref.check(f"long {dtype} y", y, yr, ref.TOL[dtype])
    ref.check(f"long {dtype} state", s, sr, ref.TOL_STATE)
    want = ref.linattn_grad(x["q"], x["k"], x["v"], x["g"], x["cu"], x["dy"], x["s0"], x["ds"], x["scale"])
    for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), bwd(kda, x), want):
        ref.check(f"long {dtype} {n}", a, b, ref.TOL_DG if n == "dg" else ref.TOL_STATE if n == "ds0" else ref.TOL[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,shape", [(1, (12, 12, 128, 128)), (3, (6, 2, 64, 128)), (2, (4, 1, 128, 64)),
                                     (80, (8, 8, 64, 64)), (70, (8, 4, 128, 128))], ids=str)
def test_single_token(kda, N, shape, dtype):
    H, Hk, dk, dv = shape
    for decay in ("token", "head", "reset"):
        x = make(dtype, [1] * N, H, Hk, dk, dv, seed=77, decay=decay)
        c = cuda(x)
        state = c["s0"].clone()
        y = kda.linattn_decode_step(c["q"], c["k"], c["v"], c["g"], state, scale=x["scale"])
        yr, sr, _ = ref.linattn(x["q"], x["k"], x["v"], x["g"], list(range(N + 1)), x["s0"], x["scale"])
        ref.check(f"token {dtype} {N} {shape} {decay} y", y, yr, ref.TOL[dtype])
        ref.check(f"token {dtype} {N} {shape} {decay} state", state, sr, ref.TOL_STATE)


def test_very_many_sequences(kda):
    """More (sequence, head) pairs than 65535, the last sequence in three blocks."""
    H, N, long = 64, 1030, 400
    x = make("bf16", [1] * (N - 1) + [long], H, H, 64, 64, seed=31, state=False)
    y, s = fwd(kda, x)
    got = bwd(kda, x)
    for n, at, m in ((0, 0, 1), (N - 2, N - 2, 1), (N - 1, N - 1, long)):
        sub = {k: x[k][at:at + m] for k in ("q", "k", "v", "g", "dy")}
        yr, sr, _ = ref.linattn(sub["q"], sub["k"], sub["v"], sub["g"], [0, m], None, x["scale"])
        ref.check(f"sequence {n} y", y[at:at + m], yr, ref.TOL["bf16"])
        ref.check(f"sequence {n} state", s[n:n + 1], sr, ref.TOL_STATE)
        want = ref.linattn_grad(sub["q"], sub["k"], sub["v"], sub["g"], [0, m], sub["dy"], None, None, x["scale"])
        for name, a, b in zip(("dq", "dk", "dv", "dg"), got, want):
            if name == "dg" and m == 1:
                assert not a[at:at + m].any()      # nothing decays before a first token without a state
                continue
            ref.check(f"sequence {n} {name}", a[at:at + m], b, ref.TOL_DG if name == "dg" else ref.TOL["bf16"])
        ref.check(f"sequence {n} ds0", got[4][n:n + 1], want[4], ref.TOL_STATE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
def test_blocks_of_many_chunks(kda, dk, dv, dtype):
    """With many heads a block holds several chunks (the operands of the next
    one arrive while one is worked on); a few heads against the recurrence."""
    H, heads = 256, [0, 77, 255]
    for lens, decay in (([500, 130], "token"), ([449, 64, 1], "reset"), ([833], "head")):
        x = make(dtype, lens, H, H, dk, dv, seed=90, decay=decay)
        y, s = fwd(kda, x)
        got = bwd(kda, x)
        sub = dict(x, **{n: x[n][:, heads] for n in ("q", "k", "v", "dy", "s0", "ds")})
        sub["g"] = x["g"][heads] if decay == "head" else x["g"][:, heads]
        yr, sr, _ = ref.linattn(sub["q"], sub["k"], sub["v"], sub["g"], x["cu"], sub["s0"], x["scale"])
        name = f"chunks {dtype} {dk}x{dv} {lens} {decay}"
        ref.check(name + " y", y[:, heads], yr, ref.TOL[dtype])
        ref.check(name + " state", s[:, heads], sr, ref.TOL_STATE)
        g = sub["g"].expand(sum(lens), len(heads))
        want = ref.linattn_grad(sub["q"], sub["k"], sub["v"], g, x["cu"], sub["dy"], sub["s0"], sub["ds"], x["scale"])
        for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), got, want):
            if n == "dg" and decay == "head":
                # a sum over tokens, of both signs: each is within TOL_DG of its
                # size, so the sum is within TOL_DG of the sum of their sizes
                # (50 times the sum here)
                err, size = (a[heads].double().cpu() - b.sum(0)).abs(), b.abs().sum(0)
                print(f"[layer] {name} dg of a head: {(err / size).max():.2e} of its terms", flush=True)
                assert bool((err <= ref.TOL_DG * size).all())
                continue
            ref.check(f"{name} {n}", a[:, heads], b,
                      ref.TOL_DG if n == "dg" else ref.TOL_STATE if n == "ds0" else ref.TOL[dtype])


def test_many_chunks_same_bits_and_streams(kda):
    x = make("bf16", [500, 130], 256, 128, 128, 128, seed=91)
    want = fwd(kda, x) + bwd(kda, x)
    torch.cuda.synchronize()
    for _ in range(3):
        for a, b in zip(fwd(kda, x) + bwd(kda, x), want):
            assert torch.equal(a, b)


def test_tokens_one_by_one_equal_the_prompt(kda):
    x = make("f32", [70, 70], 4, 2, 64, 128, seed=8)
    y, s = fwd(kda, x)
    c = cuda(x)
    state = c["s0"].clone()
    rows = torch.arange(0, 140, 70, device="cuda")
    for t in range(70):
        yt = kda.linattn_decode_step(*(c[n][rows + t] for n in ("q", "k", "v", "g")), state, scale=x["scale"])
        ref.check(f"token {t}", yt, y[rows + t].double().cpu(), ref.TOL["f32"])
    ref.check("states", state, s.double().cpu(), ref.TOL_STATE)


def test_resume_equals_one_call(kda):
    """A prompt in two calls, the second from the first one's final state, in place."""
    x = make("bf16", [500], 2, 2, 128, 128, seed=9)
    c = cuda(x)
    y, s = fwd(kda, x)
    state = c["s0"].clone()
    parts = [kda.linattn_fwd(*(c[n][a:b] for n in ("q", "k", "v", "g")), initial_state=state, final_state=state,
                             scale=x["scale"])[0] for a, b in ((0, 192), (192, 500))]
    ref.check("outputs", torch.cat(parts), y.double().cpu(), 2 * ref.TOL["bf16"])
    ref.check("state", state, s.double().cpu(), ref.TOL_STATE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_a_projection(kda, dtype):
    """q, k, v as slices of one [T, width] tensor equal packed copies, bit for bit."""
    T, H, Hk, dk, dv = 333, 4, 2, 64, 128
    x = make(dtype, [T], H, Hk, dk, dv, seed=3)
    c = cuda(x)
    w = 2 * Hk * dk + H * dv + 16
    buf = torch.full((T, w), 7.0, dtype=DT[dtype], device="cuda")
    v = {"q": buf[:, :Hk * dk].view(T, Hk, dk), "k": buf[:, Hk * dk:2 * Hk * dk].unflatten(1, (Hk, dk)),
         "v": buf[:, 2 * Hk * dk:2 * Hk * dk + H * dv].unflatten(1, (H, dv))}
    for n, t in v.items():
        t.copy_(c[n])
    for got, want in zip(kda.linattn_fwd(v["q"], v["k"], v["v"], c["g"], initial_state=c["s0"]),
                         kda.linattn_fwd(c["q"], c["k"], c["v"], c["g"], initial_state=c["s0"])):
        assert torch.equal(got, want)
    for got, want in zip(kda.linattn_bwd(v["q"], v["k"], v["v"], c["g"], c["dy"], d_final_state=c["ds"]),
                         kda.linattn_bwd(c["q"], c["k"], c["v"], c["g"], c["dy"], d_final_state=c["ds"])):
        assert torch.equal(got, want)
    s1, s2 = (torch.zeros(T, H, dk, dv, device="cuda") for _ in range(2))
    assert torch.equal(kda.linattn_decode_step(v["q"], v["k"], v["v"], c["g"], s1),
                       kda.linattn_decode_step(c["q"], c["k"], c["v"], c["g"], s2))
    assert torch.equal(s1, s2)


def test_gradient_against_differences(kda):
    """Directional differences of the fp32 forward pass.  f is linear in q, v and
    the state, so a difference is exact there but for fp32's error (1e-5 of |f|
    over a step of 1/16); in k and g the cubic term adds about step^2."""
    x = make("f32", [150, 0, 90], 2, 1, 64, 64, seed=31)
    grads = dict(zip(("q", "k", "v", "g", "s0"), bwd(kda, x)))
    gen = torch.Generator().manual_seed(1)

    def f(y):
        o, s = fwd(kda, y)
        return float((o.double().cpu() * x["dy"].double()).sum() + (s.double().cpu() * x["ds"].double()).sum())

    for n, step in (("q", 1 / 16), ("k", 1 / 64), ("v", 1 / 16), ("g", 1 / 256), ("s0", 1 / 16)):
        u = torch.randn(x[n].shape, generator=gen)
        if n == "g":
            u = u * x["g"].abs()       # stays below zero
        got = (f({**x, n: x[n] + step * u}) - f({**x, n: x[n] - step * u})) / (2 * step)
        want = float((grads[n].double().cpu() * u.double()).sum())
        size = float(grads[n].double().cpu().norm() * u.double().norm())
        assert abs(got - want) <= 2e-3 * max(abs(want), size / 20), (n, got, want, size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_bits_every_time(kda, dtype):
    x = make(dtype, [300, 70, 900], 6, 3, 128, 64, seed=12)
    a, b = (fwd(kda, x) + bwd(kda, x) for _ in range(2))
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_empty_sequences_pass_their_state(kda):
    x = make("bf16", [0, 0], 2, 2, 64, 64, seed=2)
    y, s = fwd(kda, x)
    assert y.shape == (0, 2, 64) and torch.equal(s.cpu(), x["s0"])
    got = bwd(kda, x)
    assert torch.equal(got[4].cpu(), x["ds"])
    x["g"] = torch.zeros(2)
    assert torch.equal(bwd(kda, x)[3].cpu(), torch.zeros(2))


def test_rows_outside_the_sequences_are_left(kda):
    """y and the states keep what is behind what the call writes."""
    x = make("bf16", [100, 30], 2, 2, 64, 64, seed=4)
    y = torch.full((131, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    s = torch.full((3, 2, 64, 64), 5.0, device="cuda")
    fwd(kda, x, y=y[:130], final_state=s[:2])
    assert bool((y[130] == 5).all()) and bool((s[2] == 5).all())


@pytest.mark.parametrize("decay", ["token", "head"])
def test_offsets_inside_the_rows(kda, decay):
    """Offsets that begin after row 0 and end before the last row: the rows
    around hold NaN, which nothing takes in, and gradients' rows stay."""
    x = make("bf16", [5, 200, 90, 7], 4, 2, 64, 64, seed=21, decay=decay)
    inner = dict(x, cu=[5, 205, 295], s0=x["s0"][1:3], ds=x["ds"][1:3])
    part = {n: x[n][5:295] for n in ("q", "k", "v", "dy")}
    part.update(inner, cu=[0, 200, 290], **part)
    if decay == "token":
        part["g"] = x["g"][5:295]
        inner["g"] = x["g"].clone()
        inner["g"][:5] = inner["g"][295:] = float("nan")
    for n in ("q", "k", "v", "dy"):
        inner[n] = x[n].clone()
        inner[n][:5] = inner[n][295:] = float("nan")
    y, s = fwd(kda, inner)
    yr, sr = fwd(kda, part)
    assert torch.equal(y[5:295], yr) and torch.equal(s, sr)
    got, want = bwd(kda, inner), bwd(kda, part)
    for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), got, want):
        a = a[5:295] if a.shape[0] == 302 else a
        # the same tokens in the same blocks: the same bits, but for the order
        # in which dg of a head is summed
        if n == "dg" and decay == "head":
            ref.check("dg of a head", a, b.double().cpu(), 1e-6)
        else:
            assert torch.equal(a, b), n


def test_two_calls_at_once(kda):
    """Two streams with a workspace each."""
    xs = [make("bf16", [900, 300], 4, 4, 128, 128, seed=s) for s in (61, 62)]
    want = [fwd(kda, x) + bwd(kda, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, st in zip(xs, streams):
            with torch.cuda.stream(st):
                got.append(fwd(kda, x) + bwd(kda, x))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)


def test_decays_next_to_each_other(kda):
    """Hard to tell apart in fp32 sums: a near-clearing decay and, behind it,
    tiny ones whose products still have to be exact."""
    x = make("f32", [256], 2, 2, 64, 64, seed=23)
    x["g"][:] = -1e-4
    x["g"][10::64] = -150.0
    x["g"][33::64] = -200.0
    y, s = fwd(kda, x)
    yr, sr, _ = ref.linattn(x["q"], x["k"], x["v"], x["g"], x["cu"], x["s0"], x["scale"])
    ref.check("y", y, yr, ref.TOL["f32"])
    ref.check("state", s, sr, ref.TOL_STATE)
    want = ref.linattn_grad(x["q"], x["k"], x["v"], x["g"], x["cu"], x["dy"], x["s0"], x["ds"], x["scale"])
    for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), bwd(kda, x), want):
        ref.check(n, a, b, ref.TOL_DG if n == "dg" else ref.TOL["f32"])


def test_many_sequences(kda):
    """More sequences than a wave has lanes, empty ones among them."""
    lens = [(7 * i) % 5 for i in range(200)]
    x = make("bf16", lens, 2, 2, 64, 64, seed=24)
    y, s = fwd(kda, x)
    yr, sr, _ = ref.linattn(x["q"], x["k"], x["v"], x["g"], x["cu"], x["s0"], x["scale"])
    ref.check("y", y, yr, ref.TOL["bf16"])
    ref.check("state", s, sr, ref.TOL_STATE)
    want = ref.linattn_grad(x["q"], x["k"], x["v"], x["g"], x["cu"], x["dy"], x["s0"], x["ds"], x["scale"])
    for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), bwd(kda, x), want):
        ref.check(n, a, b, ref.TOL_DG if n == "dg" else ref.TOL_STATE if n == "ds0" else ref.TOL["bf16"])


def test_weak_and_strong_decay_of_whole_sequences(kda):
    """g = 0 keeps everything, g = -5 forgets within a tile: the state's scale
    is renewed never and in every chunk."""
    for g in (0.0, -5.0):
        x = make("bf16", [400], 2, 2, 128, 128, seed=25)
        x["g"][:] = g
        y, s = fwd(kda, x)
        yr, sr, _ = ref.linattn(x["q"], x["k"], x["v"], x["g"], x["cu"], x["s0"], x["scale"])
        ref.check(f"g {g} y", y, yr, ref.TOL["bf16"])
        ref.check(f"g {g} state", s, sr, ref.TOL_STATE)
        want = ref.linattn_grad(x["q"], x["k"], x["v"], x["g"], x["cu"], x["dy"], x["s0"], x["ds"], x["scale"])
        for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), bwd(kda, x), want):
            ref.check(f"g {g} {n}", a, b, ref.TOL_DG if n == "dg" else ref.TOL_STATE if n == "ds0" else ref.TOL["bf16"])


def test_other_stream(kda):
    x = make("bf16", [700], 2, 2, 128, 128, seed=6)
    want = fwd(kda, x) + bwd(kda, x)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = fwd(kda, x) + bwd(kda, x)
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_in_a_graph(kda):
    """Prompt, gradient and single token recorded once and replayed."""
    x = make("bf16", [700, 40], 2, 1, 128, 64, seed=16)
    c, cu = cuda(x), cu_of(x)
    state = c["s0"].clone()

    def once():
        a = kda.linattn_fwd(c["q"], c["k"], c["v"], c["g"], cu_seqlens=cu, initial_state=c["s0"], scale=x["scale"])
        b = kda.linattn_bwd(c["q"], c["k"], c["v"], c["g"], c["dy"], cu_seqlens=cu, initial_state=c["s0"],
                            d_final_state=c["ds"], scale=x["scale"])
        y = kda.linattn_decode_step(c["q"][:2], c["k"][:2], c["v"][:2], c["g"][:2], state, scale=x["scale"])
        return a + b + (y,)

    want = [t.clone() for t in once()]
    after = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once()
    noise = torch.zeros(1 << 20, device="cuda")
    for r in range(4):
        state.copy_(c["s0"])
        for t in out:
            t.zero_()
        noise.mul_(1.0001).add_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), f"replay {r}"
        assert torch.equal(state, after)
