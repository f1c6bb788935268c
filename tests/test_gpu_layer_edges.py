"""The layer operators on the GPU where their main path differs from small
calls: precision in blocks of many chunks, and calls at the edges of what the
documentation allows."""
import pytest
import torch

from tests import layer_ref as ref
from tests.test_gpu_linattn import bwd, fwd, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import gated_delta_rule_75_amd as m
    m.lib()
    return m


def heads_of(x, heads, decay):
    """The case's chosen heads alone, for the 64-bit recurrence."""
    sub = dict(x, **{n: x[n][:, heads] for n in ("q", "k", "v", "dy")})
    sub.update({n: None if x[n] is None else x[n][:, heads] for n in ("s0", "ds")})
    sub["g"] = x["g"][heads] if decay == "head" else x["g"][:, heads]
    return sub


def only_rounded(name, got, want):
    """bf16 `got` is the 64-bit `want` but for the rounding to bf16.

    Inside, each term passes at most one operand of two bf16 parts, each rounded
    to nearest: off by at most 2^-8 2^-8 = 2^-16 of its size, and fp32 sums add
    less.  Terms have random signs, as those of `want` have, so this part is at
    most about 2^-16 of the size of `want`: against the rounding's own error of
    about 1.66e-3, added in squares, 2^-16 changes the sum by 5e-5 of it.  1 %
    leaves room for the sample."""
    alone = ref.rel(want.to(torch.bfloat16), want)
    e = ref.rel(got, want)
    print(f"[layer] {name}: rel {e:.4e}, the rounding alone {alone:.4e}", flush=True)
    assert e <= 1.01 * alone, name


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
def test_precision_does_not_depend_on_the_cut(kda, dk, dv):
    """256 heads: blocks of many chunks, the last one of 1 to 64 rows.  The same
    sequences with 2 heads: blocks of one chunk."""
    heads = [0, 100, 255]
    for lens, decay in (([449, 323, 64], "token"), ([700, 2], "head")):
        x = make("bf16", lens, 256, 256, dk, dv, seed=140, decay=decay)
        sub = heads_of(x, heads, decay)
        y, _ = fwd(kda, x)
        yr, _, _ = ref.linattn(sub["q"], sub["k"], sub["v"], sub["g"], x["cu"], sub["s0"], x["scale"])
        dv_out = bwd(kda, x)[2]
        want = ref.linattn_grad(sub["q"], sub["k"], sub["v"], sub["g"], x["cu"], sub["dy"], sub["s0"], sub["ds"],
                                x["scale"])
        name = f"{dk}x{dv} {lens} {decay}"
        only_rounded(f"{name} y", y[:, heads], yr)
        only_rounded(f"{name} dv", dv_out[:, heads], want[2])
        for n, end in enumerate(x["cu"][1:]):
            tail = (lens[n] - 1) % 64 + 1
            only_rounded(f"{name} y of the last {tail} rows", y[end - tail:end, heads], yr[end - tail:end])
        only_rounded(f"{name} y, heads alone", fwd(kda, sub)[0], yr)


def ones_and_a_long(kda, N, long, seed):
    """N - 2 sequences of one token around one of `long` tokens and an empty one,
    one head: no state enters, so a token's output is scale (q.k) v."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    at = N // 3
    lens = torch.ones(N, dtype=torch.int64)
    lens[at], lens[at + 1] = long, 0
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    T = int(cu[-1])
    x = {n: torch.randn(T, 1, 64, generator=gen, device="cuda") for n in ("q", "k", "v", "dy")}
    x["g"] = -torch.rand(T, 1, generator=gen, device="cuda")
    return x, cu.cuda(), int(cu[at])


@pytest.mark.parametrize("N", [257, 4095, 4096, 4097, 70000])
def test_sequences_by_the_thousand(kda, N):
    """Cut into blocks, with the block of each workgroup found by the table of
    first blocks: sizes around a step of the scan and of the search."""
    x, cu, at = ones_and_a_long(kda, N, 500, seed=N)
    y, _ = kda.linattn_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, output_final_state=False, scale=0.125)
    dq, dk, dv, dg, _ = kda.linattn_bwd(x["q"], x["k"], x["v"], x["g"], x["dy"], cu_seqlens=cu, scale=0.125)
    q, k, v, dy = (x[n].double() for n in ("q", "k", "v", "dy"))
    dot = lambda a, b: 0.125 * (a * b).sum(-1, keepdim=True)  # noqa: E731
    mid = slice(at, at + 500)
    sub = {n: x[n][mid].cpu() for n in x}
    want = [dot(q, k) * v, dot(dy, v) * k, dot(dy, v) * q, dot(q, k) * dy, torch.zeros_like(x["g"]).double()]
    args = (sub["q"], sub["k"], sub["v"], sub["g"], [0, 500])
    inner = (ref.linattn(*args, None, 0.125)[0],) + ref.linattn_grad(*args, sub["dy"], None, None, 0.125)[:4]
    for n, a, b, c in zip(("y", "dq", "dk", "dv", "dg"), (y, dq, dk, dv, dg), want, inner):
        b[mid] = c.cuda()
        ref.check(f"{N} sequences {n}", a, b.cpu(), ref.TOL_DG if n == "dg" else ref.TOL["f32"])


def test_time_grows_with_the_sequences_not_their_square(kda):
    """16 times the sequences of one token: 16 times the work.  A search through
    all sequences in every workgroup would be 256 times as much."""
    ms = []
    for N in (1 << 14, 1 << 18):
        x, cu, _ = ones_and_a_long(kda, N, 500, seed=1)
        best = float("inf")
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            kda.linattn_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, output_final_state=False)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        ms.append(best)
    print(f"[layer] 2^14 and 2^18 sequences: {ms[0]:.3f} and {ms[1]:.3f} ms", flush=True)
    assert ms[1] <= 64 * ms[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 257, 1000, 2047, 4100, 8192, 16384])
def test_norm_over_its_input_or_gate_at_every_width(kda, D, dtype):
    """Lane groups of every size, one to four runs a thread; x and z in one buffer too."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    x, z = (torch.randn(37, 3, D, generator=gen, device="cuda").to(dtype) for _ in range(2))
    w, b = (torch.randn(3, D, generator=gen, device="cuda") for _ in range(2))
    for gate in (z, x):
        want, mean, rstd = kda.norm_fwd(x, w, b, gate)
        for k in range(2):
            t = [x.clone(), gate.clone()]
            if gate is x:
                t[1] = t[0]
            y, m, r = kda.norm_fwd(t[0], w, b, t[1], y=t[k])
            assert torch.equal(y, want) and torch.equal(m, mean) and torch.equal(r, rstd), (gate is x, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [128, 1000])
def test_gate_far_from_zero(kda, D, dtype):
    """z from -100 to 100, each value of y and dz for itself: a product of a few
    fp32 factors, each off by a few 2^-24 (rstd's sum of up to 1000 squares by
    less than 8), so 32 2^-24 = 2^-19 in all, and for bf16 the output's rounding
    of 2^-8 and the fast exponential's 100 2^-24.  Below the least normal value,
    2^-126, steps of a subnormal output and factor take over."""
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    tol = {"bf16": 2.0 ** -8 + 2.0 ** -16, "f32": 2.0 ** -19}[dtype]
    gen = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(64, 1, D, generator=gen).to(dt) for _ in range(2))
    z = (200 * torch.rand(64, 1, D, generator=gen) - 100).to(dt)
    z[0, 0, :8] = torch.tensor([0.0, -0.0, 88.0, -88.0, float("inf"), -float("inf"), 1e-8, -1e-8])
    w = 1 + 0.2 * torch.randn(1, D, generator=gen)
    c = [t.cuda() for t in (x, w, z, dy)]
    y, _, rstd = kda.norm_fwd(c[0], c[1], z=c[2], kind="rms")
    dx, dw, _, dz = kda.norm_bwd(c[3], c[0], c[1], None, rstd, z=c[2], kind="rms")
    s, r = torch.sigmoid(z.double()), torch.sigmoid(-z.double())
    n, _, _ = ref.norm(x, w, None, None, 1e-5, "rms")
    step = 2.0 ** -126 if dtype == "bf16" else 2.0 ** -147
    for name, got, want, factor in (("y", y, n * s, n), ("dz", dz, dy.double() * n * s * r, dy.double() * n)):
        far = (got.cpu().double() - want).abs() - step * (1 + factor.abs())
        print(f"[layer] gate {dtype} {name}: {float((far / want.abs().clamp_min(2.0 ** -126)).max()):.2e}", flush=True)
        assert bool((far <= tol * want.abs()).all()), name
    xr, wr, _, _ = ref.norm_grad(x, w, None, z, 1e-5, "rms", dy)
    ref.check(f"gate {dtype} dx", dx, xr, 2.0 ** -8 if dtype == "bf16" else 2e-6)
    ref.check(f"gate {dtype} dw", dw, wr, 2e-6)


def dirty(nbytes):
    """Leaves NaN in the memory that the next allocations get."""
    for n in (nbytes, nbytes // 2, nbytes // 4, 1 << 20):
        torch.full((n // 4,), float("nan"), device="cuda")


PADDED = [([5, 200, 90, 7], (2, 2, 64, 64), "token"), ([0, 130, 61], (4, 2, 128, 64), "token"),
          ([70, 333, 0], (3, 1, 64, 128), "head"), ([3000, 100, 1000], (4, 4, 128, 128), "token"),
          ([64, 0, 9], (2, 1, 64, 64), "token"), ([1, 1, 1], (2, 2, 64, 64), "head")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,shape,decay", PADDED, ids=str)
def test_rows_of_no_sequence_are_zeros(kda, lens, shape, decay, dtype):
    """Padding in front of and behind one or two sequences.  Outputs that the
    call makes are zeros there, whatever was in their memory."""
    before, after = lens[0], lens[-1]
    x = make(dtype, lens, *shape, seed=160, decay=decay)
    T = sum(lens)
    x.update(cu=[before, before, T - after], s0=x["s0"][:2], ds=x["ds"][:2])
    rest = torch.ones(T, dtype=torch.bool)
    rest[before:T - after] = False
    for n in ("q", "k", "v", "dy") + (("g",) if decay == "token" else ()):
        x[n][rest] = float("nan")
    dirty(T * shape[0] * 128 * 4)
    y, s = fwd(kda, x)
    dirty(T * shape[0] * 128 * 4)
    got = bwd(kda, x)
    inner = {n: x[n][~rest] for n in ("q", "k", "v", "dy")}
    inner["g"] = x["g"][~rest] if decay == "token" else x["g"]
    cu = [0, 0, T - after - before]
    yr, sr, _ = ref.linattn(inner["q"], inner["k"], inner["v"], inner["g"], cu, x["s0"], x["scale"])
    want = ref.linattn_grad(inner["q"], inner["k"], inner["v"], inner["g"], cu, inner["dy"], x["s0"], x["ds"], x["scale"])
    ref.check("y", y[~rest], yr, ref.TOL[dtype])
    ref.check("state", s, sr, ref.TOL_STATE)
    assert not bool(y[rest].any()), "y"
    for n, a, b in zip(("dq", "dk", "dv", "dg"), got, want):
        if a.shape[0] == T:
            assert not bool(a[rest].any()), n
            a = a[~rest]
        ref.check(n, a, b, ref.TOL_DG if n == "dg" else ref.TOL[dtype])
    ref.check("ds0", got[4], want[4], ref.TOL_STATE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,shape,decay", PADDED, ids=str)
def test_rows_of_no_sequence_stay_in_the_callers_outputs(kda, lens, shape, decay, dtype):
    """A y that is given, and the C calls without _padded: those rows keep what they held."""
    H, Hk, dk, dv = shape
    before, after, T = lens[0], lens[-1], sum(lens)
    x = make(dtype, lens, *shape, seed=161, decay=decay)
    x.update(cu=[before, before, T - after], s0=x["s0"][:2], ds=x["ds"][:2])
    rest = torch.ones(T, dtype=torch.bool)
    rest[before:T - after] = False
    fives = lambda t: torch.full_like(t, 5.0)  # noqa: E731
    want = fwd(kda, x)[0]
    y = fives(want)
    fwd(kda, x, y=y)
    assert torch.equal(y[~rest], want[~rest]) and bool((y[rest] == 5).all())

    want = bwd(kda, x)
    out = [fives(t) for t in want]
    c = {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
    cu = torch.tensor(x["cu"], dtype=torch.int32).cuda()
    dt = kda.KDA_BF16 if dtype == "bf16" else kda.KDA_F32
    ws = torch.empty(kda.linattn_bwd_workspace_size(dt, H, Hk, dk, dv, 2, T), dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    st = kda.lib().kda_linattn_bwd(dt, H, Hk, dk, dv, x["scale"], 2, T, p(cu), p(c["q"]), Hk * dk, p(c["k"]), Hk * dk,
                                   p(c["v"]), H * dv, p(c["g"]), int(decay == "token"), p(c["s0"]), p(c["dy"]),
                                   p(c["ds"]), *(p(t) for t in out), p(ws), ws.numel(),
                                   torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), out, want):
        if a.shape[0] == T:
            assert torch.equal(a[~rest], b[~rest]) and bool((a[rest] == 5).all()), n
        else:
            assert torch.equal(a, b), n


# rows a slot of the norm's gradient, for each lane group: 16, 64 (one, two and
# for fp32 four runs a thread), 256, and 1024 threads a row
ROWS = [(40000, 1, 64), (30011, 1, 128), (29001, 1, 100), (7001, 1, 512), (7000, 1, 203), (9000, 1, 1024), (4097, 2, 1000),
        (2003, 1, 2048), (2500, 1, 1999), (1801, 1, 4096), (1700, 1, 8192), (1301, 1, 7001), (1100, 1, 16384),
        (1200, 1, 16001), (5000, 40, 128), (3100, 13, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D", ROWS)
def test_norm_gradient_of_many_rows(kda, T, H, D, dtype):
    """Each slot walks several rows: the row ahead, the running sums of the
    weight's gradient, the two buffers in turn.  The definition in 64 bits on the
    GPU.  A sum over T tokens of terms of random sign in fp32: tens of roundings
    a slot and up to 400 behind it, each 2^-24 at most of sums that are smaller
    than the whole: 1e-5 of the gradient's size."""
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    vec = 8 if dtype == "bf16" else 4
    slots = kda.norm_bwd_workspace_size(kda.KDA_BF16 if dtype == "bf16" else kda.KDA_F32, T, H, D) // (8 * D)
    assert T * H > slots, "one row a slot"
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    for kind, gated, biased in (("layer", False, True), ("rms", True, False), ("layer", True, True)):
        x, dy = (rnd(T, H, D) + 0.5).to(dt), rnd(T, H, D).to(dt)
        z = rnd(T, H, D).to(dt) if gated else None
        w, b = 1 + 0.3 * rnd(H, D), 0.3 * rnd(H, D) if biased else None
        _, mean, rstd = kda.norm_fwd(x, w, b, z, kind=kind)
        dx, dw, db, dz = kda.norm_bwd(dy, x, w, mean, rstd, b, z, kind=kind)
        want = ref.norm_grad(x, w, b, z, 1e-5, kind, dy)
        name = f"rows {dtype} {T}x{H}x{D} ({T * H / slots:.1f} a slot, {-(-D // vec)} runs) {kind}{' gated' if gated else ''}"
        e = 2.0 ** -8 if dtype == "bf16" else 2e-6
        for n, a, r, tol in zip(("dx", "dw", "db", "dz"), (dx, dw, db, dz), want, (e, 1e-5, 1e-5, e)):
            assert (a is None) == (r is None)
            if a is not None:
                ref.check(f"{name} {n}", a, r.cpu(), tol)


def linattn_grad_gpu(x):
    """linattn_grad of layer_ref for one sequence after the other, on the GPU and
    with the states before a token kept for 256 tokens at a time."""
    c = {n: t.cuda().double() for n, t in x.items() if isinstance(t, torch.Tensor)}
    T, H = c["v"].shape[:2]
    q, k = (c[n].repeat_interleave(H // c[n].shape[1], 1) for n in ("q", "k"))
    v, dy, a = c["v"], c["dy"] * x["scale"], torch.exp(c["g"]).expand(T, H)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, R0, y = torch.zeros(T, H, dtype=torch.float64, device="cuda"), c["ds"].clone(), torch.zeros_like(v)
    S_end = torch.empty_like(R0)
    step = lambda S, t: a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]  # noqa: E731
    for n in range(len(x["cu"]) - 1):
        lo, hi = x["cu"][n], x["cu"][n + 1]
        S, kept = c["s0"][n], []
        for t in range(lo, hi):
            if (t - lo) % 256 == 0:
                kept.append(S)
            S = step(S, t)
            y[t] = x["scale"] * (q[t][:, :, None] * S).sum(1)
        S_end[n] = S
        R = c["ds"][n].clone()
        for i in range(len(kept) - 1, -1, -1):
            part = range(lo + 256 * i, min(lo + 256 * (i + 1), hi))
            before = [kept[i]]
            for t in part:
                before.append(step(before[-1], t))
            for j in range(len(part) - 1, -1, -1):
                t = part[j]
                dq[t] = (before[j + 1] * dy[t][:, None, :]).sum(-1)
                R = R + q[t][:, :, None] * dy[t][:, None, :]
                dk[t] = (R * v[t][:, None, :]).sum(-1)
                dv[t] = (R * k[t][:, :, None]).sum(-2)
                dg[t] = a[t] * (R * before[j]).sum((-1, -2))
                R = a[t][:, None, None] * R
        R0[n] = R
    fold = lambda g: g.view(T, x["q"].shape[1], -1, g.shape[-1]).sum(2)  # noqa: E731
    return y, S_end, fold(dq), fold(dk), dv, dg, R0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,shape,decay", [([2500], (32, 32, 128, 128), "token"), ([1100, 1500], (16, 4, 64, 128), "reset"),
                                              ([2049], (12, 12, 64, 64), "head"), ([1985], (24, 8, 128, 64), "token")],
                         ids=str)
def test_several_blocks_of_several_chunks(kda, lens, shape, decay, dtype):
    """What a training step has: the states of both directions pass between
    blocks of many chunks, and dg starts anew at their ends."""
    x = make(dtype, lens, *shape, seed=170, decay=decay)
    H, T = shape[0], sum(lens)
    y, s, dq, dk, dv, dg, ds0 = linattn_grad_gpu(x)
    name = f"blocks {dtype} {lens} {shape} {decay}"
    got = fwd(kda, x)
    ref.check(name + " y", got[0], y.cpu(), ref.TOL[dtype])
    ref.check(name + " state", got[1], s.cpu(), ref.TOL_STATE)
    got = bwd(kda, x)
    for n, a, b in zip(("dq", "dk", "dv", "dg", "ds0"), got, (dq, dk, dv, dg, ds0)):
        if n == "dg" and decay == "head":
            # within TOL_DG of the sum of the terms' sizes, as each term is of its own
            err, size = (a.double() - b.sum(0)).abs(), b.abs().sum(0)
            print(f"[layer] {name} dg of a head: {(err / size).max():.2e} of its terms", flush=True)
            assert bool((err <= ref.TOL_DG * size).all())
            continue
        ref.check(f"{name} {n}", a, b.cpu(), ref.TOL_DG if n == "dg" else ref.TOL_STATE if n == "ds0" else ref.TOL[dtype])
    if dtype == "bf16":
        only_rounded(name + " dv", got[2], dv.cpu())


def test_calls_side_by_side_on_two_streams(kda):
    """Everything is on the GPU beforehand, with a workspace for each stream, and
    several calls are queued on each before anything is waited for."""
    jobs = []
    for seed, lens, shape in ((181, [4000, 1300], (8, 4, 128, 128)), (182, [2600, 0, 3100], (8, 8, 128, 128))):
        x = make("bf16", lens, *shape, seed=seed)
        c = {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
        cu, T, N = torch.tensor(x["cu"], dtype=torch.int32).cuda(), sum(lens), len(lens)
        size = [f(kda.KDA_BF16, *shape, N, T) for f in (kda.linattn_fwd_workspace_size, kda.linattn_bwd_workspace_size)]
        ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in size]
        w = torch.randn(shape[0], shape[3], device="cuda")

        def call(c=c, cu=cu, ws=ws, w=w, scale=x["scale"]):
            y, s = kda.linattn_fwd(c["q"], c["k"], c["v"], c["g"], cu_seqlens=cu, initial_state=c["s0"], scale=scale,
                                   workspace=ws[0])
            n, mean, rstd = kda.norm_fwd(y, w, z=c["v"])
            dx, dw, _, dz = kda.norm_bwd(c["dy"], y, w, mean, rstd, z=c["v"])
            return (y, s, n, dx, dw, dz) + kda.linattn_bwd(c["q"], c["k"], c["v"], c["g"], dx, cu_seqlens=cu,
                                                           initial_state=c["s0"], d_final_state=c["ds"], scale=scale,
                                                           workspace=ws[1])
        jobs.append(call)
    want = [call() for call in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(6):
        for i, call in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(call())
    torch.cuda.synchronize()
    for i, calls in enumerate(got):
        for r, out in enumerate(calls):
            for m, (a, b) in enumerate(zip(out, want[i])):
                assert torch.equal(a, b), (i, r, m)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,shape", [([40, 1, 0], (4, 2, 128, 128)), ([500, 64, 200], (4, 4, 64, 64)),
                                        ([300, 700, 0], (256, 128, 64, 128)), ([1, 1, 1], (3, 1, 128, 64))], ids=str)
def test_a_decay_of_zero_ends_any_state(kda, lens, shape, dtype):
    """States that hold NaN and infinities, cleared by the first token's decay or
    by a later one's: nothing behind it sees them.  An empty sequence keeps its own."""
    H, heads = shape[0], [0, 1, shape[0] - 1]
    x = make(dtype, lens, *shape, seed=190)
    at = [0 if n % 2 == 0 else length // 2 for n, length in enumerate(lens)]
    for n, length in enumerate(lens):
        if length:
            x["g"][x["cu"][n] + at[n]] = -float("inf")
    good = dict(x, s0=torch.zeros_like(x["s0"]))
    x["s0"][:, :, ::3] = float("nan")
    x["s0"][:, :, 1::3] = float("inf")
    y, s = fwd(kda, x)
    grads = bwd(kda, x)
    shared = shape[1] != H     # for the recurrence each value head has its own copy of the key head
    good.update({n: good[n].repeat_interleave(H // shape[1], 1) for n in ("q", "k")})
    sub = heads_of(good, heads, "token")
    yr, sr, _ = ref.linattn(sub["q"], sub["k"], sub["v"], sub["g"], x["cu"], sub["s0"], x["scale"])
    want = ref.linattn_grad(sub["q"], sub["k"], sub["v"], sub["g"], x["cu"], sub["dy"], sub["s0"], sub["ds"], x["scale"])
    for n, length in enumerate(lens):
        lo, hi = x["cu"][n] + at[n], x["cu"][n + 1]
        if length == 0:
            assert torch.equal(torch.nan_to_num(s[n]).cpu(), torch.nan_to_num(x["s0"][n]))
            continue
        ref.check(f"zero {dtype} {n} y", y[lo:hi, heads], yr[lo:hi], ref.TOL[dtype])
        ref.check(f"zero {dtype} {n} state", s[n, heads], sr[n], ref.TOL_STATE)
        if at[n] == 0:     # no gradient but that of the state itself passes the first token
            for m, i in (("dq", 0), ("dk", 1), ("dv", 2), ("dg", 3)):
                if shared and i < 2:
                    assert bool(torch.isfinite(grads[i][lo:hi]).all()), m
                elif i == 3 and length == 1:
                    # 0 as the difference of <S, R> and the token's own products:
                    # within fp32's error of their terms
                    S = sub["k"][lo].double()[:, :, None] * sub["v"][lo].double()[:, None]
                    R = sub["ds"][n].double() + x["scale"] * sub["q"][lo].double()[:, :, None] * sub["dy"][lo].double()[:, None]
                    assert bool((grads[i][lo, heads].double().cpu().abs() <= ref.TOL_DG * (S * R).abs().sum((1, 2))).all())
                else:
                    ref.check(f"zero {dtype} {n} {m}", grads[i][lo:hi, heads], want[i][lo:hi],
                              ref.TOL_DG if m == "dg" else ref.TOL[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,shape", [(1, (3, 1, 128, 64)), (70, (8, 8, 64, 64)), (70, (8, 4, 128, 128))], ids=str)
def test_a_token_starts_any_state_anew(kda, N, shape, dtype):
    x = make(dtype, [1] * N, *shape, seed=191)
    anew = torch.arange(N * shape[0]).view(N, -1) % 3 == 0
    x["g"][anew] = -float("inf")
    good = x["s0"].clone()
    good[anew] = 0
    x["s0"][anew] = float("nan")
    c = {n: t.cuda() for n, t in x.items() if isinstance(t, torch.Tensor)}
    y = kda.linattn_decode_step(c["q"], c["k"], c["v"], c["g"], c["s0"], scale=x["scale"])
    yr, sr, _ = ref.linattn(x["q"], x["k"], x["v"], x["g"], x["cu"], good, x["scale"])
    ref.check(f"anew {dtype} y", y, yr, ref.TOL[dtype])
    ref.check(f"anew {dtype} state", c["s0"], sr, ref.TOL_STATE)


@pytest.mark.parametrize("N", [40, 300])
def test_a_graph_follows_its_offsets(kda, N):
    """Recorded once; between the replays the offsets change, padding in front and
    behind included, so blocks, their table and the zeros are found anew."""
    T, H, Hk, dk, dv = 4000, 4, 2, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dy = r(T, Hk, dk), r(T, Hk, dk), r(T, H, dv), r(T, H, dv)
    g = -torch.rand(T, H, generator=gen, device="cuda")
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    offsets = []
    for seed in range(3):
        c = torch.randint(0, T + 1, (N + 1,), generator=torch.Generator().manual_seed(seed)).sort().values
        if seed == 1:
            c[-1], c[0] = T, 0
        if seed == 2:
            c[:N // 2] = 17        # many empty ones, one long
            c[N // 2:] = 3100
        offsets.append(c.int())

    def once():
        return kda.linattn_fwd(q, k, v, g, cu_seqlens=cu) + kda.linattn_bwd(q, k, v, g, dy, cu_seqlens=cu)

    want = []
    for c in offsets:
        cu.copy_(c)
        want.append([t.clone() for t in once()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once()
    for n in (0, 1, 2, 1, 0):
        cu.copy_(offsets[n])
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        lo, hi = int(offsets[n][0]), int(offsets[n][-1])
        for i, (a, b) in enumerate(zip(out, want[n])):
            assert torch.equal(a, b), (n, i)
            if a.shape[0] == T:
                assert not bool(a[:lo].any()) and not bool(a[hi:].any()), (n, i)


@pytest.mark.parametrize("shape", [(32, 32, 128, 128), (32, 8, 64, 128)], ids=str)
def test_offsets_that_pass_32_bits(kda, shape):
    """v, dy, y and the gradients hold more than 2^31 elements.  The long sequence
    starts anew 300 tokens before its end, so that its last rows and the short
    sequence behind it have values in 64 bits of their own."""
    H, Hk, dk, dv = shape
    long, short, tail = 600000, 90, 300
    T = long + short
    assert T * H * dv > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x = dict(q=r(T, Hk, dk), k=r(T, Hk, dk), v=r(T, H, dv), dy=r(T, H, dv))
    x["g"] = -torch.rand(T, H, generator=gen, device="cuda") * 0.1
    x["g"][long - tail] = -float("inf")
    cu = torch.tensor([0, long, T], dtype=torch.int32, device="cuda")
    y, s = kda.linattn_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, scale=dk ** -0.5)
    got = kda.linattn_bwd(x["q"], x["k"], x["v"], x["g"], x["dy"], cu_seqlens=cu, scale=dk ** -0.5)
    end = {n: t[long - tail:].cpu() for n, t in x.items()}
    args = (end["q"], end["k"], end["v"], end["g"], [0, tail, tail + short])
    yr, sr, _ = ref.linattn(*args, None, dk ** -0.5)
    ref.check(f"far {shape} y", y[long - tail:], yr, ref.TOL["bf16"])
    ref.check(f"far {shape} state", s, sr, ref.TOL_STATE)
    want = ref.linattn_grad(*args, end["dy"], None, None, dk ** -0.5)
    for n, a, b in zip(("dq", "dk", "dv", "dg"), got, want):
        ref.check(f"far {shape} {n}", a[long - tail:], b, ref.TOL_DG if n == "dg" else ref.TOL["bf16"])
    # the first rows, which hold no carry of an index that wrapped around
    head = {n: t[:100].cpu() for n, t in x.items()}
    yr, _, _ = ref.linattn(head["q"], head["k"], head["v"], head["g"], [0, 100], None, dk ** -0.5)
    ref.check(f"far {shape} first rows", y[:100], yr, ref.TOL["bf16"])
