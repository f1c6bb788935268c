"""The gated delta rule with a decay for each head, on the GPU: prompt, single
token and gradient against the 64-bit recurrence, at lengths around the chunk
(64), empty sequences, shared heads, strides, no decay, decays that clear the
state, and keys that are nearly the same."""
import itertools

import pytest
import torch

from tests import delta_ref as delta
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "ds0")


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import gated_delta_rule_75_amd as m
    m.lib()
    return m


def make(dtype, lens, H, Hk, dk, dv, seed, decay="token", state=True, like=0.3):
    """like: the part of its direction that all keys of a head share."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True)).to(DT[dtype])
    x = dict(q=unit(r(T, Hk, dk)), k=unit((1 - like) * r(T, Hk, dk) + like * dk ** 0.5 * unit(r(1, Hk, dk)).float()),
             v=r(T, H, dv).to(DT[dtype]), dy=r(T, H, dv).to(DT[dtype]), s0=0.3 * r(N, H, dk, dv) if state else None,
             ds=0.3 * r(N, H, dk, dv) if state else None)
    x["beta"] = torch.rand(T, H, generator=gen)
    x["g"] = -torch.rand(T, H, generator=gen) * torch.logspace(-3, 0, H)[None]
    if decay == "reset":          # clears the state now and then, strongly or wholly; tokens that write nothing, or twice
        hit = torch.rand(T, H, generator=gen)
        x["g"][hit < 0.02] = -float("inf")
        x["g"][(hit >= 0.02) & (hit < 0.05)] = -90.0
        x["g"][(hit >= 0.05) & (hit < 0.2)] = 0.0
        x["beta"][hit > 0.9] = 0.0
        x["beta"][(hit > 0.85) & (hit < 0.9)] = 1.9
    if decay == "none":
        x["g"] = None
    x["cu"] = [sum(lens[:i]) for i in range(N + 1)]
    x["scale"] = 0.7
    return x


def cuda(x):
    return {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in x.items()}


def cu_of(x):
    return torch.tensor(x["cu"], dtype=torch.int32).cuda()


def fwd(kda, x, **kw):
    c = cuda(x)
    return kda.gdr_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], cu_seqlens=cu_of(x), initial_state=c["s0"],
                       scale=x["scale"], **kw)


def bwd(kda, x, **kw):
    c = cuda(x)
    return kda.gdr_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], c["dy"], cu_seqlens=cu_of(x),
                       initial_state=c["s0"], d_final_state=c["ds"], scale=x["scale"], **kw)


def want_fwd(x):
    return delta.steps(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["s0"], x["scale"])


def want_bwd(x):
    return delta.grad(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["dy"], x["s0"], x["ds"], x["scale"])


def tol(name, dtype):
    return delta.TOL_DG if name == "dg" else delta.TOL_STATE if name in ("dbeta", "ds0") else ref.TOL[dtype]


LENS = [[1], [63], [64], [65], [300], [0, 1, 130, 0, 500, 64], [2, 1, 1, 0, 5]]
SHAPES = [(4, 4, 128, 128), (6, 2, 64, 128), (3, 1, 128, 64), (2, 2, 64, 64)]
DECAYS = ["token", "reset", "none", "token"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_prompt(kda, lens, dtype):
    for i, (shape, decay) in enumerate(zip(SHAPES, DECAYS)):
        x = make(dtype, lens, *shape, seed=10 + i, decay=decay, state=i % 2 == 0)
        y, s = fwd(kda, x)
        yr, sr, _ = want_fwd(x)
        name = f"prompt {dtype} {lens} {shape} {decay}"
        ref.check(name + " y", y, yr, ref.TOL[dtype])
        ref.check(name + " state", s, sr, delta.TOL_STATE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_gradient(kda, lens, dtype):
    for i, (shape, decay) in enumerate(zip(SHAPES, DECAYS)):
        x = make(dtype, lens, *shape, seed=50 + i, decay=decay, state=i % 2 == 0)
        name = f"gradient {dtype} {lens} {shape} {decay}"
        want = want_bwd(x)
        for n, a, b in zip(NAMES, bwd(kda, x), want):
            if b is None:
                assert a is None
                continue
            if n == "dg" and lens == [1] and x["s0"] is None:
                # nothing decays before a first token without a state: what is left is the difference of q.dq and
                # v.dv, whose terms go through at most five operands of 16 bits (E, W, P, the inverse, its
                # right-hand side), each off by 2^-18
                H = b.shape[1]
                size = (ref.expand(x["q"], H) * ref.expand(want[0], H)).abs().sum(-1) + (x["v"].double() * want[2]).abs().sum(-1)
                assert bool((a.double().cpu().abs() <= 5 * 2.0 ** -18 * size).all())
                continue
            ref.check(f"{name} {n}", a, b, tol(n, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,shape", [(1, (12, 12, 128, 128)), (3, (6, 2, 64, 128)), (2, (4, 1, 128, 64)),
                                     (80, (8, 8, 64, 64)), (70, (8, 4, 128, 128))], ids=str)
def test_single_token(kda, N, shape, dtype):
    for decay in ("token", "reset", "none"):
        x = make(dtype, [1] * N, *shape, seed=77, decay=decay)
        c = cuda(x)
        state = c["s0"].clone()
        y = kda.gdr_decode_step(c["q"], c["k"], c["v"], c["g"], c["beta"], state, scale=x["scale"])
        yr, sr, _ = want_fwd(x)
        ref.check(f"token {dtype} {N} {shape} {decay} y", y, yr, ref.TOL[dtype])
        ref.check(f"token {dtype} {N} {shape} {decay} state", state, sr, delta.TOL_STATE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nearly_equal_keys(kda, dtype):
    """Keys of which 97 % is one direction, beta near 1: the chunk's matrix is far from
    the unit matrix, and its inverse must not lose digits."""
    x = make(dtype, [200, 64], 2, 2, 128, 64, seed=3, like=0.97)
    x["beta"] = 0.9 + 0.1 * x["beta"]
    y, s = fwd(kda, x)
    yr, sr, _ = want_fwd(x)
    ref.check(f"equal keys {dtype} y", y, yr, ref.TOL[dtype])
    ref.check(f"equal keys {dtype} state", s, sr, delta.TOL_STATE)
    for n, a, b in zip(NAMES, bwd(kda, x), want_bwd(x)):
        ref.check(f"equal keys {dtype} {n}", a, b, tol(n, dtype))


LONG = [([2100], (1, 1, 128, 128)), ([700, 0, 65, 1300], (2, 1, 64, 128)), ([1150, 900], (1, 1, 128, 64)),
        ([2049], (3, 3, 64, 64))]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,shape", LONG, ids=str)
def test_long_sequences_of_few_heads(kda, lens, shape, dtype):
    """Cut into segments that run side by side; decays of every kind pass from one to the next."""
    for i, decay in enumerate(("token", "reset", "none")):
        x = make(dtype, lens, *shape, seed=90 + i, decay=decay, state=i < 2)
        if decay == "token":
            x["g"] = x["g"] * 0.02       # memories of several segments
        if decay == "none":
            x["beta"] = 0.05 * x["beta"]
        y, s = fwd(kda, x)
        yr, sr, _ = want_fwd(x)
        name = f"long {dtype} {lens} {shape} {decay}"
        ref.check(name + " y", y, yr, ref.TOL[dtype])
        ref.check(name + " state", s, sr, delta.TOL_STATE)
        for n, a, b in zip(NAMES, bwd(kda, x), want_bwd(x)):
            if b is not None:
                ref.check(f"{name} {n}", a, b, tol(n, dtype))


@pytest.mark.parametrize("lens,H", [([130], 2), ([2100], 1)], ids=str)
def test_a_decay_of_zero_ends_a_state_that_is_not_finite(kda, lens, H):
    """Infinities and NaN in the initial state are in what comes before a decay of zero, and in nothing behind it;
    a column of the state that is finite is not touched by the others."""
    x = make("bf16", lens, H, H, 64, 64, seed=6)
    at = lens[0] // 2 + 3
    x["g"][at] = -float("inf")
    good, sg = fwd(kda, x)
    x["s0"][:, :, 5, 7], x["s0"][:, :, 9, 40] = float("nan"), float("inf")
    y, s = fwd(kda, x)
    assert torch.equal(y[at:], good[at:]) and torch.equal(s, sg)
    rest = [c for c in range(64) if c not in (7, 40)]
    assert torch.equal(y[:at][..., rest], good[:at][..., rest])
    assert not bool(torch.isfinite(y[0, :, [7, 40]]).any())
    c = cuda({n: (v[:1] if n in ("q", "k", "v", "beta") else v) for n, v in x.items()})
    state = c["s0"].clone()
    y1 = kda.gdr_decode_step(c["q"], c["k"], c["v"], torch.full((1, H), -float("inf")).cuda(), c["beta"], state)
    assert bool(torch.isfinite(y1).all()) and bool(torch.isfinite(state).all())


def test_prompt_then_tokens(kda):
    """A prompt's state carried on by single tokens, as one sequence."""
    x = make("bf16", [90], 4, 2, 128, 128, seed=8, state=False)
    yr, sr, _ = want_fwd(x)
    c = cuda(x)
    m = 83
    y, s = kda.gdr_fwd(*(c[n][:m].contiguous() for n in ("q", "k", "v", "g", "beta")), scale=x["scale"])
    ys = [y]
    for t in range(m, 90):
        ys.append(kda.gdr_decode_step(*(c[n][t:t + 1] for n in ("q", "k", "v", "g", "beta")), s, scale=x["scale"]))
    ref.check("prompt then tokens y", torch.cat(ys), yr, ref.TOL["bf16"])
    ref.check("prompt then tokens state", s, sr, delta.TOL_STATE)
