"""The gradient of the gated delta rule's decays where these are strong, on the GPU against 64 bits:
each head and each token by itself, since a norm over all of them shows the weak decays only."""
import pytest
import torch

from tests import delta_ref as delta
from tests import layer_ref as ref
from tests.test_gpu_delta import NAMES, bwd, make, tol, want_bwd

pytestmark = pytest.mark.gpu

RATES = (0.002, 1.0, 4.0, 8.0, 12.0, 20.0)      # of the heads


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import gated_delta_rule_75_amd as m
    m.lib()
    return m


def sizes(x):
    """The norms of each token's decayed state u and of its gradient U, whose product is dg: [T, H]."""
    T, H, dv = x["v"].shape
    seen = delta.steps(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["s0"], x["scale"])[2]
    q, k, dy, beta = ref.expand(x["q"], H), ref.expand(x["k"], H), x["scale"] * x["dy"].double(), x["beta"].double()
    a, out = torch.exp(x["g"].double()), torch.zeros(T, H, dtype=torch.float64)
    for n in range(len(x["cu"]) - 1):
        R = torch.zeros(H, q.shape[-1], dv, dtype=torch.float64) if x["ds"] is None else x["ds"][n].double()
        for t in range(x["cu"][n + 1] - 1, x["cu"][n] - 1, -1):
            D = R + q[t][:, :, None] * dy[t][:, None, :]
            U = D - k[t][:, :, None] * (beta[t][:, None] * (D * k[t][:, :, None]).sum(1))[:, None, :]
            out[t] = U.norm(dim=(1, 2)) * seen[t][1].norm(dim=(1, 2))
            R = U * a[t][:, None, None]
    return out


def check(name, x, got):
    want = want_bwd(x)
    for n, a, b in zip(NAMES, got, want):
        if float(b.abs().max()) < 2.0 ** -150:      # less than half of the least number of 32 bits: 0 there
            assert not bool(a.any()), (name, n)
            continue
        ref.check(f"{name} {n}", a, b, tol(n, "bf16" if a.dtype == torch.bfloat16 else "f32"))
    dg, true = got[3].double().cpu(), want[3]
    # by heads: the norm's own bound.  By tokens: dg is the product of u and U, each within TOL_STATE of its norm
    by_head = (dg - true).norm(dim=0) / true.norm(dim=0)
    print(name, "dg by heads:", [f"{e:.1e}" for e in by_head.tolist()])
    assert bool((by_head <= delta.TOL_DG).all()), (name, by_head)
    # (below 1e-37 fp32 loses digits, then all)
    off, allowed = (dg - true).abs(), 2 * delta.TOL_STATE * sizes(x) + 1e-37
    assert bool((off <= allowed).all()), (name, float((off / allowed).max()))


SHAPES = [(6, 6, 128, 128), (6, 2, 64, 128), (6, 3, 128, 64), (6, 6, 64, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[200], [1, 64, 65, 0, 130, 2]], ids=str)
@pytest.mark.parametrize("state", [False, True])
def test_every_head_and_token(kda, dtype, lens, state):
    for i, shape in enumerate(SHAPES):
        x = make(dtype, lens, *shape, seed=20 + i, state=state)
        gen = torch.Generator().manual_seed(i)
        x["g"] = -(torch.tensor(RATES)[None] * (0.75 + 0.5 * torch.rand(sum(lens), 6, generator=gen)))
        check(f"decays {dtype} {lens} {shape} {state}", x, bwd(kda, x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_segments(kda, dtype):
    """A long sequence of two heads, one of decays from -12 to -4 and one that mixes weak and strong ones."""
    x = make(dtype, [2070], 2, 1, 64, 64, seed=30)
    gen = torch.Generator().manual_seed(5)
    u = torch.rand(2070, 2, generator=gen)
    x["g"] = -(4 + 8 * u)
    x["g"][:, 1] = torch.where(u[:, 1] < 0.9, -0.001 * u[:, 1], -10 * u[:, 1])
    check(f"decays in segments {dtype}", x, bwd(kda, x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_where_the_decay_is(kda, dtype):
    """exp(g) = 0 in 32 bits: nothing crosses the token."""
    x = make(dtype, [300, 64], 4, 2, 128, 64, seed=31)
    gone = [0, 1, 63, 64, 65, 200, 299, 300, 363]
    x["g"][gone[::2]], x["g"][gone[1::2]] = -float("inf"), -150.0
    dg = bwd(kda, x)[3]
    assert not bool(dg[gone].any())
    rest = torch.ones(364, dtype=torch.bool, device="cuda")
    rest[gone] = False
    assert bool(dg[rest].all())
    check(f"zeros {dtype}", x, bwd(kda, x))
