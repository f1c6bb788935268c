"""Packed sequences of which the long ones are cut into segments: the others are walked whole, and
pay nothing for it."""
import pytest
import torch

import gated_delta_rule_75_amd as kda
from tests import delta_ref as delta
from tests import layer_ref as ref
from tests.test_gpu_delta import NAMES, bwd, cu_of, cuda, fwd, make, tol, want_bwd, want_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    kda.lib()


def alone(x, n):
    """Sequence n of x as a call of its own."""
    a, b = x["cu"][n], x["cu"][n + 1]
    one = {k: (v[a:b] if k in ("q", "k", "v", "g", "beta", "dy") else v) for k, v in x.items()}
    for k in ("s0", "ds"):
        one[k] = None if x[k] is None else x[k][n:n + 1]
    one["cu"] = [0, b - a]
    return one


# 320 tokens a segment: two segments, less, none, three, four
LENS = [640, 300, 0, 64, 641, 1200]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 64, 64), (1, 1, 64, 128), (1, 1, 128, 64)], ids=str)
def test_fewer_than_three_segments_stay_whole(dtype, shape):
    x = make(dtype, LENS, *shape, seed=70)
    x["g"] = 0.05 * x["g"]
    y, s = fwd(kda, x)
    g = bwd(kda, x)
    for n in range(4):
        one, a, b = alone(x, n), x["cu"][n], x["cu"][n + 1]
        y1, s1 = fwd(kda, one)
        assert torch.equal(y[a:b], y1) and torch.equal(s[n], s1[0]), n
        for name, all_, mine in zip(NAMES, g, bwd(kda, one)):
            assert torch.equal(all_[n:n + 1] if name == "ds0" else all_[a:b], mine), (n, name)
    yr, sr, _ = want_fwd(x)
    ref.check(f"segments {dtype} {shape} y", y, yr, ref.TOL[dtype])
    ref.check(f"segments {dtype} {shape} state", s, sr, delta.TOL_STATE)
    for n, a, b in zip(NAMES, g, want_bwd(x)):
        ref.check(f"segments {dtype} {shape} {n}", a, b, tol(n, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_ones_among_many(dtype):
    lens = [3] * 60 + [1500] + [0, 7] * 60 + [980] + [70] * 10
    x = make(dtype, lens, 2, 1, 64, 64, seed=71, decay="reset")
    x["g"] = 0.02 * x["g"]
    y, s = fwd(kda, x)
    yr, sr, _ = want_fwd(x)
    ref.check(f"among many {dtype} y", y, yr, ref.TOL[dtype])
    ref.check(f"among many {dtype} state", s, sr, delta.TOL_STATE)
    for n, a, b in zip(NAMES, bwd(kda, x), want_bwd(x)):
        ref.check(f"among many {dtype} {n}", a, b, tol(n, dtype))


@pytest.mark.parametrize("grad", [False, True])
def test_states_of_whole_sequences_stay_out_of_the_workspace(grad):
    """128 sequences of one chunk: segments are 8 chunks long, so none is cut, and the workspace's last part, the
    segments' states, is left as it is."""
    N, H, d = 128, 2, 64
    x = make("bf16", [64] * N, H, H, d, d, seed=72)
    c = cuda(x)
    size = (kda.gdr_bwd_workspace_size if grad else kda.gdr_fwd_workspace_size)(kda.KDA_BF16, H, H, d, d, N, 64 * N)
    ws = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    args = [c[n] for n in ("q", "k", "v", "g", "beta")] + ([c["dy"]] if grad else [])
    kw = dict(d_final_state=c["ds"]) if grad else {}
    (kda.gdr_bwd if grad else kda.gdr_fwd)(*args, cu_seqlens=cu_of(x), initial_state=c["s0"], workspace=ws, **kw)
    assert bool((ws[-N * H * d * d * 4:] == 7).all())
