"""Calls of the gated delta rule that its documentation allows: states on one side alone, factors of any sign,
gradients into given rows, no gradient of the initial state, two host threads at once."""
import threading

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


def check(name, x, dtype):
    y, s = fwd(kda, x)
    yr, sr, _ = want_fwd(x)
    ref.check(name + " y", y, yr, ref.TOL[dtype])
    ref.check(name + " state", s, sr, delta.TOL_STATE)
    for n, a, b in zip(NAMES, bwd(kda, x), want_bwd(x)):
        ref.check(f"{name} {n}", a, b, tol(n, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,shape", [([70, 0, 130], (4, 2, 64, 128)), ([2060, 30], (1, 1, 128, 64))], ids=str)
@pytest.mark.parametrize("given", ["s0", "ds"])
def test_a_state_on_one_side(dtype, lens, shape, given):
    x = make(dtype, lens, *shape, seed=90)
    x["g"] = 0.1 * x["g"]
    x["ds" if given == "s0" else "s0"] = None
    check(f"only {given} {dtype} {lens}", x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-1.5, 0.0, 3.0])
def test_factors(dtype, scale):
    x = make(dtype, [130, 5], 2, 1, 128, 128, seed=91)
    x["scale"] = scale
    check(f"scale {scale} {dtype}", x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_into_given_rows(dtype):
    """kda_gdr_bwd itself: rows of no sequence stay as they are, and the initial state's gradient need not be asked for."""
    x = make(dtype, [70, 0, 31], 4, 2, 64, 128, seed=92)
    T, H, Hk, dk, dv, N = 101, 4, 2, 64, 128, 3
    want = bwd(kda, x)
    c = cuda(x)
    pad = lambda t: torch.cat([t[:3], t, t[:4]])  # noqa: E731
    q, k, v, g, b, dy = (pad(c[n]) for n in ("q", "k", "v", "g", "beta", "dy"))
    cu = cu_of(x) + 3
    like = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    dq, dkk, dvv, dg, db = like(q), like(k), like(v), like(g), like(b)
    code = kda.KDA_BF16 if dtype == "bf16" else kda.KDA_F32
    size = kda.gdr_bwd_workspace_size(code, H, Hk, dk, dv, N, T + 7)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    st = kda.lib().kda_gdr_bwd(code, H, Hk, dk, dv, x["scale"], N, T + 7, p(cu), p(q), Hk * dk, p(k), Hk * dk, p(v), H * dv,
                               p(g), p(b), p(c["s0"]), p(dy), p(c["ds"]), p(dq), p(dkk), p(dvv), p(dg), p(db), None, p(ws),
                               size, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for n, a, e in zip(NAMES, (dq, dkk, dvv, dg, db), want):
        assert torch.equal(a[3:3 + T], e), n
        assert bool((a[:3] == 7).all()) and bool((a[3 + T:] == 7).all()), n


def test_two_host_threads():
    """Calls from two threads on streams of their own, the bits of calls one after the other."""
    xs = [make("bf16", [200, 65], 4, 2, 128, 128, seed=93), make("bf16", [2060], 1, 1, 128, 128, seed=94)]
    want = [[*fwd(kda, x), *bwd(kda, x)] for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(4):
                    got = [*fwd(kda, xs[i]), *bwd(kda, xs[i])]
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
