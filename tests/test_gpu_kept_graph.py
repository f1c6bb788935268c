"""The norm that keeps its inputs in 8 bits and the gradient that reads them, recorded in a graph and
replayed over inputs that change: every kind of call, rows of one wave, of a workgroup, of odd width."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import gated_delta_rule_75_amd as m
    m.lib()
    return m


def bits(t):
    return None if t is None else t.view(torch.uint8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D", [(50, 3, 200), (7, 1, 2047), (33, 4, 64), (2, 1, 9000)], ids=str)
@pytest.mark.parametrize("kind,gated,biased", [("layer", True, True), ("layer", False, True), ("rms", True, False)])
def test_replayed(kda, dtype, T, H, D, kind, gated, biased):
    gen = torch.Generator("cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, dy = r(T, H, D).to(DT[dtype]), r(T, H, D).to(DT[dtype])
    z = r(T, H, D).to(DT[dtype]) if gated else None
    w, b = r(H, D), r(H, D) if biased else None

    def call():
        y, mean, rstd, kept = kda.norm_fwd_kept(x, w, bias=b, z=z, kind=kind)
        return [y, mean, rstd, *kept, *kda.norm_bwd_kept(dy, kept, w, mean, rstd, bias=b, kind=kind)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        for t in (x, dy, z, w, b):
            if t is not None:
                t.copy_(r(*t.shape) * 2.0 ** (i - 1))
        graph.replay()
        torch.cuda.synchronize()
        for n, (a, e) in enumerate(zip(out, call())):
            assert (a is None) == (e is None) and (a is None or torch.equal(bits(a), bits(e))), (i, n)
