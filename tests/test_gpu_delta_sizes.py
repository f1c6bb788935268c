"""The gated delta rule with more sequences than one axis of a launch holds as workgroups."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import gated_delta_rule_75_amd as m
    m.lib()
    yield m
    torch.cuda.empty_cache()


def test_no_tokens_of_many_sequences(kda):
    """2^22 sequences of 128 value columns: 2^23 workgroups of 512 threads are 2^32."""
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, v, g = e(0, 1, 64), e(0, 1, 128), e(0, 1, dtype=torch.float32)
    cu = torch.zeros((1 << 22) + 1, dtype=torch.int32, device="cuda")
    y, s = kda.gdr_fwd(q, q, v, g, g, cu_seqlens=cu, output_final_state=False)
    torch.cuda.synchronize()
    assert y.shape == (0, 1, 128) and s is None


def test_tokens_behind_a_million_workgroups(kda):
    """Two workgroups a sequence and 2^19 + 40 sequences: the grid takes a second axis.  A few sequences at either
    end have tokens, and the bits of a call of their own."""
    N, dk, dv = (1 << 19) + 40, 64, 128
    gen = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    lens = {0: 3, 7: 70, N - 41: 1, N - 39: 66, N - 1: 9}
    T = sum(lens.values())
    q, k = (torch.nn.functional.normalize(r(T, 1, dk), dim=-1).bfloat16() for _ in range(2))
    v, dy, g, beta = r(T, 1, dv).bfloat16(), r(T, 1, dv).bfloat16(), -torch.rand(T, 1, device="cuda"), torch.rand(T, 1, device="cuda")
    counts = torch.zeros(N, dtype=torch.int32)
    for n, m in lens.items():
        counts[n] = m
    offsets = lambda c: torch.cat([torch.zeros(1, dtype=torch.int32), c.cumsum(0).int()]).cuda()  # noqa: E731
    few = offsets(torch.tensor(list(lens.values())))
    at = torch.tensor(list(lens), device="cuda")
    y0, s0 = kda.gdr_fwd(q, k, v, g, beta, cu_seqlens=few)
    g0 = kda.gdr_bwd(q, k, v, g, beta, dy, cu_seqlens=few)
    cu = offsets(counts)
    y, s = kda.gdr_fwd(q, k, v, g, beta, cu_seqlens=cu)
    assert torch.equal(y, y0) and torch.equal(s[at], s0)
    for a, b in zip(list(lens), list(lens)[1:]):
        assert not bool(s[a + 1:b].any())
    del s
    torch.cuda.empty_cache()
    got = kda.gdr_bwd(q, k, v, g, beta, dy, cu_seqlens=cu)
    for a, b in zip(got[:-1], g0[:-1]):
        assert torch.equal(a, b)
    assert torch.equal(got[-1][at], g0[-1])
