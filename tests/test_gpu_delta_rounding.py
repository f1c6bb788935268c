"""bf16 outputs of the gated delta rule are the exact values' roundings, but for the few that what is
computed inside, with 16 bits, takes to the neighbour."""
import pytest
import torch

from tests.test_gpu_delta import bwd, fwd, make, want_bwd, want_fwd

pytestmark = pytest.mark.gpu

# Operands of 16 bits (two bf16 parts) are off by 2^-18 at most, at random.  An output takes at most four such
# roundings, of terms up to twice its size: e = 2^-16 of the outputs' norm in all.  A value goes to the neighbour,
# one step s <= 2^-7 |y| away, as often as its error takes it across a border, |error| / s of the time: the
# differences' squares sum to |error| s <= 2^-7 |error| |y| each, 2^-7 e = 2^-23 of the outputs' in all.
BOUND = 2.0 ** -11.5


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import gated_delta_rule_75_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("lens,shape", [([500], (4, 4, 128, 128)), ([1, 130, 64], (4, 2, 64, 128)), ([300], (3, 3, 128, 64))],
                         ids=str)
def test_nearly_all_are_the_nearest(kda, lens, shape):
    x = make("bf16", lens, *shape, seed=80)
    got, want = [fwd(kda, x)[0], *bwd(kda, x)[:3]], [want_fwd(x)[0], *want_bwd(x)[:3]]
    for n, a, b in zip(("y", "dq", "dk", "dv"), got, want):
        a, b = a.double().cpu(), b.to(torch.bfloat16).double()
        e = float((a - b).norm() / b.norm())
        print(f"[rounding] {lens} {shape} {n}: {float((a != b).double().mean()):.2%} differ, rel {e:.1e}")
        assert e <= BOUND, (n, e)
