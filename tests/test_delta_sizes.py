"""The most (chunk, head) pairs that the gated delta rule takes: both sides of the bound."""
import pytest

import gated_delta_rule_75_amd as kda
from tests.test_delta_abi import A, INVALID, WS_SMALL, bwd, fwd

BF16 = kda.KDA_BF16
MOST = (1 << 23) - 1


@pytest.mark.parametrize("size,call", [(kda.gdr_fwd_workspace_size, fwd), (kda.gdr_bwd_workspace_size, bwd)])
@pytest.mark.parametrize("dv", [64, 128])
def test_both_sides_of_the_bound(size, call, dv):
    a = dict(H=1, Hk=1, dk=64, dv=dv, cu=A, qs=64, ks=64, vs=dv)
    # sequences alone, and with the chunks of 64000 tokens
    for N, T in ((MOST, 0), (MOST, 63), (MOST - 1000, 64000)):
        assert size(BF16, 1, 1, 64, dv, N, T) > 0
        assert call(N=N, T=T, wsb=255, **a) == WS_SMALL       # taken, but for the workspace
    for N, T in ((MOST + 1, 0), (MOST, 64), (MOST - 999, 64000)):
        assert size(BF16, 1, 1, 64, dv, N, T) == 0
        assert call(N=N, T=T, **a) == INVALID


def test_axes_of_too_many_pairs_are_refused_before_memory_is_asked_for():
    for bad in ((513,), ((1 << 31) - 1,) * 255, (500, 13)):
        with pytest.raises(kda.KDAError):
            kda.rope_pair_axes(bad)
    assert kda.rope_pair_axes((500, 12)).tolist() == [0] * 500 + [1] * 12
