"""Arguments and workspaces of the layer operators at their edges, without a GPU."""
import pytest

import gated_delta_rule_75_amd as kda

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
BF16, F32 = kda.KDA_BF16, kda.KDA_F32
A = 1 << 20                                # a fake, aligned, never dereferenced address


def fwd(name, dt=BF16, H=4, Hk=2, dk=128, dv=64, N=2, T=1000, cu=A, q=A, qs=256, g=A, y=A, ws=A, wsb=1 << 40):
    return getattr(kda.lib(), name)(dt, H, Hk, dk, dv, 1.0, N, T, cu, q, qs, A, 256, A, 256, g, 1, None, None, y, ws,
                                    wsb, None)


def bwd(name, dt=BF16, H=4, Hk=2, dk=128, dv=64, N=2, T=1000, cu=A, q=A, qs=256, g=A, y=A, ws=A, wsb=1 << 40):
    return getattr(kda.lib(), name)(dt, H, Hk, dk, dv, 1.0, N, T, cu, q, qs, A, 256, A, 256, g, 1, None, A, None, y, A,
                                    A, A, None, ws, wsb, None)


@pytest.mark.parametrize("call,name", [(fwd, "kda_linattn_fwd"), (bwd, "kda_linattn_bwd")])
def test_padded_calls_refuse_what_the_plain_ones_do(call, name):
    for bad, want in ((dict(dt=3), INVALID), (dict(H=3), INVALID), (dict(N=0), INVALID), (dict(cu=None), INVALID),
                      (dict(q=None), INVALID), (dict(q=A + 8), INVALID), (dict(qs=255), INVALID), (dict(g=A + 2), INVALID),
                      (dict(y=None), INVALID), (dict(y=A + 2), INVALID), (dict(ws=None), INVALID), (dict(dk=96), UNSUPPORTED),
                      (dict(T=1 << 31), INVALID), (dict(wsb=1000), WS_SMALL)):
        assert call(name, **bad) == call(name + "_padded", **bad) == want, bad


def test_the_table_of_first_blocks_has_its_room():
    """From 257 sequences on, where they are cut: 4 bytes a sequence and one more."""
    f, b = kda.linattn_fwd_workspace_size, kda.linattn_bwd_workspace_size
    state = 64 * 64 * 4
    for size, arrays in ((f, 1), (b, 2)):
        at = [size(BF16, 1, 1, 64, 64, n, 100000) for n in (255, 256, 257)]
        rest = 2 * 1024 if size is b else 1024
        assert state * arrays <= at[1] - at[0] <= state * (arrays + 1) + rest
        table = (258 * 4 + 255) // 256 * 256
        assert at[2] - at[1] >= state * arrays + table
    assert f(BF16, 1, 1, 64, 64, 1000, 64) == 256           # not cut: no states, no table
