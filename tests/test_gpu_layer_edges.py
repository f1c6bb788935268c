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
