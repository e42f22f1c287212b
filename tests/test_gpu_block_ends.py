"""GPU tests of a block's backward where one of the two gradients that reach it is absent: the same as
with zeros in its place, every result there."""
import pytest
import torch

import routing_permute_grouped_amd as rpg
from tests.test_gpu_block import BF16, F32, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("absent", ["dx_next", "dout"])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_an_absent_gradient_is_zero(dt, absent):
    p = inputs(dt, T=37, seed=11)
    kw = dict(gamma_pre=p["gamma_pre"], gamma_post=p["gamma_post"], gamma_next=p["gamma_next"], gate=p["gate"], scale=0.75)
    w = (p["w1"], p["w3"], p["w2"])
    fwd = rpg.moe_block(p["resid"], *w, 3, 32, p["wg"], save_for_backward=True, **kw)

    def back(**g):
        return rpg.moe_block_backward(fwd, g["dout"], p["resid"], *w, 32, p["wg"], dx_next=g["dx_next"], **kw)

    both = dict(dout=p["dout"], dx_next=p["dx_next"])
    got = back(**{**both, absent: None})
    want = back(**{**both, absent: torch.zeros_like(both[absent])})
    assert sorted(got) == sorted(want) and {"dgamma_next", "dgamma_post", "dgamma_pre", "dgate"} <= set(got)
    rows = int(fwd["offsets"][-1])    # the permuted rows behind the last segment are nobody's
    for n in want:
        if n in ("dab", "dx_perm", "dy_perm"):
            got[n], want[n] = got[n][:rows], want[n][:rows]
        assert got[n].dtype == want[n].dtype and torch.equal(got[n], want[n]), n
    assert bool((got["dgamma_next"] == 0).all()) == (absent == "dx_next")
