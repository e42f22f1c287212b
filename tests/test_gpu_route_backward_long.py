"""GPU tests of the router's backward over more tokens than its first kernel has workgroups for at one
workgroup for 32 along one dimension: past its 2^32 threads, and past the 2^16 workgroups that it takes."""
import pytest
import torch

import routing_permute_grouped_amd as rpg
from tests import _block_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def test_more_threads_than_a_launch_has():
    """Past 2^27 tokens. Only a few tokens have a gradient of their weights: the others' dlogits are exact
    zeros and add nothing to the sums, whose bounds are then those of the few."""
    T, E, k, D = (1 << 27) + 37, 2, 1, 64
    at = torch.tensor([0, 31, 32, 131071, 131072, (1 << 26) + 1, (1 << 27) - 1, 1 << 27, T - 1], device="cuda")
    n = at.numel()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = torch.ones(T, D, dtype=BF16, device="cuda")
    x[at] = rn(n, D).to(BF16)
    wg = (rn(E, D) / 8).to(BF16)
    logits, idx, dw = torch.zeros(T, E, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    logits[at], dw[at] = rn(n, E), rn(n, k)
    got = rpg.moe_route_backward(dw, idx, logits, x, wg)
    want = R.route_backward(dw[at], idx[at], logits[at], x[at], wg)
    for name in ("dlogits", "dx"):
        R.within(got[name][at], *want[name], name)
        got[name][at] = 0
        assert int(torch.count_nonzero(got[name])) == 0, name
    for name in ("dwg", "dbias"):
        R.within(got[name], *want[name], name)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("E,k,renorm", [(3, 2, False), (40, 4, True), (100, 3, False), (300, 2, True)])
def test_more_workgroups_than_one_dimension_takes(E, k, renorm, dt):
    """Past 2^16 workgroups of 32 tokens. A token's dlogits and dx are those of a call over its piece, bit
    for bit; the sums over the tokens are taken where few of them have a gradient of their weights (the
    others add exact zeros), so that their bounds are those of the few."""
    T, D = (1 << 21) + 4099, 64
    print(E, k, renorm, dt, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    logits = rn(T, E)
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    idx[torch.rand(T, device="cuda", generator=g) < 0.1] = -1
    x, wg = rn(T, D).to(dt), (rn(E, D) / 8).to(dt)
    a = dict(dtopk_w=rn(T, k), topk_idx=idx, logits=logits, x=x, wg=wg, renorm=renorm, dlogits_add=0.1 * rn(T, E), dx_add=rn(T, D).to(dt))
    got = rpg.moe_route_backward(**a)
    for b in (0, (1 << 21) - 1024, T - 1501):
        s = slice(b, b + 2048)
        part = {n: t[s].contiguous() if isinstance(t, torch.Tensor) and n != "wg" else t for n, t in a.items()}
        one = rpg.moe_route_backward(**part)
        assert torch.equal(one["dlogits"], got["dlogits"][s]) and torch.equal(one["dx"], got["dx"][s])
        want = R.route_backward(**part)
        for n in ("dlogits", "dx"):
            R.within(one[n], *want[n], n)
    at = torch.cat([torch.arange(0, T, 9973), torch.arange((1 << 21) - 40, (1 << 21) + 40), torch.tensor([T - 1])]).unique().cuda()
    dw = torch.zeros_like(a["dtopk_w"])
    dw[at] = a["dtopk_w"][at]
    got = rpg.moe_route_backward(dw, idx, logits, x, wg, renorm=renorm)
    want = R.route_backward(dw[at], idx[at], logits[at], x[at], wg, renorm)
    for n in ("dwg", "dbias"):
        R.within(got[n], *want[n], n)
