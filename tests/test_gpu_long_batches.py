"""GPU tests of routing, permute and combine with more tokens than one launch takes at 64 (permute, combine)
or 32 (routing) threads a token: 2^32 threads and more. Rows repeat every P, so a long call's results are
those of one period; positions are counted by torch."""
import pytest
import torch

import routing_permute_grouped_amd as rpg

pytestmark = pytest.mark.gpu

P, D = 4099, 64


def rows(T, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    base = torch.randn(P, D, device="cuda", generator=g).to(torch.bfloat16)
    return base, long(base, T)


def long(t, T):
    r = torch.empty(T, *t.shape[1:], dtype=t.dtype, device="cuda")
    r[:T // P * P].view(-1, *t.shape).copy_(t)
    r[T // P * P:] = t[:T % P]
    return r


def same(got, t):
    T = got.shape[0]
    assert bool((got[:T // P * P].view(-1, *t.shape) == t).all()) and torch.equal(got[T // P * P:], t[:T % P])


@pytest.mark.parametrize("E,k", [(4, 2), (16, 3)])
@pytest.mark.parametrize("T", [1 << 27, (1 << 27) + 5])
def test_route(T, E, k):
    base, x = rows(T)
    wg = torch.randn(E, D, device="cuda").to(torch.bfloat16) / 8
    want = rpg.moe_route(base, wg, k, want_logits=True)
    for got, one in zip(rpg.moe_route(x, wg, k, want_logits=True), want):
        same(got, one)
