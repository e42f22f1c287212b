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


@pytest.mark.parametrize("T", [1 << 26, (1 << 26) + 5])
def test_permute_and_combine(T):
    E, mt = 3, 16
    base, x = rows(T)
    idx = (torch.arange(T, device="cuda") % 7 % 4).to(torch.int32)[:, None].contiguous()
    idx[idx == 3] = -1
    p = rpg.moe_permute(x, idx, E, mt)
    counts = torch.stack([(idx == e).sum() for e in range(E)])
    seg = (counts + mt - 1) // mt * mt
    start = torch.cumsum(seg, 0) - seg
    assert torch.equal(p["counts"].long(), counts) and torch.equal(p["offsets"][:E].long(), start) and int(p["dev_err"]) == 0
    dst = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    for e in range(E):
        at = (idx[:, 0] == e).nonzero()[:, 0]
        dst[at] = (start[e] + torch.arange(at.numel(), device="cuda")).to(torch.int32)
        assert torch.equal(p["src_row"][start[e]:start[e] + counts[e]].long(), at)
        assert torch.equal(p["x_perm"][start[e]:start[e] + counts[e]], x[at])
        assert not bool(p["x_perm"][start[e] + counts[e]:start[e] + seg[e]].any())
        del at
    assert torch.equal(p["dst_row"][:, 0], dst)
    # combine takes the rows back, weighted
    w = torch.full((T, 1), 0.5, device="cuda")
    out = rpg.moe_combine(p["x_perm"], p["dst_row"], w, shared=x, m_cap=p["m_cap"])
    gone = dst < 0
    assert torch.equal(out[gone], x[gone])
    # half of a value is exact, the sum with the shared row is rounded once
    one = (base.float() * 0.5 + base.float()).to(torch.bfloat16)
    assert bool(torch.where(gone[:, None], True, out == long(one, T)).all())
