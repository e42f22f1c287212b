"""GPU tests of the backward calls at a block's border and of the router's with a caller's buffers: exactly
the bytes that the workspace call names, full of NaN, and guards behind them. The results are those of the
call's own buffers bit for bit, and nothing behind a buffer is written."""
import pytest
import torch

import routing_permute_grouped_amd as rpg
from tests import _block_ref as R
from tests.test_gpu_route_backward import case

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
GUARD = 4096


class Buffers:
    """Buffers of bytes 0xFF (NaN in every type here) with a guard behind each."""

    def __init__(self):
        self.all = []

    def bytes(self, n):
        t = torch.full((n + GUARD,), 255, dtype=torch.uint8, device="cuda")
        self.all.append((t, n))
        return t[:n]

    def new(self, shape, dt):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dt).element_size()
        return self.bytes(n).view(dt).view(shape)

    def intact(self):
        return all(bool((t[n:] == 255).all()) for t, n in self.all)


def equal(got, want):
    assert sorted(got) == sorted(want)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("E", [1, 16, 33, 65, 97, 130, 300])
@pytest.mark.parametrize("T,D", [(1, 64), (31, 192), (1023, 320), (1025, 128), (2500, 704)])
def test_router_backward(T, D, E, dt):
    print(T, D, E, dt, flush=True)
    k = min(E, 4)
    a = case(T, E, k, D, dt, seed=31, add=T % 2 == 1, absent=T > 3)
    for renorm in (False, True):
        want = rpg.moe_route_backward(renorm=renorm, **a)
        b = Buffers()
        ws = b.bytes(rpg.moe_route_backward_workspace_bytes(dt, T, D, E))
        got = rpg.moe_route_backward(renorm=renorm, dx=b.new((T, D), dt), dwg=b.new((E, D), F32), workspace=ws, **a)
        torch.cuda.synchronize()
        equal(got, want)
        assert b.intact()
    with pytest.raises(rpg.MoEError):
        rpg.moe_route_backward(workspace=ws[:ws.numel() - 16], **a)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D", [64, 1088, 4096, 7168, 16384])
@pytest.mark.parametrize("T", [1, 255, 257, 700])
def test_border_and_norm_backward(T, D, dt):
    print(T, D, dt, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(32)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    u, out, dout, dx = (rn(T, D).to(dt) for _ in range(4))
    gp, gn = (1 + 0.1 * rn(D)).to(dt), (1 + 0.1 * rn(D)).to(dt)
    gate = torch.rand(T, device="cuda", generator=g)
    rstd = lambda t: torch.rsqrt(t.double().square().mean(1) + 1e-6).float()  # noqa: E731
    kw = dict(out=out, rstd_post=rstd(u), rstd_next=rstd(out), dx_next=dx, gate=gate, gamma_post=gp, gamma_next=gn, scale=0.75)
    need = rpg.moe_norm_workspace_bytes(T, D)
    b = Buffers()
    equal(rpg.moe_combine_norm_backward(dout, u, workspace=b.bytes(need), **kw), rpg.moe_combine_norm_backward(dout, u, **kw))
    x, r = rpg.moe_norm(out, gn, x=b.new((T, D), dt), rstd=b.new((T,), F32))
    want = rpg.moe_norm(out, gn)
    assert torch.equal(x, want[0]) and torch.equal(r, want[1])
    got = rpg.moe_norm_backward(dx, out, gn, r, dresid=dout, dr=b.new((T, D), dt), dgamma=b.new((D,), F32), workspace=b.bytes(need))
    want = rpg.moe_norm_backward(dx, out, gn, r, dresid=dout)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    assert b.intact()
    with pytest.raises(rpg.MoEError):
        rpg.moe_norm_backward(dx, out, gn, r, workspace=b.bytes(need - 16))


@pytest.mark.parametrize("T,D,dt", [(1111, 4096, BF16), (777, 5056, BF16), (1300, 8192, BF16), (601, 8256, BF16), (515, 16384, BF16), (3000, 2048, BF16),
                                    (1030, 4096, F32), (900, 4160, F32), (1111, 8192, F32), (515, 16384, F32)])
def test_border_backward_over_several_tokens_a_workgroup(T, D, dt):
    """Each body with several tokens in turn for every group of waves, and an odd end."""
    print(T, D, dt, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(33)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    u, out, dout, dx = rn(T, D).to(dt), (2 * rn(T, D)).to(dt), rn(T, D).to(dt), rn(T, D).to(dt)
    gp, gn = (1 + 0.1 * rn(D)).to(dt), (1 + 0.1 * rn(D)).to(dt)
    gate = torch.rand(T, device="cuda", generator=g)
    rstd = lambda t: torch.rsqrt(t.double().square().mean(1) + 1e-6).float()  # noqa: E731
    kw = dict(out=out, rstd_post=rstd(u), rstd_next=rstd(out), dx_next=dx, gate=gate, gamma_post=gp, gamma_next=gn, scale=0.75)
    got = rpg.moe_combine_norm_backward(dout, u, **kw)
    want = R.border_backward(dout, dx, u, out, gate, gp, gn, kw["rstd_post"], kw["rstd_next"], 0.75)
    assert sorted(got) == sorted(want)
    for n in want:
        R.within(got[n], *want[n], n)
    again = rpg.moe_combine_norm_backward(dout, u, **kw)
    equal(again, got)
    dr, dgamma = rpg.moe_norm_backward(dx, out, gn, kw["rstd_next"], dresid=dout)
    assert torch.equal(dr, got["dresid"]) and torch.equal(dgamma, got["dgamma_next"])


@pytest.mark.parametrize("E,k", [(4, 2), (70, 4)])
def test_router_weight_gradient_past_2_31_elements(E, k):
    """Rows of x past 2^31 elements. Only four tokens' rows are not zero, and zeros add nothing to the
    sums, so dwg is held to those four's bound (tests/test_block_bounds.py shows what that excludes)."""
    T, D = 33000, 65536
    x = torch.zeros(T, D, dtype=BF16, device="cuda")
    at = torch.tensor([0, 32767, 32768, T - 1], device="cuda")
    a = case(T, E, k, 64, BF16, seed=34)
    g = torch.Generator(device="cuda")
    g.manual_seed(35)
    x[at] = torch.randn(4, D, device="cuda", generator=g).to(BF16)
    wg = (torch.randn(E, D, device="cuda", generator=g) / 256).to(BF16)
    got = rpg.moe_route_backward(a["dtopk_w"], a["topk_idx"], a["logits"], x, wg)
    want = R.route_backward(a["dtopk_w"][at], a["topk_idx"][at], a["logits"][at], x[at], wg)
    R.within(got["dwg"], *want["dwg"], "dwg")
    R.within(got["dx"][at], *want["dx"], "dx")
