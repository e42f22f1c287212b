"""GPU tests of the border and its norm with more tokens than one workgroup each: sizes whose threads, one
row after another, would pass the 2^32 of a launch, and workgroups that take several turns. A row's result
does not depend on which workgroup takes it, so a long call equals calls over its pieces bit for bit; the
pieces are held to float64."""
import pytest
import torch

import routing_permute_grouped_amd as rpg
from tests import _block_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *n: torch.randn(*n, device="cuda", generator=g)


@pytest.mark.parametrize("T", [1 << 26, (1 << 26) + 5])
def test_more_threads_than_a_launch_has(T):
    """T rows of 64 values at 64 threads a row are 2^32 threads and more; the rows repeat every P."""
    D, P = 64, 4099
    rn = gen(1)
    base, gp, gn = rn(P, D).to(BF16), (1 + 0.1 * rn(D)).to(BF16), (1 + 0.1 * rn(D)).to(BF16)
    want, wstd = rpg.moe_norm(base, gn)
    x, dx, r, rel = R.norm(base.double(), torch.zeros(P, D, dtype=torch.float64, device="cuda"), gn.double(), 1e-6)
    R.within(want, x, dx + R.HALF[BF16] * (x.abs() + dx) + R.TINY, "x")
    rep = T // P
    rows = torch.empty(T, D, dtype=BF16, device="cuda")
    rows[:rep * P].view(rep, P, D).copy_(base)
    rows[rep * P:] = base[:T - rep * P]

    def same(got, one):
        assert bool((got[:rep * P].view(rep, *one.shape) == one).all()) and torch.equal(got[rep * P:], one[:T - rep * P])

    got, rstd = rpg.moe_norm(rows, gn)
    same(got, want)
    same(rstd, wstd)
    del got, rstd
    dst = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
    w = torch.full((T, 1), 0.5, device="cuda")
    kw = dict(gamma_post=gp, gamma_next=gn, scale=0.75)
    one = rpg.moe_combine_norm(base, base, dst[:P], w[:P], **kw)
    R.within(one["out"], *R.border(base, base, dst[:P], w[:P], **kw)["out"], "out")
    long = rpg.moe_combine_norm(rows, rows, dst, w, **kw)
    for n in one:
        same(long[n], one[n])


@pytest.mark.parametrize("T,D,dt", [((1 << 23) + 5, 64, BF16), ((1 << 23) + 5, 64, F32), ((1 << 22) + 3, 2048, BF16), ((1 << 21) + 5, 4096, BF16),
                                    ((1 << 21) + 5, 4096, F32), ((1 << 22) + 3, 4160, BF16)])
def test_several_turns_a_workgroup(T, D, dt):
    """Past 2^21 workgroups, with one to eight waves a token; the rows repeat every P."""
    print(T, D, dt, flush=True)
    P, k = 1021, 2
    rn = gen(2)
    resid, y = rn(P, D).to(dt), rn(P, D).to(dt)
    gate, w = torch.rand(P, device="cuda"), torch.rand(P, k, device="cuda")
    dst = torch.randint(0, P, (P, k), device="cuda", dtype=torch.int32)
    dst[5, 0] = -1
    kw = dict(gamma_post=(1 + 0.1 * rn(D)).to(dt), gamma_next=(1 + 0.1 * rn(D)).to(dt), scale=0.75, eps=1e-5)
    one = rpg.moe_combine_norm(resid, y, dst, w, gate=gate, **kw)
    for n, (ref, tol) in R.border(resid, y, dst, w, gate=gate, **kw).items():
        if n in one:
            R.within(one[n], ref, tol, n)

    def long(t):
        r = torch.empty(T, *t.shape[1:], dtype=t.dtype, device="cuda")
        r[:T // P * P].view(-1, *t.shape).copy_(t)
        r[T // P * P:] = t[:T % P]
        return r

    def same(got, t):
        for a in range(0, T // P, 64):    # pieces: a comparison makes a mask of its size
            part = got[a * P:min(a + 64, T // P) * P].view(-1, *t.shape)
            assert bool((part == t).all()), a
        assert torch.equal(got[T // P * P:], t[:T % P])

    rows = long(resid)
    if D > 64:     # in place, so that two buffers of the size are enough
        got = rpg.moe_combine_norm(rows, y, long(dst), long(w), gate=long(gate), out=rows, **kw)
    else:
        got = rpg.moe_combine_norm(rows, y, long(dst), long(w), gate=long(gate), **kw)
        same(rows, resid)
        x, rstd = rpg.moe_norm(rows, kw["gamma_next"])
        want = rpg.moe_norm(resid, kw["gamma_next"])
        same(x, want[0])
        same(rstd, want[1])
    for n in one:
        same(got[n], one[n])
