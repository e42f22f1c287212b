"""GPU tests of the 4-bit products and of the checkpoint's GEMMs where every workgroup takes
several tiles one after the other: more than two rounds of 256 tiles of uneven segments (full,
half and padded tiles, the next tile's first loads under the last one's end), and whole rounds
followed by a last round that is cut over k. Element by element against 64-bit sums on the
GPU, with the bounds of the smaller tests:
  a float32 sum of K terms is off by at most K * 2^-23 * sum |x||w|; one rounding to bf16 by
  2^-8; the float32 exponential and reciprocal by 2^-20; a checkpoint code by half an e4m3
  step, 2^-4 of the value or 2^-10 of the block's power of two.
The 4-bit operands' values are the library's, which other tests compare bit for bit."""
import numpy as np
import pytest
import torch

import routing_permute_grouped_amd as rpg
from tests import _parity as P
from tests.test_gpu_mxfp4 import FUN, HALF, segments

pytestmark = pytest.mark.gpu

KSTEPS = rpg.MOE_MX_KSTEPS
UNEVEN = [300, 128, 1, 257, 0, 40, 256, 130]   # nine row blocks with segments of 32
BF = dict(dtype=torch.bfloat16, device="cuda")

# counts, m_tile, D (the checkpoint's k), F; nine blocks of UNEVEN times the column tiles
CKPT = {
    "rounds_ring": (UNEVEN * 8, 32, 192, 1984),             # 1152 tiles of fc1, 576 of the backward
    "rounds_many_experts": (UNEVEN * 8 + [3, 70], 32, 192, 1984),
    "rounds_tall": ([9000], 256, 128, 4096),
    "cut_ring": (UNEVEN * 3 + [90, 1, 33], 32, 1600, 2304),           # 30 blocks: 540 and 270 tiles
    "cut_many_experts": ([40] * 60 + [100, 3, 0, 128, 64, 1, 70], 32, 1600, 1024),   # 66: 528, 264
    "cut_tall": ([4300, 2900], 128, 1600, 2368),                      # 29: 551 and 290
}
MX4 = {   # counts, m_tile, K (odd numbers of 128), N
    "rounds": (UNEVEN * 8, 32, 384, 1984),
    "rounds_many_experts": (UNEVEN * 8 + [3, 70], 32, 640, 1984),
    "cut": (UNEVEN * 3 + [90, 1, 33], 32, 6272, 2304),
    "cut_tall": ([4300, 2900], 128, 6272, 2368),
}


def cases(shapes):
    """(name, with a workspace); without one too where it cuts tiles."""
    return [(n, split) for n in shapes for split in ((True, False) if n.startswith("cut") else (True,))]


def setup(counts, mt):
    offs, te, m_cap = segments(counts, mt, spare=2)
    tok = np.zeros(m_cap, dtype=bool)
    for e, c in enumerate(counts):
        tok[offs[e]:offs[e] + c] = True
    cnt = P.to_dev(np.array(counts, dtype=np.int32))
    return offs, P.to_dev(offs), P.to_dev(te), m_cap, P.to_dev(tok), cnt


def within(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off"


def experts(counts, offs):
    return ((e, slice(int(offs[e]), int(offs[e]) + c)) for e, c in enumerate(counts) if c)


def silu(a):
    return a * torch.sigmoid(a)


def h_bound(x, w1, w3):
    g = x.shape[1] * 2.0 ** -23
    a, b = x @ w1.T, x @ w3.T
    ga, gb = g * (x.abs() @ w1.abs().T), g * (x.abs() @ w3.abs().T)
    h = silu(a) * b
    return h, 1.1 * (ga * b.abs() + gb * a.abs() + ga * gb) + (HALF + FUN) * h.abs(), a, b, ga, gb


def poisoned(m_cap, cols):
    return P.poison(torch.empty((m_cap, cols), **BF))


def edges(t, tok, used, poison):
    """Pad rows are zeros, rows behind the last segment as they were."""
    assert not t[:used][~tok[:used]].any()
    rest = t[used:]
    assert rest.isnan().all() if poison is None else (rest == poison).all()


@pytest.mark.parametrize("name,split", cases(CKPT))
def test_save(name, split):
    counts, mt, D, F = CKPT[name]
    P.log(f"[tiles] save {name} split={split}")
    torch.manual_seed(51)
    offs, do, te, m_cap, tok, cnt = setup(counts, mt)
    x = torch.randn((m_cap, D), **BF)
    x[~tok] = 0
    x[int(offs[-1]):] = float("nan")
    w1, w3 = (torch.randn((len(counts), F, D), **BF) / D ** 0.5 for _ in range(2))
    h = poisoned(m_cap, F)
    q = torch.full((m_cap, 2 * F), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full((m_cap, F // 16), 255, dtype=torch.uint8, device="cuda")
    rpg.moe_grouped_fc1_swiglu_ckpt8(x, do, te, w1, w3, mt, m_cap, h=h, ab_codes=q, ab_scales=s, counts=cnt,
                                     workspace=rpg.grouped_workspace("cuda") if split else None)
    used = int(offs[-1])
    for t, p in ((h, None), (q, 0x7F), (s, 255)):
        edges(t, tok, used, p)
    v = rpg.moe_dequantize_mxfp8(q, s, dtype=torch.float32)
    power = torch.exp2(s.double() - 127)
    for e, r in experts(counts, offs):
        ref, tol, a, b, ga, gb = h_bound(x[r].double(), w1[e].double(), w3[e].double())
        within(h[r], ref, tol, f"h of expert {e}")
        sums, err = torch.cat([a, b], 1), torch.cat([ga, gb], 1)
        p = power[r]
        half = torch.maximum(2.0 ** -4 * (sums.abs() + err), 2.0 ** -10 * p.repeat_interleave(32, 1))
        within(v[r], sums, half + err, f"checkpoint of expert {e}")
        blocks = (p.shape[0], -1, 32)   # the smallest power of two that holds the block
        amax, slack = sums.abs().view(blocks).amax(2), err.view(blocks).amax(2)
        assert (amax - slack <= 448 * p).all() and (amax + slack > 224 * p).all()


@pytest.mark.parametrize("name,split", cases(CKPT))
def test_use(name, split):
    counts, mt, D, F = CKPT[name]
    P.log(f"[tiles] use {name} split={split}")
    torch.manual_seed(52)
    offs, do, te, m_cap, tok, cnt = setup(counts, mt)
    used, k = int(offs[-1]), 2
    d = torch.randn((m_cap, D), **BF)
    d[~tok] = 0
    d[used:] = float("nan")
    q, s = rpg.moe_quantize_mxfp8(torch.randn((m_cap, 2 * F), device="cuda") * torch.rand((m_cap, 1), device="cuda") * 4)
    ab = rpg.moe_dequantize_mxfp8(q, s, dtype=torch.float32)
    q[~tok], s[~tok] = 0x7F, 255   # not read
    w2 = torch.randn((len(counts), D, F), **BF) / F ** 0.5
    rows = torch.nonzero(tok).view(-1)
    T = -(-rows.numel() // k) + 3
    slot = torch.randperm(T * k, device="cuda")[:rows.numel()]
    dst = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    dst[slot] = rows.int()
    src = torch.full((m_cap,), -1, dtype=torch.int32, device="cuda")
    src[rows] = slot.int()
    tw = torch.rand((T, k), device="cuda")
    dab, hw = poisoned(m_cap, 2 * F), poisoned(m_cap, F)
    scratch = P.poison(torch.empty(rpg.moe_ckpt8_scratch_bytes(F, m_cap) // 4, device="cuda"))
    _, _, dtw = rpg.moe_grouped_dgrad_swiglu_ckpt8(
        d, do, te, w2, q, s, mt, m_cap, src_row=src, dst_row=dst.view(T, k), topk_w=tw, dab=dab, hw=hw, counts=cnt,
        scratch=scratch, workspace=rpg.grouped_workspace("cuda") if split else None)
    for t in (dab, hw):
        edges(t, tok, used, None)
    ref_w = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    tol_w = torch.zeros_like(ref_w)
    for e, r in experts(counts, offs):
        x, w = d[r].double(), w2[e].double()
        u, err = x @ w, D * 2.0 ** -23 * (x.abs() @ w.abs())
        a, b = ab[r, :F].double(), ab[r, F:].double()
        sg = torch.sigmoid(a)
        si, grad = a * sg, sg * (1 + a * (1 - sg))
        at = src[r].long()
        tr = tw.view(-1)[at].double()[:, None]
        da, db, hr = tr * u * b * grad, tr * u * si, tr * si * b
        within(dab[r, :F], da, HALF * da.abs() + err * (tr * b * grad).abs() + FUN * 2 * (tr * u * b).abs(), "da")
        within(dab[r, F:], db, HALF * db.abs() + err * (tr * si).abs() + FUN * db.abs(), "db")
        within(hw[r], hr, (HALF + FUN) * hr.abs(), "hw")
        h = (si * b).abs()
        ref_w[at] = (u * si * b).sum(1)
        tol_w[at] = (err * h).sum(1) + (F * 2.0 ** -23 + FUN) * (u.abs() * h).sum(1)
    within(dtw.view(-1), ref_w, tol_w, "dtopk_w")


@pytest.mark.parametrize("fc", [1, 2])
@pytest.mark.parametrize("name,split", cases(MX4))
def test_products(name, fc, split):
    counts, mt, K, N = MX4[name]
    P.log(f"[tiles] 4-bit fc{fc} {name} split={split}")
    torch.manual_seed(53)
    offs, do, te, m_cap, tok, cnt = setup(counts, mt)
    used, E = int(offs[-1]), len(counts)
    x = torch.randn((m_cap, K), **BF) * torch.exp2(torch.randint(-2, 3, (m_cap, 1), device="cuda"))
    xq, xs = rpg.moe_quantize_mxfp4(x, layout=KSTEPS)
    xv = rpg.moe_dequantize_mxfp4(xq, xs, layout=KSTEPS, dtype=torch.float32)
    xq[~tok], xs[:, ~tok] = 0x77, 255   # not read
    ws = [rpg.moe_quantize_mxfp4(torch.randn((E, N, K), **BF) / K ** 0.5, layout=KSTEPS) for _ in range(3 - fc)]
    wv = [rpg.moe_dequantize_mxfp4(q, s, layout=KSTEPS, dtype=torch.bfloat16) for q, s in ws]   # exact in bf16
    out = poisoned(m_cap, N)
    flat = [t for w in ws for t in w]
    kw = dict(counts=cnt, workspace=rpg.grouped_workspace("cuda") if split else None)
    if fc == 1:
        rpg.moe_grouped_fc1_swiglu_mxfp4(xq, xs, do, te, *flat, mt, m_cap, h=out, **kw)
    else:
        rpg.moe_grouped_fc2_mxfp4(xq, xs, do, te, *flat, mt, m_cap, y_perm=out, **kw)
    edges(out, tok, used, None)
    for e, r in experts(counts, offs):
        v, w = xv[r].double(), [t[e].double() for t in wv]
        if fc == 1:
            ref, tol = h_bound(v, *w)[:2]
        else:
            ref = v @ w[0].T
            tol = K * 2.0 ** -23 * (v.abs() @ w[0].abs().T) + HALF * ref.abs()
        within(out[r], ref, tol, f"expert {e}")
