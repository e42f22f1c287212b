"""GPU tests of MXFP4: quantisation, values, permute, the grouped products and the decode
product, against the plain definitions in float64.

Codes, scales, values, metadata: bit for bit. Products: operands are exact, so an element may
be off by its float32 sums and its one rounding. With S = sum |x||w| of the K terms, a sum in
float32 is off by at most K * 2^-23 * S (every addition by at most one unit of its last place,
whatever the matrix cores' order); silu has a slope of at most 1.1, so
  |h' - h| <= 1.1 K 2^-23 (S_a |b| + S_b |a| + S_a S_b K 2^-23) + (2^-8 + 2^-20) |h|
with the bf16 half step 2^-8 and 2^-20 for the float32 exponential and reciprocal."""
import numpy as np
import pytest
import torch

import routing_permute_grouped_amd as rpg
import workloads as W
from oracle import moe_oracle as orc
from oracle import mx_oracle as mx
from tests import _parity as P

pytestmark = pytest.mark.gpu

ROWS, KSTEPS = rpg.MOE_MX_ROWS, rpg.MOE_MX_KSTEPS
HALF = 2.0 ** -8      # bf16: half a step
FUN = 2.0 ** -20      # exponential and reciprocal in float32


def within(got, ref, tol, what):
    got = orc.values64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.2f} of the bound")


def h_bound(x, w1, w3):
    h, a, b, sa, sb = mx.fc1(x, w1, w3)
    ga, gb = x.shape[1] * 2.0 ** -23 * sa, x.shape[1] * 2.0 ** -23 * sb
    return h, 1.1 * (ga * np.abs(b) + gb * np.abs(a) + ga * gb) + (HALF + FUN) * np.abs(h)


def y_bound(h, w2):
    y = h @ w2.T
    return y, h.shape[1] * 2.0 ** -23 * (np.abs(h) @ np.abs(w2).T) + HALF * np.abs(y)


def bf16(a):
    return W.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


def scale_rows(s, layout):
    return mx.rows_of(s) if layout == KSTEPS else s


# ---- quantisation ---------------------------------------------------------------------

def special_rows(C):
    rng = np.random.default_rng(7)
    x = (rng.standard_normal((70, C)) * 10.0 ** rng.uniform(-30, 30, (70, 1))).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, :32] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4) * np.tile([1, -1], 16)
    x[3, :32] = 2.0 ** -133 * rng.integers(-9, 9, 32)          # below float32's normals
    x[4, :32] = 2.0 ** -126 * rng.integers(-9, 9, 32)
    x[5, :32] = np.float32(3.3e38) * rng.choice([-1, 1, 0.5, 0.125], 32)
    x[6, 5], x[6, 37], x[7, 3] = np.nan, np.inf, -np.inf
    x[8, :32] = 6.0 * 2.0 ** 10
    x[9, :32] = np.nextafter(np.float32(6.0), np.float32(7.0))
    x[10, :31] = 0.0
    x[10, 31] = 1.0
    return x


@pytest.mark.parametrize("layout", [ROWS, KSTEPS])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("C", [128, 640])
def test_quantize_bit_for_bit(dt, layout, C):
    x = special_rows(C)
    x = bf16(x) if dt == "bf16" else x
    q, s = rpg.moe_quantize_mxfp4(P.to_dev(x), layout=layout)
    torch.cuda.synchronize()
    rq, rs = mx.mx4_quantize(x)
    np.testing.assert_array_equal(scale_rows(P.to_host(s), layout), rs)
    np.testing.assert_array_equal(P.to_host(q), rq)


def test_quantize_every_bf16_pattern():
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16).reshape(-1, 32)
    q, s = rpg.moe_quantize_mxfp4(P.to_dev(bits))
    # and under the scale that the largest of each exponent's neighbours gives
    mixed = bits.reshape(64, 32, 32).transpose(0, 2, 1).reshape(-1, 32).copy()
    q2, s2 = rpg.moe_quantize_mxfp4(P.to_dev(mixed))
    torch.cuda.synchronize()
    for x, gq, gs in ((bits, q, s), (mixed, q2, s2)):
        rq, rs = mx.mx4_quantize(x)
        np.testing.assert_array_equal(P.to_host(gs), rs)
        np.testing.assert_array_equal(P.to_host(gq), rq)


@pytest.mark.parametrize("R,C,layout", [(1, 32, ROWS), (1, 128, KSTEPS), (3, 96, ROWS),
                                        (65, 128, KSTEPS), (64, 256, KSTEPS), (1, 65536, ROWS),
                                        (1, 65536, KSTEPS), (257, 2080, ROWS), (5000, 1408, KSTEPS)])
def test_quantize_and_values_at_the_edges(R, C, layout):
    rng = np.random.default_rng(R + C)
    x = bf16(rng.standard_normal((R, C)))
    q = torch.full((R * C // 2 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((R * C // 32 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    rpg.moe_quantize_mxfp4(P.to_dev(x), q=q, scales=s, layout=layout)
    out = torch.full((R * C + 64,), float("nan"), device="cuda")
    rpg.moe_dequantize_mxfp4(q[:R * C // 2].view(R, C // 2), s, out=out, layout=layout)
    torch.cuda.synchronize()
    rq, rs = mx.mx4_quantize(x)
    hq, hs = P.to_host(q), P.to_host(s)
    np.testing.assert_array_equal(hq[:R * C // 2].reshape(R, -1), rq)
    got = hs[:R * C // 32]
    got = scale_rows(got.reshape(C // 128, R, 4), layout) if layout == KSTEPS else got.reshape(R, -1)
    np.testing.assert_array_equal(got, rs)
    assert (hq[R * C // 2:] == 0xA5).all() and (hs[R * C // 32:] == 0xA5).all()
    ho = P.to_host(out)
    np.testing.assert_array_equal(ho[:R * C].reshape(R, C), mx.mx4_values(rq, rs))
    assert np.isnan(ho[R * C:]).all()


@pytest.mark.parametrize("layout", [ROWS, KSTEPS])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_values_of_every_code_and_scale(dt, layout):
    # 256 rows, one scale byte each; bytes of every code
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)
    dev = mx.words_of(s) if layout == KSTEPS else s
    q8 = np.tile(np.arange(256, dtype=np.uint8), (256, 2))
    q4 = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    v8 = rpg.moe_dequantize_mxfp8(P.to_dev(q8), P.to_dev(dev), layout=layout, dtype=dt)
    v4 = rpg.moe_dequantize_mxfp4(P.to_dev(q4), P.to_dev(dev), layout=layout, dtype=dt)
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        for got, ref in ((v8, mx.mx8_values(q8, s)), (v4, mx.mx4_values(q4, s))):
            ref = torch.from_numpy(ref).to(dt).double().numpy()
            np.testing.assert_array_equal(got.double().cpu().numpy(), ref)


def test_mxfp8_values_of_the_librarys_own_rows():
    x = bf16(np.random.default_rng(3).standard_normal((77, 256)))
    for layout in (ROWS, KSTEPS):
        q, s = rpg.moe_quantize_mxfp8(P.to_dev(x), layout=layout)
        v = rpg.moe_dequantize_mxfp8(q, s, layout=layout, dtype=torch.float32)
        torch.cuda.synchronize()
        rq, rs = orc.mx_quantize(x)
        np.testing.assert_array_equal(P.to_host(v), orc.mx_dequantize(rq, rs))


# ---- permute --------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,k,D,mt", [(1, 1, 1, 128, 16), (389, 8, 2, 640, 64),
                                        (5000, 64, 6, 128, 128), (300, 1024, 4, 256, 16)])
def test_permute_bit_for_bit(T, E, k, D, mt):
    rng = np.random.default_rng(T)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    idx[rng.random((T, k)) < 0.05] = -1
    xq = rng.integers(0, 256, (T, D // 2), dtype=np.uint8)
    xs = rng.integers(1, 255, (T, D // 32), dtype=np.uint8)
    g = rpg.moe_permute_mxfp4(P.to_dev(xq), P.to_dev(xs), P.to_dev(idx), E, mt)
    torch.cuda.synchronize()
    lay = orc.dispatch_layout(idx, E, mt)
    for key in ("counts", "offsets", "dst_row", "src_row", "tile_expert"):
        np.testing.assert_array_equal(P.to_host(g[key]), lay[key], err_msg=key)
    used = int(lay["offsets"][-1])
    np.testing.assert_array_equal(P.to_host(g["xq_perm"])[:used], orc.permute(xq, lay)[:used])
    np.testing.assert_array_equal(mx.rows_of(P.to_host(g["xs_perm"]))[:used],
                                  orc.permute(xs, lay)[:used])


# ---- the grouped products -------------------------------------------------------------

def segments(counts, mt, spare=0):
    """offsets, tile_expert and m_cap (with ``spare`` unused tiles) of given token counts."""
    seg = [-(-c // mt) * mt for c in counts]
    offs = np.concatenate([[0], np.cumsum(seg)]).astype(np.int32)
    m_cap = int(offs[-1]) + (spare + (offs[-1] == 0)) * mt
    te = np.repeat(np.arange(len(counts)), [s // mt for s in seg])
    te = np.concatenate([te, np.full(m_cap // mt - te.size, -1)]).astype(np.int32)
    return offs, te, m_cap


def rows4(rng, counts, offs, m_cap, K, spread=2.0):
    """Quantized rows of tokens; pad rows zero bytes; rows behind the last segment junk."""
    x = rng.standard_normal((m_cap, K)) * 2.0 ** rng.uniform(-spread, spread, (m_cap, 1))
    q, s = mx.mx4_quantize(bf16(x))
    tok = np.zeros(m_cap, dtype=bool)
    for e, c in enumerate(counts):
        tok[offs[e]:offs[e] + c] = True
    q[~tok], s[~tok] = 0, 0
    q[offs[-1]:], s[offs[-1]:] = 0x77, 255
    return q, s, tok


SHAPES = {   # counts, mt, K, N
    "one_row_one_step": ([1], 16, 128, 64),
    "odd_words": ([5, 0, 17], 16, 384, 192),
    "half_and_full_tiles": ([300, 128, 1, 256, 0, 257], 128, 640, 320),
    "fine": ([40, 0, 130, 7] * 16, 32, 256, 128),
    "many_experts": ([3, 0] * 100, 16, 128, 64),
    "long_k_few_tiles": ([200, 60], 64, 4224, 256),       # odd words, halved row blocks
    "longer_k_few_tiles": ([200, 60], 64, 6528, 256),     # the split last round, odd words
    "whole_row_blocks": ([300, 257] * 7 + [256, 129], 64, 384, 1088),   # tiles for half the card
    "halves_for_a_cut_in_two": ([2000], 64, 10240, 1408), # fc2: cut in five
    "tall": ([1500], 256, 256, 576),
}


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("fc", [1, 2])
@pytest.mark.parametrize("name", list(SHAPES))
def test_products(name, fc, split):
    counts, mt, K, N = SHAPES[name]
    P.log(f"[mx4] fc{fc} {name} split={split}")
    rng = np.random.default_rng(11)
    E = len(counts)
    offs, te, m_cap = segments(counts, mt, spare=2)
    q, s, tok = rows4(rng, counts, offs, m_cap, K)
    ws = [mx.quantize_weights(bf16(rng.standard_normal((E, N, K)) / np.sqrt(K)))
          for _ in range(2 if fc == 1 else 1)]
    dev = [t for wq, wsc in ws for t in (P.to_dev(wq), P.to_dev(mx.words_of(wsc.reshape(E * N, -1))))]
    wsp = rpg.grouped_workspace("cuda") if split else None
    aq, asw = P.to_dev(q), P.to_dev(mx.words_of(s))
    do, dt, dc = P.to_dev(offs), P.to_dev(te), P.to_dev(np.array(counts, dtype=np.int32))

    def call(**kw):
        out = P.poison(torch.empty((m_cap, N), dtype=torch.bfloat16, device="cuda"))
        if fc == 1:
            rpg.moe_grouped_fc1_swiglu_mxfp4(aq, asw, do, dt, *dev, mt, m_cap, h=out, workspace=wsp, **kw)
        else:
            rpg.moe_grouped_fc2_mxfp4(aq, asw, do, dt, *dev, mt, m_cap, y_perm=out, workspace=wsp, **kw)
        torch.cuda.synchronize()
        return P.to_host(out)

    got = call(counts=dc)
    np.testing.assert_array_equal(call(), got)            # pad rows are zero rows
    used = int(offs[-1])
    assert np.isnan(orc.values64(got[used:])).all()       # left as they were
    xv = mx.mx4_values(q[:used], s[:used])
    for e in range(E):
        r = slice(int(offs[e]), int(offs[e + 1]))
        if r.stop > r.start:
            w = [mx.mx4_values(wq[e], wsc[e]) for wq, wsc in ws]
            ref, tol = h_bound(xv[r], *w) if fc == 1 else y_bound(xv[r], *w)
            within(got[r], ref, tol, f"expert {e}")
            assert not orc.values64(got[r])[~tok[r]].any()
    # rows marked as pad rows are not read: junk there changes nothing
    junk = np.flatnonzero(~tok[:used])
    if junk.size:
        q[junk], s[junk] = 0xFF, 255
        aq, asw = P.to_dev(q), P.to_dev(mx.words_of(s))
        np.testing.assert_array_equal(call(counts=dc), got)


def test_product_counts_and_offsets_out_of_range_stay_inside():
    # counts past their segment and negative ones are clamped; offsets past m_cap only cut work
    mt, K, N, E = 16, 128, 64, 3
    rng = np.random.default_rng(2)
    offs, te, m_cap = segments([16, 16, 16], mt)
    q, s, _ = rows4(rng, [16] * 3, offs, m_cap, K)
    wq, wsc = mx.quantize_weights(bf16(rng.standard_normal((E, N, K))))
    args = (P.to_dev(q), P.to_dev(mx.words_of(s)))
    w = (P.to_dev(wq), P.to_dev(mx.words_of(wsc.reshape(E * N, -1))))

    def call(o, c):
        out = P.poison(torch.empty((m_cap, N), dtype=torch.bfloat16, device="cuda"))
        rpg.moe_grouped_fc2_mxfp4(*args, P.to_dev(np.array(o, dtype=np.int32)), P.to_dev(te), *w, mt,
                                  m_cap, y_perm=out, counts=P.to_dev(np.array(c, dtype=np.int32)))
        torch.cuda.synchronize()
        return P.to_host(out)

    full = call(offs, [16, 16, 16])
    np.testing.assert_array_equal(call(offs, [99, 16, 1 << 30]), full)
    cut = call(offs, [16, -5, 16])
    assert not orc.values64(cut[16:32]).any()
    np.testing.assert_array_equal(cut[32:], full[32:])
    np.testing.assert_array_equal(call([0, 16, 32, 1 << 30], [16] * 3), full)


def test_a_nan_block_stays_in_its_row_and_its_column():
    mt, K, N = 16, 384, 128
    rng = np.random.default_rng(3)
    offs, te, m_cap = segments([20], mt)
    q, s, tok = rows4(rng, [20], offs, m_cap, K, spread=0)
    wq, wsc = mx.quantize_weights(bf16(rng.standard_normal((1, N, K))))
    s[3, 11] = 255           # row 3, the last block
    wsc[0, 70, 0] = 255      # column 70, the first block
    y = rpg.moe_grouped_fc2_mxfp4(P.to_dev(q), P.to_dev(mx.words_of(s)), P.to_dev(offs), P.to_dev(te),
                                  P.to_dev(wq), P.to_dev(mx.words_of(wsc[0])), mt,
                                  counts=P.to_dev(np.array([20], dtype=np.int32)))
    torch.cuda.synchronize()
    nan = np.isnan(orc.values64(P.to_host(y)))
    assert nan[3].all() and nan[:20, 70].all()
    nan[3], nan[:, 70] = False, False
    assert not nan.any()


@pytest.mark.parametrize("fc,K", [(1, 384), (2, 384), (1, 6528), (2, 6528)])
def test_pad_rows_are_zeros_beside_a_nan_block(fc, K):
    counts, mt, N = [20, 150, 1], 64, 128
    rng = np.random.default_rng(4)
    offs, te, m_cap = segments(counts, mt)
    q, s, tok = rows4(rng, counts, offs, m_cap, K)
    wq, wsc = mx.quantize_weights(bf16(rng.standard_normal((3, N, K))))
    wsc[:, 70, 0] = 255
    w = (P.to_dev(wq), P.to_dev(mx.words_of(wsc.reshape(3 * N, -1)))) * (3 - fc)
    call = rpg.moe_grouped_fc1_swiglu_mxfp4 if fc == 1 else rpg.moe_grouped_fc2_mxfp4
    y = call(P.to_dev(q), P.to_dev(mx.words_of(s)), P.to_dev(offs), P.to_dev(te), *w, mt,
             workspace=rpg.grouped_workspace("cuda"), counts=P.to_dev(np.array(counts, dtype=np.int32)))
    torch.cuda.synchronize()
    y = orc.values64(P.to_host(y))
    assert np.isnan(y[tok][:, 70]).all() and not y[~tok].any()


# ---- decode ---------------------------------------------------------------------------

DECODE = {   # counts, cap, D, F
    "one_token": ([0, 0, 1, 0], 16, 256, 128),
    "nothing": ([0, 0], 16, 128, 128),
    "slab16": ([16, 3, 0, 9], 16, 384, 640),
    "slab32": ([32, 17, 5], 32, 1408, 256),
    "slab64": ([64, 33, 49, 0, 1], 64, 512, 384),
    "slab128": ([128, 81, 97, 113, 65, 2], 128, 256, 384),
    "two_and_a_bit_slabs": ([272, 129, 256], 272, 256, 128),
    "more_than_the_slab": ([40, -3, 100], 16, 128, 128),
    "many_experts": ([2, 0, 1] * 40, 16, 128, 256),
    "odd_chunks": ([7], 16, 1152, 1408),
    # more items of 64 columns than the card has compute units
    "many_items": ([3, 0, 20, 16, 32, 1] * 11, 32, 384, 512),
    "many_items_tall": ([16, 40, 17, 64, 0, 33] * 11, 64, 384, 512),
    "most_experts": ([0] * 511 + [5, 0, 17] + [1, 0, 0] * 170, 32, 128, 128),
}


@pytest.mark.parametrize("name", list(DECODE))
def test_decode(name):
    counts, cap, D, F = DECODE[name]
    P.log(f"[mx4] decode {name}")
    rng = np.random.default_rng(13)
    E = len(counts)
    x = bf16(rng.standard_normal((E * cap, D)))
    n = np.clip(counts, 0, cap)
    for e in range(E):     # rows behind the count hold what an earlier batch left
        x[e * cap + n[e]:(e + 1) * cap] = bf16(np.nan)
    w = {k: mx.quantize_weights(bf16(rng.standard_normal(sh) / np.sqrt(sh[2])))
         for k, sh in (("w1", (E, F, D)), ("w3", (E, F, D)), ("w2", (E, D, F)))}
    dev = [t for k in ("w1", "w3", "w2") for t in
           (P.to_dev(w[k][0]), P.to_dev(mx.words_of(w[k][1].reshape(E * w[k][1].shape[1], -1))))]
    h = P.poison(torch.empty((E * cap, F), dtype=torch.bfloat16, device="cuda"))
    y = P.poison(torch.empty((E * cap, D), dtype=torch.bfloat16, device="cuda"))
    rpg.moe_grouped_swiglu_masked_mxfp4(P.to_dev(x), P.to_dev(np.array(counts, dtype=np.int32)), *dev,
                                        cap, h=h, y=y)
    torch.cuda.synchronize()
    h, y = P.to_host(h), P.to_host(y)
    for e in range(E):
        r = slice(e * cap, e * cap + n[e])
        left = slice(r.stop, (e + 1) * cap)
        assert np.isnan(orc.values64(h[left])).all() and np.isnan(orc.values64(y[left])).all()
        if n[e]:
            v = {k: mx.mx4_values(w[k][0][e], w[k][1][e]) for k in w}
            ref, tol = h_bound(orc.values64(x[r]), v["w1"], v["w3"])
            within(h[r], ref, tol, f"h of expert {e}")
            ref, tol = y_bound(orc.values64(h[r]), v["w2"])   # from the stored h
            within(y[r], ref, tol, f"y of expert {e}")


def test_decode_nan_block_stays_in_its_column():
    E, cap, D, F = 1, 16, 256, 128
    rng = np.random.default_rng(14)
    w1, w2 = (mx.quantize_weights(bf16(rng.standard_normal(s))) for s in ((E, F, D), (E, D, F)))
    w1[1][0, 40, 1] = 255
    wd = [P.to_dev(w1[0]), P.to_dev(mx.words_of(w1[1][0])), P.to_dev(w1[0]), P.to_dev(mx.words_of(w1[1][0])),
          P.to_dev(w2[0]), P.to_dev(mx.words_of(w2[1][0]))]
    h, _ = rpg.moe_grouped_swiglu_masked_mxfp4(P.to_dev(bf16(rng.standard_normal((cap, D)))),
                                               P.to_dev(np.array([cap], dtype=np.int32)), *wd, cap)
    torch.cuda.synchronize()
    nan = np.isnan(orc.values64(P.to_host(h)))
    assert nan[:, 40].all() and nan.sum() == cap


# ---- the layers -----------------------------------------------------------------------

LAYERS = {
    "dense8": W.shrink(W.preset("dense8_bf16"), T=300, D=512, F=640),
    "fine64_shared2": W.shrink(W.preset("fine64_shared2_bf16"), T=389, D=384, F=256, F_shared=192),
    "skew32_mt32": W.shrink(W.preset("skew32_zipf_bf16"), T=500, D=256, F=384, m_tile=32),
    "etp_shard32": W.shrink(W.preset("etp_shard32_bf16"), D=512, F=256, poisson_mean=40.0),
}


def layer_inputs(cfg):
    inp = W.generate(cfg, seed=0)
    d = {n: P.to_dev(a) for n, a in inp.items() if isinstance(a, np.ndarray)}
    kw = dict(topk_idx=d["topk_idx"], topk_w=d["topk_w"]) if "topk_idx" in d else \
        dict(wg=d["wg"], bias=d.get("bias"))
    if "ws1" in d:
        kw["shared"] = rpg.SharedExperts.from_stacked(d["ws1"], d["ws3"], d["ws2"])
    return inp, d, kw


@pytest.mark.parametrize("name", list(LAYERS))
def test_layer(name):
    # h and out against the whole chain in float64 under the layer tolerance: a code of the
    # quantized h may fall to the other side of a border, one term in F of a sum
    inp, d, kw = layer_inputs(LAYERS[name])
    cfg = inp["cfg"]
    P.log(f"[mx4] layer {name}")
    mw = rpg.Mx4Weights.quantize(d["w1"], d["w3"], d["w2"])
    g = rpg.moe_layer_mxfp4(d["x"], mw, cfg.k, cfg.m_tile, **kw)
    torch.cuda.synchronize()
    ref = mx.forward_mxfp4(inp, cfg.k, cfg.m_tile)
    for key in ("xq", "xs", "counts", "offsets", "dst_row", "src_row"):
        np.testing.assert_array_equal(P.to_host(g[key]), ref[key], err_msg=key)
    used = int(ref["offsets"][-1])
    assert P.rel_err(P.to_host(g["h"])[:used], ref["h"][:used]) <= P.TOL["bf16"]
    assert P.rel_err(P.to_host(g["out"]), ref["out"]) <= P.TOL["bf16"]


@pytest.mark.parametrize("name", ["dense8", "fine64_shared2", "etp_shard32"])
def test_masked_layer(name):
    inp, d, kw = layer_inputs(LAYERS[name])
    cfg = inp["cfg"]
    cap = 48    # some slots are dropped
    P.log(f"[mx4] masked layer {name}")
    mw = rpg.Mx4Weights.quantize(d["w1"], d["w3"], d["w2"])
    g = rpg.moe_layer_masked_mxfp4(d["x"], mw, cfg.k, cap, **kw)
    torch.cuda.synchronize()
    vals = {n: np.stack([mx.mx4_values(*mx.mx4_quantize(inp[n][e])) for e in range(cfg.E)])
            for n in ("w1", "w3", "w2")}
    idx = P.to_host(g["topk_idx"])
    lay = orc.masked_layout(idx, cfg.E, cap)
    for key in ("counts", "dst_row"):
        np.testing.assert_array_equal(P.to_host(g[key]), lay[key], err_msg=key)
    _, y = mx.masked_mxfp4(orc.permute(inp["x"], lay), lay["counts"], cap, vals["w1"], vals["w3"], vals["w2"])
    sh = orc.shared_experts(inp["x"], inp["ws1"], inp["ws3"], inp["ws2"], "bf16") if "ws1" in inp else None
    out = orc.combine(y, lay["dst_row"], P.to_host(g["topk_w"]).astype(np.float64), "bf16", sh)
    assert P.rel_err(P.to_host(g["out"]), out) <= P.TOL["bf16"]


@pytest.mark.parametrize("T", [1, 2, 129])
def test_a_token_gives_the_same_bits_alone_and_in_a_batch(T):
    inp, d, kw = layer_inputs(LAYERS["dense8"])
    cfg = inp["cfg"]
    mw = rpg.Mx4Weights.quantize(d["w1"], d["w3"], d["w2"])
    full = rpg.moe_layer_mxfp4(d["x"], mw, cfg.k, cfg.m_tile, split_k=False, **kw)
    few = rpg.moe_layer_mxfp4(d["x"][:T].contiguous(), mw, cfg.k, cfg.m_tile, split_k=False, **kw)
    assert torch.equal(few["topk_idx"], full["topk_idx"][:T])
    assert torch.equal(few["out"], full["out"][:T])


# ---- sizes past 32 bits ---------------------------------------------------------------

def same_bits(a, b):
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def codes_on_device(*shape):
    """Random code bytes and words of middling scales for rows of shape[-1] bytes."""
    q = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda")
    rows = q.numel() // shape[-1]
    return q, torch.randint(118, 122, (shape[-1] // 64, rows, 4), dtype=torch.uint8, device="cuda")


def test_rows_past_32_bits():
    R, C = 70000, 65536          # 4.6e9 values
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, C), device="cuda").to(torch.bfloat16)
    for layout in (ROWS, KSTEPS):
        q, s = rpg.moe_quantize_mxfp4(x, layout=layout)
        ref = rpg.moe_quantize_mxfp4(x[-3:].contiguous(), layout=layout)
        assert torch.equal(q[-3:], ref[0]) and not q[:3].any()
        assert torch.equal(s[-3:] if layout == ROWS else s[:, -3:], ref[1])
        v = rpg.moe_dequantize_mxfp4(q, s, layout=layout)
        assert torch.equal(v[-3:], rpg.moe_dequantize_mxfp4(*ref, layout=layout)) and not v[:3].any()
        del q, s, v


def test_weights_past_32_bits():
    # 160 experts, 4.7e9 bytes of codes a matrix: the last expert's rows give the bits its weights
    # give alone
    E, D, F, cap = 160, 4096, 14336, 16
    w1q, w1s = codes_on_device(E, F, D // 2)
    w2q, w2s = codes_on_device(E, D, F // 2)
    last = lambda q, s: (q[-1:].contiguous(), s[:, -q.shape[1]:].contiguous())  # noqa: E731
    one1, one2 = last(w1q, w1s), last(w2q, w2s)
    x = torch.randn((E * cap, D), device="cuda").to(torch.bfloat16)
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    counts[-1] = 5
    h, y = rpg.moe_grouped_swiglu_masked_mxfp4(x, counts, w1q, w1s, w1q, w1s, w2q, w2s, cap)
    h1, y1 = rpg.moe_grouped_swiglu_masked_mxfp4(x[-cap:].contiguous(), counts[-1:].contiguous(), *one1,
                                                 *one1, *one2, cap)
    assert torch.equal(h[-cap:][:5], h1[:5]) and torch.equal(y[-cap:][:5], y1[:5])
    assert torch.isfinite(y1[:5].float()).all() and y1[:5].any()
    xq, xs = rpg.moe_quantize_mxfp4(x[:cap].contiguous(), layout=KSTEPS)
    hq, hs = rpg.moe_quantize_mxfp4(h1, layout=KSTEPS)
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offs[-1] = cap
    te = torch.full((1,), E - 1, dtype=torch.int32, device="cuda")
    offs1, te1 = offs[-2:].contiguous(), torch.zeros_like(te)
    a = rpg.moe_grouped_fc1_swiglu_mxfp4(xq, xs, offs, te, w1q, w1s, w1q, w1s, cap)
    same_bits(a, rpg.moe_grouped_fc1_swiglu_mxfp4(xq, xs, offs1, te1, *one1, *one1, cap))
    b = rpg.moe_grouped_fc2_mxfp4(hq, hs, offs, te, w2q, w2s, cap)
    # rows behind the five hold whatever was in memory, NaN perhaps
    same_bits(b, rpg.moe_grouped_fc2_mxfp4(hq, hs, offs1, te1, *one2, cap))


# ---- how calls are made ---------------------------------------------------------------

def test_calls_on_other_streams_and_two_at_once():
    inp, d, kw = layer_inputs(LAYERS["dense8"])
    cfg = inp["cfg"]
    mw = rpg.Mx4Weights.quantize(d["w1"], d["w3"], d["w2"])
    idx, w, _ = rpg.moe_route(d["x"], d["wg"], cfg.k)
    kw = dict(topk_idx=idx, topk_w=w)
    ref = rpg.moe_layer_mxfp4(d["x"], mw, cfg.k, cfg.m_tile, **kw)
    refm = rpg.moe_layer_masked_mxfp4(d["x"], mw, cfg.k, 96, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append((rpg.moe_layer_mxfp4(d["x"], mw, cfg.k, cfg.m_tile, **kw)["out"],
                         rpg.moe_layer_masked_mxfp4(d["x"], mw, cfg.k, 96, **kw)["out"]))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, ref["out"]) and torch.equal(b, refm["out"])


def test_graph_replays_equal_the_eager_layers():
    inp, d, kw = layer_inputs(LAYERS["dense8"])
    cfg = inp["cfg"]
    mw = rpg.Mx4Weights.quantize(d["w1"], d["w3"], d["w2"])
    x = d["x"].clone()
    xs = [d["x"], d["x"].flip(0).contiguous(), (d["x"].float() * 0.5).to(torch.bfloat16)]

    def step():
        return (rpg.moe_layer_mxfp4(x, mw, cfg.k, cfg.m_tile, **kw)["out"],
                rpg.moe_layer_masked_mxfp4(x, mw, cfg.k, 96, **kw)["out"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for v in xs + xs[::-1]:
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
