"""GPU tests of the 8-bit checkpoint of fc1's pre-activations and of its backward, against the
definitions in float64.

Bounds, with S = sum |x||w| of a sum's K terms (float32 sums are off by at most K * 2^-23 * S):
  * a checkpoint value: half an e4m3 step of the quantized sum (2^-4 of it, or half the
    subnormal step 2^-10 of the block's 2^X) plus the sum's error;
  * dab = w u f(a) b ..., hw: one rounding to bf16 (half a step, 2^-8), u's sum error, and
    2^-20 for the float32 exponential, reciprocal and products;
  * dtopk_w = sum u h in float32: u's sum error times |h|, and F * 2^-23 * sum |u h|.
With the identity for w1 and w3 the sums are x itself, and codes and scales are bit for bit
the quantization of x."""
import numpy as np
import pytest
import torch

import routing_permute_grouped_amd as rpg
import workloads as W
from oracle import moe_oracle as orc
from oracle import mx_oracle as mx
from tests import _parity as P
from tests.test_gpu_mxfp4 import FUN, HALF, bf16, h_bound, segments, within

pytestmark = pytest.mark.gpu


def values(codes, scales):
    return mx.mx8_values(P.to_host(codes), P.to_host(scales))


def token_rows(rng, counts, offs, m_cap, K):
    x = bf16(rng.standard_normal((m_cap, K)))
    tok = np.zeros(m_cap, dtype=bool)
    for e, c in enumerate(counts):
        tok[offs[e]:offs[e] + c] = True
    x[~tok] = 0
    x[offs[-1]:] = bf16(np.nan)   # behind the last segment: never read
    return x, tok


def buffers(m_cap, F):
    b = dict(dtype=torch.bfloat16, device="cuda")
    u = dict(dtype=torch.uint8, device="cuda")
    return (P.poison(torch.empty((m_cap, F), **b)), torch.full((m_cap, 2 * F), 0x7F, **u),
            torch.full((m_cap, F // 16), 255, **u))


SHAPES = {   # counts, mt, D, F
    "one_row": ([1], 16, 64, 64),
    "half_and_full_tiles": ([300, 128, 1, 256, 0, 257], 128, 192, 320),
    "many_experts": ([3, 0] * 100, 16, 64, 128),              # above the ring's 64 experts
    "tall": ([1600], 256, 128, 192),                          # past the ring's row blocks
    "long_k_few_tiles": ([200, 60], 64, 4096, 256),           # the split last round
    "odd_mt32": ([40, 0, 130, 7] * 4, 32, 320, 448),
    "whole_row_blocks": ([300, 257] * 7 + [256, 129], 64, 192, 1088),   # tiles for half the card
    "cut_in_two": ([100] * 8, 64, 2560, 1408),                # the backward: in six
    "halves_for_a_cut_in_two": ([2000], 64, 2560, 1408),      # the backward: cut in five
    "narrow_with_a_rest": ([100, 7, 0, 250], 32, 128, 320),   # halved columns: 64 left over
    "narrow_many_experts": ([9, 0] * 40, 16, 64, 192),
    "shares_of_few_tiles": ([130, 90], 64, 4160, 448),
}


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("name", list(SHAPES))
def test_save(name, split):
    counts, mt, D, F = SHAPES[name]
    P.log(f"[ckpt8] save {name} split={split}")
    rng = np.random.default_rng(21)
    E = len(counts)
    offs, te, m_cap = segments(counts, mt, spare=2)
    x, tok = token_rows(rng, counts, offs, m_cap, D)
    w1, w3 = (bf16(rng.standard_normal((E, F, D)) / np.sqrt(D)) for _ in range(2))
    ws = rpg.grouped_workspace("cuda") if split else None
    args = (P.to_dev(x), P.to_dev(offs), P.to_dev(te), P.to_dev(w1), P.to_dev(w3), mt, m_cap)
    cnt = P.to_dev(np.array(counts, dtype=np.int32))
    h, q, s = buffers(m_cap, F)
    rpg.moe_grouped_fc1_swiglu_ckpt8(*args, h=h, ab_codes=q, ab_scales=s, workspace=ws, counts=cnt)
    h2, ab = P.poison(torch.empty_like(h)), torch.empty((m_cap, 2 * F), dtype=torch.bfloat16, device="cuda")
    rpg.moe_grouped_fc1_swiglu(*args, h2, ab=ab, workspace=ws, counts=cnt)
    torch.cuda.synchronize()
    used = int(offs[-1])
    if not split:   # the same sums and rounding as without a checkpoint
        assert torch.equal(h[:used], h2[:used])
    h, hq, hs = P.to_host(h), P.to_host(q), P.to_host(s)
    assert (hq[used:] == 0x7F).all() and (hs[used:] == 255).all() and np.isnan(orc.values64(h[used:])).all()
    v = mx.mx8_values(hq, hs)[:used]
    assert not hq[:used][~tok[:used]].any() and not hs[:used][~tok[:used]].any()
    assert not orc.values64(h[:used])[~tok[:used]].any()
    for e in range(E):
        r = slice(int(offs[e]), int(offs[e]) + counts[e])
        if not counts[e]:
            continue
        xe, we = orc.values64(x[r]), (orc.values64(w1[e]), orc.values64(w3[e]))
        ref, tol = h_bound(xe, *we)
        within(h[r], ref, tol, f"h of expert {e}")
        _, a, b, sa, sb = mx.fc1(xe, *we)
        sums, err = np.concatenate([a, b], 1), D * 2.0 ** -23 * np.concatenate([sa, sb], 1)
        power = np.repeat(np.ldexp(1.0, hs[r].astype(int) - 127), 32, axis=1)
        half = np.maximum(2.0 ** -4 * (np.abs(sums) + err), 2.0 ** -10 * power)
        within(v[r], sums, half + err, f"checkpoint of expert {e}")
        # the smallest power of two that holds the block
        amax = np.abs(sums).reshape(counts[e], -1, 32).max(axis=2)
        slack = err.reshape(counts[e], -1, 32).max(axis=2)
        p = power[:, ::32]
        assert (amax - slack <= 448 * p).all() and (amax + slack > 224 * p).all()


@pytest.mark.parametrize("rows,kernel_experts", [(300, 1), (40, 70)])
def test_codes_of_known_sums_bit_for_bit(rows, kernel_experts):
    # w1 = w3 = identity: the sums are x, so the checkpoint is the quantization of x, in both
    # pipelines (the second serves more than 64 experts)
    D = F = 256
    rng = np.random.default_rng(22)
    x = (rng.standard_normal((rows, D)) * 10.0 ** rng.uniform(-20, 20, (rows, 1))).astype(np.float32)
    x[0] = 0.0
    x[1, :32] = 448.0
    x[2, 32:64] = -449.0
    x[3, 64:96] = 2.0 ** -20 * rng.integers(-9, 9, 32)
    x[4, :] = 2.0 ** -6 * (1 + np.arange(256) / 16)       # ties of the 3-bit fraction
    x[4, ::32] = 448.0
    x[5, 5] = np.inf
    x[6, 40] = np.nan
    x = bf16(x)
    # 0 * inf in the other sums of the row makes every block of rows 5 and 6 NaN
    eye = np.broadcast_to(np.eye(F, D, dtype=np.float32), (kernel_experts, F, D))
    E = kernel_experts
    mt = 16
    counts = [rows] + [0] * (E - 1)
    offs, te, m_cap = segments(counts, mt)
    xp = np.zeros((m_cap, D), dtype=np.uint16)
    xp[:rows] = x
    w = P.to_dev(bf16(eye))
    _, q, s = rpg.moe_grouped_fc1_swiglu_ckpt8(P.to_dev(xp), P.to_dev(offs), P.to_dev(te), w, w, mt, m_cap)
    torch.cuda.synchronize()
    fin = np.ones(rows, dtype=bool)
    fin[5:7] = False
    rq, rs = orc.mx_quantize(x[fin])
    hq, hs = P.to_host(q)[:rows], P.to_host(s)[:rows]
    np.testing.assert_array_equal(hs[fin], np.tile(rs, 2))
    # -0 sums lose their sign in a sum that starts at +0; codes are compared as values
    np.testing.assert_array_equal(mx.mx8_values(hq[fin], hs[fin]), mx.mx8_values(np.tile(rq, 2), np.tile(rs, 2)))
    assert (hs[5:7] == 255).all() and not hq[5:7].any()


def use_case(counts, mt, D, F, seed=23, k=2):
    rng = np.random.default_rng(seed)
    E = len(counts)
    offs, te, m_cap = segments(counts, mt, spare=2)
    d, tok = token_rows(rng, counts, offs, m_cap, D)
    q, s = orc.mx_quantize(rng.standard_normal((m_cap, 2 * F)) * 2.0 ** rng.uniform(-2, 2, (m_cap, 1)))
    q[~tok], s[~tok] = 0, 0
    w2 = bf16(rng.standard_normal((E, D, F)) / np.sqrt(F))
    rows = np.flatnonzero(tok)
    T = -(-rows.size // k) + 3                       # some slots have no row
    dst = np.full(T * k, -1, dtype=np.int32)
    dst[rng.permutation(T * k)[:rows.size]] = rows
    src = np.full(m_cap, -1, dtype=np.int32)
    src[dst[dst >= 0]] = np.flatnonzero(dst >= 0)
    w = rng.random(T * k).astype(np.float32)
    w[dst == rows[0]] = 0.0                          # a weight of zero still has a gradient
    return dict(offs=offs, te=te, m_cap=m_cap, d=d, tok=tok, q=q, s=s, w2=w2, dst=dst.reshape(T, k),
                src=src, w=w.reshape(T, k), counts=counts, mt=mt, D=D, F=F)


def run_use(c, split, weights=True, counts=True, codes=None, scales=None):
    b = dict(dtype=torch.bfloat16, device="cuda")
    dab = P.poison(torch.empty((c["m_cap"], 2 * c["F"]), **b))
    hw = P.poison(torch.empty((c["m_cap"], c["F"]), **b))
    kw = {}
    if weights:
        kw = dict(src_row=P.to_dev(c["src"]), dst_row=P.to_dev(c["dst"]), topk_w=P.to_dev(c["w"]),
                  dtopk_w=P.poison(torch.empty(c["w"].shape, device="cuda")),
                  scratch=P.poison(torch.empty(rpg.moe_ckpt8_scratch_bytes(c["F"], c["m_cap"]) // 4,
                                               device="cuda")))
    if counts:
        kw["counts"] = P.to_dev(np.array(c["counts"], dtype=np.int32))
    if split:
        kw["workspace"] = rpg.grouped_workspace("cuda")
    q, s = c["q"] if codes is None else codes, c["s"] if scales is None else scales
    _, _, dtw = rpg.moe_grouped_dgrad_swiglu_ckpt8(
        P.to_dev(c["d"]), P.to_dev(c["offs"]), P.to_dev(c["te"]), P.to_dev(c["w2"]), P.to_dev(q),
        P.to_dev(s), c["mt"], c["m_cap"], dab=dab, hw=hw, **kw)
    torch.cuda.synchronize()
    return P.to_host(dab), P.to_host(hw), None if dtw is None else P.to_host(dtw)


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("name", list(SHAPES))
def test_use(name, weights, split):
    counts, mt, D, F = SHAPES[name]
    P.log(f"[ckpt8] use {name} weights={weights} split={split}")
    c = use_case(counts, mt, D, F)
    dab, hw, dtw = run_use(c, split, weights)
    offs, src, tok = c["offs"], c["src"], c["tok"]
    used = int(offs[-1])
    assert np.isnan(orc.values64(dab[used:])).all() and np.isnan(orc.values64(hw[used:])).all()
    assert not orc.values64(dab[:used])[~tok[:used]].any()
    assert not orc.values64(hw[:used])[~tok[:used]].any()
    ab = mx.mx8_values(c["q"], c["s"])
    ref_w, tol_w = np.zeros(c["w"].size), np.zeros(c["w"].size)
    for e in range(len(counts)):
        r = slice(int(offs[e]), int(offs[e]) + counts[e])
        if not counts[e]:
            continue
        d, w2 = orc.values64(c["d"][r]), orc.values64(c["w2"][e])
        a, b = ab[r, :F], ab[r, F:]
        w = c["w"].ravel()[src[r]].astype(np.float64) if weights else np.ones(counts[e])
        da, db, hr, dw = mx.ckpt8_rows(d, w2, a, b, w)
        u = d @ w2
        err = D * 2.0 ** -23 * (np.abs(d) @ np.abs(w2))
        fa, fb = np.abs(w[:, None] * b * orc.silu_grad(a)), np.abs(w[:, None] * orc.silu(a))
        # silu' itself cancels near its zero: its float32 terms are at most 1.3 in size
        within(dab[r, :F], da, HALF * np.abs(da) + err * fa + FUN * 2 * np.abs(w[:, None] * u * b), "da")
        within(dab[r, F:], db, HALF * np.abs(db) + err * fb + FUN * np.abs(db), "db")
        within(hw[r], hr, (HALF + FUN) * np.abs(hr), "hw")
        h = np.abs(orc.silu(a) * b)
        ref_w[src[r]] = dw
        tol_w[src[r]] = (err * h).sum(1) + (F * 2.0 ** -23 + FUN) * (np.abs(u) * h).sum(1)
    if weights:
        within(dtw.ravel(), ref_w, tol_w, "dtopk_w")
        assert not dtw.ravel()[c["dst"].ravel() < 0].any()
    else:
        assert dtw is None


@pytest.mark.parametrize("split", [True, False])
def test_pad_rows_of_the_checkpoint_are_not_read(split):
    c = use_case(*SHAPES["half_and_full_tiles"])
    q, s = c["q"].copy(), c["s"].copy()
    q[~c["tok"]], s[~c["tok"]] = 0x7F, 255
    for a, b in zip(run_use(c, split), run_use(c, split, codes=q, scales=s)):
        np.testing.assert_array_equal(a.view(np.uint8), b.view(np.uint8))


@pytest.mark.parametrize("name", ["half_and_full_tiles", "many_experts", "long_k_few_tiles"])
def test_pad_rows_are_zeros_beside_infinite_weights(name):
    counts, mt, D, F = SHAPES[name]
    c = use_case(counts, mt, D, F)
    w = orc.values64(c["w2"]).copy()
    w[:, 0, 0] = np.inf
    c["w2"] = bf16(w)
    dab, hw, _ = run_use(c, True)
    pad = ~c["tok"]
    pad[int(c["offs"][-1]):] = False
    assert not orc.values64(dab[pad]).any() and not orc.values64(hw[pad]).any()
    wt = P.to_dev(bf16(np.ascontiguousarray(w.transpose(0, 2, 1))))   # [E, F, D]
    x, _ = token_rows(np.random.default_rng(7), counts, c["offs"], c["m_cap"], D)
    h, q, s = rpg.moe_grouped_fc1_swiglu_ckpt8(
        P.to_dev(x), P.to_dev(c["offs"]), P.to_dev(c["te"]), wt, wt, mt, c["m_cap"],
        workspace=rpg.grouped_workspace("cuda"), counts=P.to_dev(np.array(counts, dtype=np.int32)))
    torch.cuda.synchronize()
    assert not orc.values64(P.to_host(h))[pad].any()
    assert not P.to_host(q)[pad].any() and not P.to_host(s)[pad].any()


def test_runs_repeat_bit_for_bit():
    c = use_case(*SHAPES["long_k_few_tiles"])
    first = run_use(c, True)
    for _ in range(3):
        for a, b in zip(first, run_use(c, True)):
            np.testing.assert_array_equal(a.view(np.uint8), b.view(np.uint8))


# ---- the layer ------------------------------------------------------------------------

LAYERS = {
    "dense8": W.shrink(W.preset("dense8_bf16"), T=300, D=256, F=320),
    "fine64_shared2": W.shrink(W.preset("fine64_shared2_bf16"), T=201, D=192, F=128, F_shared=192),
    "skew32_mt32": W.shrink(W.preset("skew32_zipf_bf16"), T=500, D=128, F=192, m_tile=32),
    "etp_shard32": W.shrink(W.preset("etp_shard32_bf16"), D=256, F=128, poisson_mean=30.0),
}


def layer_case(name):
    inp = W.generate(LAYERS[name], seed=0)
    cfg = inp["cfg"]
    d = {n: P.to_dev(a) for n, a in inp.items() if isinstance(a, np.ndarray)}
    kw = dict(topk_idx=d["topk_idx"], topk_w=d["topk_w"]) if "topk_idx" in d else \
        dict(wg=d["wg"], bias=d.get("bias"))
    if "ws1" in d:
        kw["shared"] = rpg.SharedExperts.from_stacked(d["ws1"], d["ws3"], d["ws2"])
    dout = bf16(np.random.default_rng(6).standard_normal(inp["x"].shape))
    return inp, cfg, d, kw, dout


@pytest.mark.parametrize("split_k", [True, False])
@pytest.mark.parametrize("name", list(LAYERS))
def test_layer_forward_and_backward(name, split_k):
    inp, cfg, d, kw, dout = layer_case(name)
    P.log(f"[ckpt8] layer {name} split_k={split_k}")
    fwd = rpg.moe_layer(d["x"], d["w1"], d["w3"], d["w2"], cfg.k, cfg.m_tile, split_k=split_k,
                        save_for_backward="mxfp8", **kw)
    plain = rpg.moe_layer(d["x"], d["w1"], d["w3"], d["w2"], cfg.k, cfg.m_tile, split_k=split_k,
                          save_for_backward=True, **kw)
    if not split_k:
        assert torch.equal(fwd["out"], plain["out"])
    assert not {"x_perm", "h", "y_perm", "ab", "shared_h", "shared_ab"} & set(fwd)
    g = rpg.moe_layer_backward(fwd, P.to_dev(dout), d["x"], d["w1"], d["w3"], d["w2"], cfg.m_tile,
                               shared=kw.get("shared"), split_k=split_k)
    torch.cuda.synchronize()
    used = int(P.to_host(fwd["offsets"])[-1])
    ck = values(fwd["ab_codes"], fwd["ab_scales"])
    ck[used:] = 0
    sck = values(fwd["shared_ab_codes"], fwd["shared_ab_scales"])[:inp["x"].shape[0]] \
        if "shared" in kw else None
    ref = mx.backward_ckpt8(inp, dout, cfg.k, cfg.m_tile, ck, sck)
    for key in ("dx", "dtopk_w", "dw1", "dw3", "dw2") + (("dws1", "dws3", "dws2") if sck is not None else ()):
        got = P.to_host(g[key])
        e = P.rel_err(got.reshape(np.asarray(ref[key]).shape), ref[key])
        assert np.isfinite(orc.values64(got)).all() and e <= P.TOL["bf16"], f"{key}: rel err {e:.3e}"


@pytest.mark.parametrize("T", [1, 2, 129])
def test_a_token_gives_the_same_bits_alone_and_in_a_batch(T):
    inp, cfg, d, kw, dout = layer_case("dense8")
    w, dd = (d["w1"], d["w3"], d["w2"]), P.to_dev(dout)
    got = []
    for n in (dout.shape[0], T):
        x = d["x"][:n].contiguous()
        fwd = rpg.moe_layer(x, *w, cfg.k, cfg.m_tile, split_k=False, save_for_backward="mxfp8", **kw)
        g = rpg.moe_layer_backward(fwd, dd[:n].contiguous(), x, *w, cfg.m_tile, split_k=False)
        got.append((fwd["out"], g["dx"], g["dtopk_w"]))
    for a, b in zip(*got):
        assert torch.equal(a[:T], b)


def test_checkpoint_past_32_bits():
    # 65536 rows of 2 * 65536 codes: the second expert's rows give the bits they give alone
    D, F, mt = 64, 65536, 16
    counts = [65536, 5]
    offs, te, m_cap = segments(counts, mt)
    b = dict(dtype=torch.bfloat16, device="cuda")
    x = torch.randn((m_cap, D), **b)
    x[-11:] = 0
    w1, w3 = (torch.randn((2, F, D), **b) / 8 for _ in range(2))
    w2 = torch.randn((2, D, F), **b) / 256
    cnt = P.to_dev(np.array(counts, dtype=np.int32))
    src = torch.arange(m_cap, dtype=torch.int32, device="cuda")
    src[-11:] = -1
    tw = torch.rand((counts[0] + 5, 1), device="cuda")
    dst = torch.arange(tw.shape[0], dtype=torch.int32, device="cuda").view(-1, 1)

    def run(x, offs, te, w1, w3, w2, cnt, src, dst, tw, m_cap):
        h, q, s = rpg.moe_grouped_fc1_swiglu_ckpt8(x, offs, te, w1, w3, mt, m_cap, counts=cnt)
        dab, hw, dtw = rpg.moe_grouped_dgrad_swiglu_ckpt8(x, offs, te, w2, q, s, mt, m_cap, src_row=src,
                                                          dst_row=dst, topk_w=tw, counts=cnt)
        return [t[-16:].clone() for t in (h, q, s, dab, hw)] + [dtw[-5:].clone()]

    two = run(x, P.to_dev(offs), P.to_dev(te), w1, w3, w2, cnt, src, dst, tw, m_cap)
    i32 = dict(dtype=torch.int32, device="cuda")
    src1 = torch.arange(mt, **i32)
    src1[5:] = -1
    one = run(x[-16:].contiguous(), torch.tensor([0, 16], **i32), torch.zeros(1, **i32), w1[1:].contiguous(),
              w3[1:].contiguous(), w2[1:].contiguous(), cnt[1:].contiguous(), src1,
              torch.arange(5, **i32).view(-1, 1), tw[-5:].contiguous(), mt)
    for a, b in zip(two, one):
        assert torch.equal(a, b)
    assert one[3].any() and torch.isfinite(one[3].float()).all()


def test_backward_without_the_weight_gradient():
    c = use_case(*SHAPES["half_and_full_tiles"])
    dab, hw, _ = run_use(c, False)
    t = [P.to_dev(c[n]) for n in ("d", "offs", "te", "w2", "q", "s", "src", "w")]
    cnt = P.to_dev(np.array(c["counts"], dtype=np.int32))
    E, D, F, m_cap = len(c["counts"]), c["D"], c["F"], c["m_cap"]
    b = dict(dtype=torch.bfloat16, device="cuda")
    o = (P.poison(torch.empty((m_cap, 2 * F), **b)), P.poison(torch.empty((m_cap, F), **b)))
    ptr = lambda x: x.data_ptr()  # noqa: E731
    st = rpg.lib.moe_grouped_dgrad_swiglu_ckpt8(
        ptr(t[0]), ptr(t[1]), ptr(cnt), ptr(t[2]), E, D, F, c["mt"], m_cap, ptr(t[3]), ptr(t[4]),
        ptr(t[5]), ptr(t[6]), None, ptr(t[7]), *c["w"].shape, ptr(o[0]), ptr(o[1]), None, None, 0, None,
        0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    used = int(c["offs"][-1])
    for got, ref in zip(o, (dab, hw)):
        np.testing.assert_array_equal(P.to_host(got)[:used].view(np.uint8), ref[:used].view(np.uint8))


def test_weight_gradient_against_differences():
    # <dout, out> of the layer is linear in the top-k weights: its difference quotient is
    # exact up to rounding. The outputs are bf16 (half a step 2^-8 of each, random in sign)
    # and the gradient comes from a checkpoint of half a step 2^-4 a value; both average
    # over D and F terms of random sign. The bound takes every rounding at its largest,
    # added in squares: sqrt(sum (2^-8 out dout)^2) * 2 / eps + sqrt(sum (2^-3 u h)^2) * 2.
    inp, cfg, d, kw, dout = layer_case("dense8")
    idx, w, _ = rpg.moe_route(d["x"], d["wg"], cfg.k)
    dd = P.to_dev(dout)
    run = lambda tw, save=False: rpg.moe_layer(d["x"], d["w1"], d["w3"], d["w2"], cfg.k, cfg.m_tile,  # noqa: E731
                                               topk_idx=idx, topk_w=tw, save_for_backward=save)
    fwd = run(w, "mxfp8")
    g = rpg.moe_layer_backward(fwd, dd, d["x"], d["w1"], d["w3"], d["w2"], cfg.m_tile)
    eps = 0.5
    lost = orc.forward(dict(inp, topk_idx=P.to_host(idx), topk_w=P.to_host(w)), cfg.k, cfg.m_tile, "bf16")
    dst = lost["dst_row"]
    d64 = orc.values64(dout)
    for j in range(cfg.k):
        up, down = w.clone(), w.clone()
        up[:, j] += eps
        down[:, j] -= eps
        ou, od = run(up)["out"].double(), run(down)["out"].double()
        diff = ((ou - od) * dd.double()).sum(1) / (2 * eps)
        scale = (torch.maximum(ou.abs(), od.abs()) * dd.double().abs()).square().sum(1).sqrt()
        tol = 2 * HALF * scale.cpu().numpy() / eps
        for t in range(0, w.shape[0], 37):
            e = int(P.to_host(idx)[t, j])
            h = lost["h"][dst[t, j]]
            u = d64[t] @ orc.values64(inp["w2"][e])
            bound = tol[t] + 2 * np.sqrt(((2.0 ** -3 * u * h) ** 2).sum())
            assert abs(float(diff[t]) - float(g["dtopk_w"][t, j])) <= bound


def test_scratch_of_a_call_on_another_stream_is_its_own():
    # the call's own scratch must not come back to this stream's allocator while it is in use
    c = use_case(*SHAPES["many_experts"])
    _, _, ref = run_use(c, False)
    args = [P.to_dev(c[n]) for n in ("d", "offs", "te", "w2", "q", "s")]
    kw = dict(src_row=P.to_dev(c["src"]), dst_row=P.to_dev(c["dst"]), topk_w=P.to_dev(c["w"]),
              counts=P.to_dev(np.array(c["counts"], dtype=np.int32)))
    n = rpg.moe_ckpt8_scratch_bytes(c["F"], c["m_cap"])
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        out = rpg.moe_grouped_dgrad_swiglu_ckpt8(*args, c["mt"], c["m_cap"], stream=stream, **kw)
        mine = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert all((m == 0x5A).all() for m in mine)
        np.testing.assert_array_equal(P.to_host(out[2]), ref)


def test_backward_on_streams_and_in_a_graph():
    inp, cfg, d, kw, dout = layer_case("fine64_shared2")
    sh = kw["shared"]
    x, dd = d["x"].clone(), P.to_dev(dout)

    def step():
        fwd = rpg.moe_layer(x, d["w1"], d["w3"], d["w2"], cfg.k, cfg.m_tile,
                            save_for_backward="mxfp8", **kw)
        g = rpg.moe_layer_backward(fwd, dd, x, d["w1"], d["w3"], d["w2"], cfg.m_tile, shared=sh)
        return [fwd["out"]] + [g[n] for n in ("dx", "dtopk_w", "dw1", "dw3", "dw2", "dws1", "dws2")]

    ref = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            both.append(step())
    torch.cuda.synchronize()
    for got in both:
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    # DenseRows uploads its two offsets from the host, which a capture does not allow: the
    # graph holds the routed experts
    def routed():
        fwd = rpg.moe_layer(x, d["w1"], d["w3"], d["w2"], cfg.k, cfg.m_tile, wg=d["wg"],
                            save_for_backward="mxfp8")
        g = rpg.moe_layer_backward(fwd, dd, x, d["w1"], d["w3"], d["w2"], cfg.m_tile)
        return [fwd["out"]] + [g[n] for n in ("dx", "dtopk_w", "dw1", "dw3", "dw2")]

    with torch.cuda.stream(streams[0]):
        routed()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = routed()
    for v in (d["x"], d["x"].flip(0).contiguous(), d["x"]):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = routed()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
