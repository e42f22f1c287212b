"""Plain NumPy definitions, in float64, of the block-scaled operators: MXFP4 rows, the 4-bit
products of prefill and decode, and the 8-bit checkpoint of fc1's pre-activations with its
backward. Test infrastructure only; it shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

from . import moe_oracle as orc

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _blocks(x):
    v = orc.values64(x)
    return v.reshape(v.shape[0], -1, 32)


def _exponents(amax, largest):
    """Smallest integer X >= -127 with amax <= largest * 2^X (finite amax), -127 for 0."""
    f, e = np.frexp(amax)
    fl, el = np.frexp(largest)
    X = np.where(f <= fl, e - el, e - el + 1)
    return np.where(amax > 0, np.maximum(X, -127), -127)


def mx4_quantize(x):
    """Rows x [R, C] -> (codes [R, C/2], two a byte, even element low; scales [R, C/32])."""
    b = _blocks(x)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    X = _exponents(np.abs(b).max(axis=2), 6.0)
    a = np.abs(b) / np.ldexp(1.0, X)[:, :, None]
    # nearest code; a tie goes to the even one of the two
    d = np.abs(a[..., None] - E2M1)
    lo = d.argmin(axis=-1)                       # the lower code of a tie
    tie = (lo < 7) & (np.take_along_axis(d, lo[..., None], -1)[..., 0] ==
                      np.take_along_axis(d, np.minimum(lo + 1, 7)[..., None], -1)[..., 0])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    code = np.where(np.signbit(b), code | 8, code)
    code = np.where(bad[:, :, None], 0, code).reshape(b.shape[0], -1, 2).astype(np.uint8)
    scales = np.where(bad, 255, X + 127).astype(np.uint8)
    return code[..., 0] | (code[..., 1] << 4), scales


def mx4_values(codes, scales):
    """Values [..., C] of codes [..., C/2] and scales [..., C/32] (NaN under byte 255)."""
    nib = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    return v * _powers(scales)


def mx8_values(codes, scales):
    """Values [..., C] of e4m3 codes [..., C] and scales [..., C/32] (NaN under byte 255)."""
    return orc.e4m3_decode(codes) * _powers(scales)


def _powers(scales):
    s = scales.astype(np.int64)
    return np.repeat(np.where(s == 255, np.nan, np.ldexp(1.0, s - 127)), 32, axis=-1)


def mx8_quantize(v):
    """Rows v [R, C] of finite values -> (e4m3 codes, scales), by the FP8 payload's rule."""
    return orc.mx_quantize(v)


def rows_of(words):
    """Scales in k-step words [C/128, R, 4] as rows [R, C/32]."""
    return np.ascontiguousarray(words.transpose(1, 0, 2)).reshape(words.shape[1], -1)


def words_of(scales):
    """Scale rows [R, C/32] in k-step words [C/128, R, 4]."""
    R, nb = scales.shape
    return np.ascontiguousarray(scales.reshape(R, nb // 4, 4).transpose(1, 0, 2))


def quantize_weights(w):
    """[E, N, K] -> codes [E, N, K/2], scale rows [E, N, K/32]."""
    E, N, K = w.shape
    q, s = mx4_quantize(np.asarray(w).reshape(E * N, K))
    return q.reshape(E, N, K // 2), s.reshape(E, N, K // 32)


def fc1(x, w1, w3):
    """silu(x w1^T) * (x w3^T) of values, with the sums of magnitudes a bound needs:
    (h, a, b, sum|x||w1|, sum|x||w3|)."""
    a, b = x @ w1.T, x @ w3.T
    return orc.silu(a) * b, a, b, np.abs(x) @ np.abs(w1).T, np.abs(x) @ np.abs(w3).T


def forward_mxfp4(inputs, k, m_tile):
    """The layer with 4-bit rows and weights: route on the bf16 x, quantize x, permute, fc1,
    h rounded to bf16 and quantized, fc2, shared experts and combine in bf16."""
    x = inputs["x"]
    E, F, D = inputs["w1"].shape
    if "topk_idx" in inputs:
        idx = np.asarray(inputs["topk_idx"], dtype=np.int32)
        w = np.asarray(inputs["topk_w"], dtype=np.float64)
    else:
        idx, w, _ = orc.route(x, inputs["wg"], k, "bf16", inputs.get("bias"))
    lay = orc.dispatch_layout(idx, E, m_tile)
    xq, xs = mx4_quantize(x)
    res = dict(lay, topk_idx=idx, topk_w=w, xq=xq, xs=xs)
    xp = mx4_values(orc.permute(xq, lay), orc.permute(xs, lay))
    h, y = np.zeros((xp.shape[0], F)), np.zeros((xp.shape[0], D))
    for e in range(E):
        r = slice(int(lay["offsets"][e]), int(lay["offsets"][e + 1]))
        if r.stop > r.start:
            w1, w3, w2 = (mx4_values(*mx4_quantize(inputs[n][e])) for n in ("w1", "w3", "w2"))
            h[r] = orc.round_bf16(fc1(xp[r], w1, w3)[0])
            y[r] = orc.round_bf16(mx4_values(*mx4_quantize(h[r])) @ w2.T)
    res["h"], res["y_perm"] = h, y
    shared = None
    if "ws1" in inputs:
        shared = orc.shared_experts(x, inputs["ws1"], inputs["ws3"], inputs["ws2"], "bf16")
    res["out"] = orc.combine(y, lay["dst_row"], w, "bf16", shared)
    return res


def masked_mxfp4(x_masked, counts, cap, w1, w3, w2):
    """bf16 rows of the slabs through weights given as values [E, F, D], [E, D, F]: (h, y),
    zero in rows past counts."""
    E, F, D = w1.shape
    h, y = np.zeros((E * cap, F)), np.zeros((E * cap, D))
    x = orc.values64(x_masked)
    for e in range(E):
        n = max(0, min(int(counts[e]), cap))
        if n:
            r = slice(e * cap, e * cap + n)
            h[r] = orc.round_bf16(fc1(x[r], w1[e], w3[e])[0])
            y[r] = orc.round_bf16(h[r] @ w2[e].T)
    return h, y


def ckpt8_rows(dout, w2e, a, b, w):
    """One expert's rows of the checkpoint's backward, values only: dout [n, D] unweighted,
    a, b [n, F], row weights w [n] -> (da, db, hw, dw)."""
    u = dout @ w2e
    w = np.asarray(w)[:, None]
    h = orc.silu(a) * b
    return w * u * b * orc.silu_grad(a), w * u * orc.silu(a), w * h, (u * h).sum(axis=1)


def backward_ckpt8(inputs, dout, k, m_tile, ckpt=None, shared_ckpt=None):
    """The bf16 layer's forward and its backward from an 8-bit checkpoint of [a | b]:
    dX, dx, the weight gradients and dtopk_w. The checkpoint's values are ``ckpt`` [m_cap, 2F]
    (``shared_ckpt`` [T, 2*S*Fs]) or quantized from the exact sums; intermediates are rounded
    to bf16 where the layer stores them."""
    fwd = orc.forward(inputs, k, m_tile, "bf16")
    E, F, D = inputs["w1"].shape
    offs, src, w = fwd["offsets"], fwd["src_row"], np.asarray(fwd["topk_w"], dtype=np.float64)
    M = fwd["x_perm"].shape[0]
    lay = orc.dispatch_layout(fwd["topk_idx"], E, m_tile)
    dp = orc.values64(orc.permute(dout, lay))
    xp = orc.values64(fwd["x_perm"])
    res = {"fwd": fwd, "dX": np.zeros((M, D)), "dab": np.zeros((M, 2 * F)),
           "dtopk_w": np.zeros(w.size), "dw1": np.zeros((E, F, D)), "dw3": np.zeros((E, F, D)),
           "dw2": np.zeros((E, D, F))}

    def expert(drows, xrows, wrow, w1, w3, w2, ab):
        if ab is None:
            ab = mx8_values(*mx8_quantize(np.concatenate([xrows @ w1.T, xrows @ w3.T], axis=1)))
        n = w1.shape[0]
        da, db, hw, dw = ckpt8_rows(drows, w2, ab[:, :n], ab[:, n:], wrow)
        da, db, hw = orc.round_bf16(da), orc.round_bf16(db), orc.round_bf16(hw)
        return da, db, dw, orc.round_bf16(da @ w1 + db @ w3), da.T @ xrows, db.T @ xrows, drows.T @ hw

    for e in range(E):
        r = slice(int(offs[e]), int(offs[e + 1]))
        if r.stop <= r.start:
            continue
        s = src[r]
        wrow = np.where(s >= 0, w.ravel()[np.maximum(s, 0)], 0.0)
        da, db, dw, res["dX"][r], res["dw1"][e], res["dw3"][e], res["dw2"][e] = expert(
            dp[r], xp[r], wrow, *(orc.values64(inputs[n][e]) for n in ("w1", "w3", "w2")),
            None if ckpt is None else ckpt[r])
        res["dab"][r, :F], res["dab"][r, F:] = da, db
        res["dtopk_w"][s[s >= 0]] = dw[s >= 0]
    res["dtopk_w"] = res["dtopk_w"].reshape(w.shape)
    dxs = None
    if "ws1" in inputs:
        ws1 = np.concatenate(list(orc.values64(inputs["ws1"])), axis=0)
        ws3 = np.concatenate(list(orc.values64(inputs["ws3"])), axis=0)
        ws2 = np.concatenate(list(orc.values64(inputs["ws2"])), axis=1)
        x, d = orc.values64(inputs["x"]), orc.values64(dout)
        _, _, _, dxs, res["dws1"], res["dws3"], res["dws2"] = expert(d, x, np.ones(x.shape[0]),
                                                                     ws1, ws3, ws2, shared_ckpt)
    res["dx"] = orc.permute_backward(res["dX"], fwd["dst_row"], "bf16", dxs)
    return res
