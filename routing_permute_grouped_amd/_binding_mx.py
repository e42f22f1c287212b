"""ctypes binding of the calls include/moe_mx.h declares: 4-bit quantisation and products,
8-bit checkpoints of fc1's pre-activations. Argument marshalling only, in the manner of
``_binding``; each call runs on the device of its first tensor (all others must be there)
and, without ``stream``, on that device's current stream. With ``stream``, what the caller does
not give is allocated there, so the call is ordered by that stream alone.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _binding as B

_P, _I, _I64, _SZ = B._P, B._I, B._I64, B._SZ
MX_SIGNATURES = [
    ("moe_quantize_mxfp4", _I, [_I, _P, _I64, _I, _P, _P, _I, _P]),
    ("moe_dequantize_mxfp4", _I, [_I, _P, _P, _I64, _I, _I, _P, _P]),
    ("moe_dequantize_mxfp8", _I, [_I, _P, _P, _I64, _I, _I, _P, _P]),
    ("moe_permute_mxfp4", _I, [_P, _P, _P, _I, _I, _I, _I, _I, _I64, _P, _P, _P, _P, _P, _P, _P,
                               _P, _SZ, _P, _P]),
    ("moe_grouped_fc1_swiglu_mxfp4", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _P,
                                          _P, _P, _P, _SZ, _P]),
    ("moe_grouped_fc2_mxfp4", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _P, _P, _SZ,
                                   _P]),
    ("moe_grouped_swiglu_masked_mxfp4", _I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                             _P, _P]),
    ("moe_grouped_fc1_swiglu_ckpt8", _I, [_P, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _P, _P,
                                          _P, _P, _SZ, _P]),
    ("moe_grouped_dgrad_swiglu_ckpt8", _I, [_P, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _P, _P,
                                            _P, _P, _I, _I, _P, _P, _P, _P, _SZ, _P, _SZ, _P]),
    ("moe_ckpt8_scratch_bytes", _SZ, [_I, _I64]),
]
for _name, _res, _args in MX_SIGNATURES:
    _fn = getattr(B.lib, _name)
    _fn.restype, _fn.argtypes = _res, _args


# The current stream's handle of a device: what torch.cuda.current_stream(dev).cuda_stream
# gives, without making the Stream object (1.1 us of a call that takes 8).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _run(name: str, stream, *args) -> None:
    """Call ``name`` with its C arguments in order, the stream last. A tensor is given as
    (argument name, tensor or None); every one must be contiguous and on the first one's GPU,
    where the call is made."""
    dev, c = None, []
    for a in args:
        if a.__class__ is not tuple:
            c.append(a)
            continue
        n, t = a
        if t is None:
            c.append(None)
            continue
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise ValueError(f"{n}: tensor must live on the GPU")
            if dev is not None:
                raise ValueError(f"{n}: on cuda:{d}, expected cuda:{dev}")
            dev = d
        if not t.is_contiguous():
            raise ValueError(f"{n}: tensor must be contiguous")
        c.append(t.data_ptr())
    fn = getattr(B.lib, name)
    if torch.cuda.current_device() == dev:
        B._check(name, fn(*c, _raw_stream(dev) if stream is None else B._stream(stream)))
        return
    with torch.cuda.device(dev):
        B._check(name, fn(*c, _raw_stream(dev) if stream is None else B._stream(stream)))


def _new(stream, like: torch.Tensor, shape, dtype: torch.dtype) -> torch.Tensor:
    """A buffer of the call's own on ``like``'s device, from the memory of the stream that the call
    runs on: a block of the current stream's may come from a tensor that work queued there
    still uses, and nothing orders ``stream`` behind that work. What the current stream does
    with the buffer later keeps it from reuse."""
    if stream is None or not like.is_cuda:
        return like.new_empty(shape, dtype=dtype)
    dev = like.device
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(B._stream(stream), device=dev)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _scales(t: Optional[torch.Tensor], name: str, rows: int, C: int, layout: int) -> None:
    """t (if given) holds the scales of ``rows`` rows of C values in ``layout``. Both layouts have
    as many bytes, so the shape tells them apart: scale rows [..., C/32]; k-step words
    [C/128, rows, 4] (the rows' axis may be split), over exactly these rows, which are the
    words' stride. A flat buffer has no such shape and is taken as it is; of one row or one step
    both layouts are the same bytes."""
    if t is None:
        return
    words = layout == B.MOE_MX_KSTEPS
    if words and t.shape == (C // 128, rows, 4) and t.dtype == torch.uint8:
        return
    n = rows * (C // 32)
    B._numel(t, name, n, torch.uint8)
    if t.dim() < 2 or C % (128 if words else 32) or (rows == 1 and t.numel() == n):
        return
    if words and C > 128:
        ok = t.shape[0] == C // 128 and t.shape[-1] == 4 and t.numel() == n
    else:
        ok = t.shape[-1] == C // 32
    if not ok:
        kind = f"k-step words {(C // 128, rows, 4)}" if words else f"scale rows [{rows}, {C // 32}]"
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {kind}")


def _block_rows(codes: torch.Tensor, name: str, per: int) -> Tuple[int, int]:
    """(R, C) of code rows [..., C * per / 2]: per 2 for a byte a code, 1 for two a byte."""
    B._dtype(codes, name, torch.uint8)
    if codes.dim() < 1 or codes.numel() == 0:
        raise ValueError(f"{name}: shape {tuple(codes.shape)}, expected rows of codes")
    width = codes.shape[-1]
    return codes.numel() // width, width * 2 // per


def moe_quantize_mxfp4(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                       scales: Optional[torch.Tensor] = None, layout: int = B.MOE_MX_ROWS,
                       stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """MXFP4 codes and E8M0 scales of the rows of x [..., C]. Returns (q uint8 [..., C/2], the
    even element in the low half, and scales): layout MOE_MX_ROWS, uint8 [..., C/32] (C a
    multiple of 32); MOE_MX_KSTEPS, the products' k-step words as uint8 [C/128, R, 4] (R
    rows, C a multiple of 128)."""
    B._layer_dtype(x, "x")
    n = x.numel()
    if n == 0 or x.dim() < 1:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected rows of values")
    *lead, C = x.shape
    R = n // C
    if q is None:
        q = _new(stream, x, (*lead, C // 2), torch.uint8)
    else:
        B._numel(q, "q", n // 2, torch.uint8)
    if scales is None:
        scales = _new(stream, x, (C // 128, R, 4) if layout == B.MOE_MX_KSTEPS
                      else (*lead, C // 32), torch.uint8)
    else:
        _scales(scales, "scales", R, C, layout)
    _run("moe_quantize_mxfp4", stream, B._dt(x), ("x", x), R, C, ("q", q), ("scales", scales),
         layout)
    return q, scales


def _dequantize(name: str, per: int, q, scales, out, layout, dtype, stream) -> torch.Tensor:
    R, C = _block_rows(q, "q", per)
    _scales(scales, "scales", R, C, layout)
    if out is None:
        if dtype not in B._LAYER_DTYPES:
            raise TypeError(f"dtype {dtype}, expected float32 or bfloat16")
        out = _new(stream, q, (*q.shape[:-1], C), dtype)
    else:
        B._layer_dtype(out, "out")
        B._numel(out, "out", R * C)
    _run(name, stream, B._dt(out), ("q", q), ("scales", scales), R, C, layout, ("out", out))
    return out


def moe_dequantize_mxfp4(q: torch.Tensor, scales: torch.Tensor,
                         out: Optional[torch.Tensor] = None, layout: int = B.MOE_MX_ROWS,
                         dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The values [..., C] of MXFP4 codes q [..., C/2] and their scales, in ``dtype`` (or
    out's)."""
    return _dequantize("moe_dequantize_mxfp4", 1, q, scales, out, layout, dtype, stream)


def moe_dequantize_mxfp8(q: torch.Tensor, scales: torch.Tensor,
                         out: Optional[torch.Tensor] = None, layout: int = B.MOE_MX_ROWS,
                         dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The values [..., C] of MXFP8 (e4m3) codes q [..., C] and their scales, in ``dtype`` (or
    out's)."""
    return _dequantize("moe_dequantize_mxfp8", 2, q, scales, out, layout, dtype, stream)


def moe_permute_mxfp4(xq: torch.Tensor, xs: torch.Tensor, topk_idx: torch.Tensor, E: int,
                      m_tile: int, m_cap: Optional[int] = None, out: Optional[dict] = None,
                      stream=None) -> dict:
    """moe_permute for the 4-bit payload xq [T, D/2], xs [T, D/32]: dict with xq_perm
    [m_cap, D/2], xs_perm (the scales in k-step words, uint8 [D/128, m_cap, 4]) and the
    metadata. Buffers given in ``out`` are reused."""
    B._dims(xq, "xq", 2)
    T, D = _block_rows(xq, "xq", 1)
    _scales(xs, "xs", T, D, B.MOE_MX_ROWS)
    k = B._check_idx(topk_idx, T)
    if m_cap is None:
        m_cap = B.moe_capacity(T, k, E, m_tile)
        if m_cap < 0:
            raise ValueError(f"no capacity for T={T}, k={k}, E={E}, m_tile={m_tile}")
    o = dict(out or {})
    B._rows(o.get("xq_perm"), "xq_perm", m_cap, D // 2, torch.uint8)
    _scales(o.get("xs_perm"), "xs_perm", m_cap, D, B.MOE_MX_KSTEPS)
    B._check_layout_out(o, T, k, E, m_cap, m_tile)
    ws = max(4, B.moe_permute_workspace_bytes(T, k, E))
    B._nbytes(o.get("workspace"), "workspace", ws)
    u8, i32 = torch.uint8, torch.int32
    for n, shape, dt in (("xq_perm", (m_cap, D // 2), u8), ("xs_perm", (D // 128, m_cap, 4), u8),
                         ("counts", E, i32), ("offsets", E + 1, i32), ("dst_row", (T, k), i32),
                         ("src_row", m_cap, i32), ("tile_expert", m_cap // m_tile, i32),
                         ("dev_err", 1, i32), ("workspace", ws, u8)):
        if n not in o:
            o[n] = _new(stream, xq, shape, dt)
    wsb = o["workspace"].numel() * o["workspace"].element_size()
    _run("moe_permute_mxfp4", stream, ("xq", xq), ("xs", xs), ("topk_idx", topk_idx), T, D, E, k,
         m_tile, m_cap, ("xq_perm", o["xq_perm"]), ("xs_perm", o["xs_perm"]),
         ("counts", o["counts"]), ("offsets", o["offsets"]), ("dst_row", o["dst_row"]),
         ("src_row", o["src_row"]), ("tile_expert", o["tile_expert"]),
         ("workspace", o["workspace"]), wsb, ("dev_err", o["dev_err"]))
    o["m_cap"] = m_cap
    return o


def _mx4_weight(q: torch.Tensor, s: torch.Tensor, name: str, shape=None) -> Tuple[int, int, int]:
    """(E, N, K) of codes [E, N, K/2] (of ``shape`` [E, N, K], if given) with their k-step
    words [K/128, E*N, 4]."""
    B._dtype(q, name + "q", torch.uint8)
    B._dims(q, name + "q", 3)
    E, N, K = q.shape[0], q.shape[1], q.shape[2] * 2
    if shape is not None and (E, N, K) != tuple(shape):
        raise ValueError(f"{name}q: shape {tuple(q.shape)}, expected "
                         f"{(shape[0], shape[1], shape[2] // 2)}")
    _scales(s, name + "s", E * N, K, B.MOE_MX_KSTEPS)
    return E, N, K


def _mx4_rows(q: torch.Tensor, s: torch.Tensor, name: str, m_cap: int, K: int) -> None:
    B._rows(q, name + "q", m_cap, K // 2, torch.uint8)
    _scales(s, name + "s", m_cap, K, B.MOE_MX_KSTEPS)


def _wsz(ws: Optional[torch.Tensor]) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


def moe_grouped_fc1_swiglu_mxfp4(xq_perm: torch.Tensor, xs_perm: torch.Tensor,
                                 offsets: torch.Tensor, tile_expert: torch.Tensor,
                                 w1q: torch.Tensor, w1s: torch.Tensor, w3q: torch.Tensor,
                                 w3s: torch.Tensor, m_tile: int, m_cap: Optional[int] = None,
                                 h: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, stream=None,
                                 counts: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h [m_cap, F] bf16 = silu(a)*b from 4-bit rows (codes [m_cap, D/2], k-step words
    [D/128, m_cap, 4]) and 4-bit w1, w3 (codes [E, F, D/2], k-step words [D/128, E*F, 4])."""
    E, F, D = _mx4_weight(w1q, w1s, "w1")
    _mx4_weight(w3q, w3s, "w3", (E, F, D))
    if m_cap is None:
        m_cap = xq_perm.shape[0]
    _mx4_rows(xq_perm, xs_perm, "x", m_cap, D)
    B._check_segments(offsets, tile_expert, E, m_cap, m_tile)
    B._numel(counts, "counts", E, torch.int32)
    B._rows(h, "h", m_cap, F, torch.bfloat16)
    if h is None:
        h = _new(stream, xq_perm, (m_cap, F), torch.bfloat16)
    _run("moe_grouped_fc1_swiglu_mxfp4", stream, ("xq_perm", xq_perm), ("xs_perm", xs_perm),
         ("offsets", offsets), ("counts", counts), ("tile_expert", tile_expert), E, D, F, m_tile,
         m_cap, ("w1q", w1q), ("w1s", w1s), ("w3q", w3q), ("w3s", w3s), ("h", h),
         ("workspace", workspace), _wsz(workspace))
    return h


def moe_grouped_fc2_mxfp4(hq: torch.Tensor, hs: torch.Tensor, offsets: torch.Tensor,
                          tile_expert: torch.Tensor, w2q: torch.Tensor, w2s: torch.Tensor,
                          m_tile: int, m_cap: Optional[int] = None,
                          y_perm: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None,
                          counts: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y_perm [m_cap, D] bf16 = h w2[e]^T from 4-bit rows (codes [m_cap, F/2], k-step words
    [F/128, m_cap, 4]) and 4-bit w2 (codes [E, D, F/2], k-step words [F/128, E*D, 4])."""
    E, D, F = _mx4_weight(w2q, w2s, "w2")
    if m_cap is None:
        m_cap = hq.shape[0]
    _mx4_rows(hq, hs, "h", m_cap, F)
    B._check_segments(offsets, tile_expert, E, m_cap, m_tile)
    B._numel(counts, "counts", E, torch.int32)
    B._rows(y_perm, "y_perm", m_cap, D, torch.bfloat16)
    if y_perm is None:
        y_perm = _new(stream, hq, (m_cap, D), torch.bfloat16)
    _run("moe_grouped_fc2_mxfp4", stream, ("hq", hq), ("hs", hs), ("offsets", offsets),
         ("counts", counts), ("tile_expert", tile_expert), E, D, F, m_tile, m_cap, ("w2q", w2q),
         ("w2s", w2s), ("y_perm", y_perm), ("workspace", workspace), _wsz(workspace))
    return y_perm


def moe_grouped_swiglu_masked_mxfp4(x_masked: torch.Tensor, counts: torch.Tensor,
                                    w1q: torch.Tensor, w1s: torch.Tensor, w3q: torch.Tensor,
                                    w3s: torch.Tensor, w2q: torch.Tensor, w2s: torch.Tensor,
                                    cap: int, h: Optional[torch.Tensor] = None,
                                    y: Optional[torch.Tensor] = None, stream=None):
    """(h, y) on the valid rows of every slab of the masked layout, bf16 rows against 4-bit
    weights (codes and k-step words as moe_grouped_fc1_swiglu_mxfp4 and
    moe_grouped_fc2_mxfp4 take them); the other rows of h and y are left as they are."""
    E, F, D = _mx4_weight(w1q, w1s, "w1")
    _mx4_weight(w3q, w3s, "w3", (E, F, D))
    _mx4_weight(w2q, w2s, "w2", (E, D, F))
    B._rows(x_masked, "x_masked", E * cap, D, torch.bfloat16)
    B._numel(counts, "counts", E, torch.int32)
    B._rows(h, "h", E * cap, F, torch.bfloat16)
    B._rows(y, "y", E * cap, D, torch.bfloat16)
    if h is None:
        h = _new(stream, x_masked, (E * cap, F), torch.bfloat16)
    if y is None:
        y = _new(stream, x_masked, (E * cap, D), torch.bfloat16)
    _run("moe_grouped_swiglu_masked_mxfp4", stream, ("x_masked", x_masked), ("counts", counts), E,
         D, F, cap, ("w1q", w1q), ("w1s", w1s), ("w3q", w3q), ("w3s", w3s), ("w2q", w2q),
         ("w2s", w2s), ("h", h), ("y", y))
    return h, y


def moe_grouped_fc1_swiglu_ckpt8(x_perm: torch.Tensor, offsets: torch.Tensor,
                                 tile_expert: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor,
                                 m_tile: int, m_cap: Optional[int] = None,
                                 h: Optional[torch.Tensor] = None,
                                 ab_codes: Optional[torch.Tensor] = None,
                                 ab_scales: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, stream=None,
                                 rows_used: Optional[int] = None,
                                 counts: Optional[torch.Tensor] = None):
    """moe_grouped_fc1_swiglu (bf16) that keeps the pre-activations [a | b] for the backward as
    MXFP8. Returns (h [m_cap, F], ab_codes uint8 [m_cap, 2F], ab_scales uint8
    [m_cap, 2F/32])."""
    B._dims(w1, "w1", 3)
    E, F, D = w1.shape
    B._weights(w1, w3, None, torch.bfloat16, E, F, D)
    if m_cap is None:
        m_cap = x_perm.shape[0]
    B._rows(x_perm, "x_perm", B._used(rows_used, m_cap), D, torch.bfloat16)
    B._check_segments(offsets, tile_expert, E, m_cap, m_tile)
    B._numel(counts, "counts", E, torch.int32)
    B._rows(h, "h", m_cap, F, torch.bfloat16)
    B._rows(ab_codes, "ab_codes", m_cap, 2 * F, torch.uint8)
    B._rows(ab_scales, "ab_scales", m_cap, F // 16, torch.uint8)
    if h is None:
        h = _new(stream, x_perm, (m_cap, F), torch.bfloat16)
    if ab_codes is None:
        ab_codes = _new(stream, x_perm, (m_cap, 2 * F), torch.uint8)
    if ab_scales is None:
        ab_scales = _new(stream, x_perm, (m_cap, F // 16), torch.uint8)
    _run("moe_grouped_fc1_swiglu_ckpt8", stream, ("x_perm", x_perm), ("offsets", offsets),
         ("counts", counts), ("tile_expert", tile_expert), E, D, F, m_tile, m_cap, ("w1", w1),
         ("w3", w3), ("h", h), ("ab_codes", ab_codes), ("ab_scales", ab_scales),
         ("workspace", workspace), _wsz(workspace))
    return h, ab_codes, ab_scales


def moe_ckpt8_scratch_bytes(F: int, m_cap: int) -> int:
    return int(B.lib.moe_ckpt8_scratch_bytes(F, m_cap))


def moe_grouped_dgrad_swiglu_ckpt8(dout_perm: torch.Tensor, offsets: torch.Tensor,
                                   tile_expert: torch.Tensor, w2: torch.Tensor,
                                   ab_codes: torch.Tensor, ab_scales: torch.Tensor, m_tile: int,
                                   m_cap: Optional[int] = None,
                                   src_row: Optional[torch.Tensor] = None,
                                   dst_row: Optional[torch.Tensor] = None,
                                   topk_w: Optional[torch.Tensor] = None,
                                   dab: Optional[torch.Tensor] = None,
                                   hw: Optional[torch.Tensor] = None,
                                   dtopk_w: Optional[torch.Tensor] = None,
                                   scratch: Optional[torch.Tensor] = None,
                                   workspace: Optional[torch.Tensor] = None, stream=None,
                                   rows_used: Optional[int] = None,
                                   counts: Optional[torch.Tensor] = None):
    """The backward of combine, fc2 and silu(a)*b from an 8-bit checkpoint, for the output
    gradient's rows dout_perm [m_cap, D] (moe_permute of dout, unweighted). Returns
    (dab [m_cap, 2F], hw [m_cap, F], dtopk_w [T, k] float32): dab for moe_grouped_dgrad_fc1
    and the wgrad of w1 and w3, hw = w*silu(a)*b for the wgrad of w2 (dW2 = dout_perm^T hw).
    Without ``topk_w`` every row's weight is 1 and dtopk_w is None (``src_row``, ``dst_row``
    and ``scratch`` are then not used); with it, ``src_row`` and ``dst_row`` are needed."""
    B._dims(w2, "w2", 3)
    E, D, F = w2.shape
    B._weights(None, None, w2, torch.bfloat16, E, F, D)
    if m_cap is None:
        m_cap = dout_perm.shape[0]
    ru = B._used(rows_used, m_cap)
    B._rows(dout_perm, "dout_perm", ru, D, torch.bfloat16)
    B._check_segments(offsets, tile_expert, E, m_cap, m_tile)
    B._numel(counts, "counts", E, torch.int32)
    B._rows(ab_codes, "ab_codes", ru, 2 * F, torch.uint8)
    B._rows(ab_scales, "ab_scales", ru, F // 16, torch.uint8)
    B._rows(dab, "dab", m_cap, 2 * F, torch.bfloat16)
    B._rows(hw, "hw", m_cap, F, torch.bfloat16)
    T = k = need = 0
    if topk_w is not None:
        B._dims(topk_w, "topk_w", 2)
        B._dtype(topk_w, "topk_w", torch.float32)
        T, k = topk_w.shape
        if src_row is None or dst_row is None:
            raise ValueError("topk_w needs src_row and dst_row")
        B._numel(src_row, "src_row", m_cap, torch.int32)
        B._exact(dst_row, "dst_row", (T, k), torch.int32)
        B._exact(dtopk_w, "dtopk_w", (T, k), torch.float32)
        need = moe_ckpt8_scratch_bytes(F, m_cap)
        B._nbytes(scratch, "scratch", need)
    elif dtopk_w is not None:
        raise ValueError("dtopk_w needs topk_w")
    if dab is None:
        dab = _new(stream, dout_perm, (m_cap, 2 * F), torch.bfloat16)
    if hw is None:
        hw = _new(stream, dout_perm, (m_cap, F), torch.bfloat16)
    if topk_w is None:
        src_row = dst_row = scratch = None
    else:
        if dtopk_w is None:
            dtopk_w = _new(stream, dout_perm, (T, k), torch.float32)
        if scratch is None:
            scratch = _new(stream, dout_perm, need, torch.uint8)
    _run("moe_grouped_dgrad_swiglu_ckpt8", stream, ("dout_perm", dout_perm), ("offsets", offsets),
         ("counts", counts), ("tile_expert", tile_expert), E, D, F, m_tile, m_cap, ("w2", w2),
         ("ab_codes", ab_codes), ("ab_scales", ab_scales), ("src_row", src_row),
         ("dst_row", dst_row), ("topk_w", topk_w), T, k, ("dab", dab), ("hw", hw),
         ("dtopk_w", dtopk_w), ("scratch", scratch), _wsz(scratch), ("workspace", workspace),
         _wsz(workspace))
    return dab, hw, dtopk_w
