"""The whole layer as one chain of the four library calls on the current stream.

route -> permute -> grouped SwiGLU (routed experts) [-> grouped SwiGLU (shared
experts as one expert over all tokens)] -> combine, following the layer order of
"Expert Parallelism (EP)" (llm-infra-atlas), section 1.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Union

import torch

from . import _binding as B
from . import _binding_block as K
from . import _binding_mx as X


@dataclass
class SharedExperts:
    """Shared experts stored as one expert whose intermediate dimension is the
    concatenation of theirs: sum_s w2_s(silu(w1_s x) * w3_s x) equals the single
    expert with w1, w3 stacked along F and w2 concatenated along its F axis."""
    w1: torch.Tensor       # [1, S*Fs, D]
    w3: torch.Tensor       # [1, S*Fs, D]
    w2: torch.Tensor       # [1, D, S*Fs]

    @staticmethod
    def from_stacked(ws1: torch.Tensor, ws3: torch.Tensor, ws2: torch.Tensor) -> "SharedExperts":
        S, Fs, D = ws1.shape
        return SharedExperts(ws1.reshape(1, S * Fs, D).contiguous(),
                             ws3.reshape(1, S * Fs, D).contiguous(),
                             torch.cat(list(ws2), dim=1).reshape(1, D, S * Fs).contiguous())


class DenseRows:
    """offsets/tile_expert describing one expert over T rows (the shared-expert call)."""

    def __init__(self, T: int, m_tile: int, device):
        self.T = T
        self.m_cap = -(-T // m_tile) * m_tile
        # made on the device: a copy from the host waits for the stream and cannot be captured
        self.offsets = torch.arange(2, dtype=torch.int32, device=device).mul_(T)
        self.tile_expert = torch.zeros(self.m_cap // m_tile, dtype=torch.int32, device=device)


def moe_layer(x: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, k: int,
              m_tile: int, wg: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
              topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
              shared: Optional[SharedExperts] = None, renorm: bool = False,
              check: bool = False, split_k: bool = True,
              save_for_backward: Union[bool, str] = False) -> dict:
    """Run the layer; returns every intermediate (dict). With routing given
    (``topk_idx``/``topk_w``) the route step is skipped. ``check`` synchronises and
    raises if the permute saw an expert index outside [-1, E). ``split_k`` gives the
    grouped GEMMs a workspace so they can split a partly filled last round of tiles.
    ``save_for_backward`` also keeps fc1's pre-activations (``ab``, and ``shared_ab`` /
    ``shared_h`` for the shared experts), which ``moe_layer_backward`` reads;
    ``save_for_backward="mxfp8"`` (bf16) keeps them in 8 bits instead (``ab_codes``,
    ``ab_scales``, and ``shared_`` ones), and returns neither ``x_perm``, ``h`` nor ``y_perm``
    (nor ``shared_h``), which that backward does without: per routed row 2F*33/32 bytes in
    place of 4D + 6F."""
    res, y, sh = _layer_rows(x, w1, w3, w2, k, m_tile, wg, bias, topk_idx, topk_w, shared, renorm,
                             split_k, save_for_backward)
    res["out"] = B.moe_combine(y, res["dst_row"], res["topk_w"], shared=sh, m_cap=res["m_cap"])
    if check:
        torch.cuda.current_stream().synchronize()
        if int(res["dev_err"].item()) != 0:
            raise ValueError("topk_idx holds expert indices outside [-1, E)")
    return res


def _layer_rows(x, w1, w3, w2, k, m_tile, wg, bias, topk_idx, topk_w, shared, renorm, split_k,
                save_for_backward, want_logits=False):
    """moe_layer up to its combine: (its results so far, the expert rows y, the shared experts'
    rows or None). ``want_logits`` keeps the router's logits (``logits``)."""
    E, F, D = w1.shape
    ckpt8 = save_for_backward == "mxfp8"
    if isinstance(save_for_backward, str) and not ckpt8:
        raise ValueError(f"save_for_backward: {save_for_backward!r}, expected True, False or 'mxfp8'")
    res = {}
    if topk_idx is None:
        topk_idx, topk_w, logits = B.moe_route(x, wg, k, bias=bias, renorm=renorm,
                                               want_logits=want_logits)
        if want_logits:
            res["logits"] = logits
    res["topk_idx"], res["topk_w"] = topk_idx, topk_w
    p = B.moe_permute(x, topk_idx, E, m_tile)
    res.update(p)
    m_cap = p["m_cap"]
    ws = B.grouped_workspace(x.device) if split_k else None
    if ckpt8:
        h, res["ab_codes"], res["ab_scales"] = X.moe_grouped_fc1_swiglu_ckpt8(
            p["x_perm"], p["offsets"], p["tile_expert"], w1, w3, m_tile, m_cap, workspace=ws,
            counts=p["counts"])
        y = torch.empty((m_cap, D), dtype=x.dtype, device=x.device)
        B.moe_grouped_fc2(h, p["offsets"], p["tile_expert"], w2, m_tile, m_cap, y, workspace=ws,
                          counts=p["counts"])
        del res["x_perm"]
    elif save_for_backward:
        h = torch.empty((m_cap, F), dtype=x.dtype, device=x.device)
        ab = torch.empty((m_cap, 2 * F), dtype=x.dtype, device=x.device)
        y = torch.empty((m_cap, D), dtype=x.dtype, device=x.device)
        B.moe_grouped_fc1_swiglu(p["x_perm"], p["offsets"], p["tile_expert"], w1, w3, m_tile,
                                 m_cap, h, ab=ab, workspace=ws, counts=p["counts"])
        B.moe_grouped_fc2(h, p["offsets"], p["tile_expert"], w2, m_tile, m_cap, y, workspace=ws,
                          counts=p["counts"])
        res["ab"] = ab
    else:
        h, y = B.moe_grouped_swiglu(p["x_perm"], p["offsets"], p["tile_expert"], w1, w3, w2,
                                    m_tile, m_cap=m_cap, workspace=ws, counts=p["counts"])
    if not ckpt8:
        res["h"], res["y_perm"] = h, y
    sh = None
    if shared is not None:
        rows = DenseRows(x.shape[0], m_tile, x.device)
        if ckpt8:
            hs, res["shared_ab_codes"], res["shared_ab_scales"] = X.moe_grouped_fc1_swiglu_ckpt8(
                x, rows.offsets, rows.tile_expert, shared.w1, shared.w3, m_tile, rows.m_cap,
                workspace=ws, rows_used=rows.T)
            ys = torch.empty((rows.m_cap, D), dtype=x.dtype, device=x.device)
            B.moe_grouped_fc2(hs, rows.offsets, rows.tile_expert, shared.w2, m_tile, rows.m_cap,
                              ys, workspace=ws)
        elif save_for_backward:
            SF = shared.w1.shape[1]
            hs = torch.empty((rows.m_cap, SF), dtype=x.dtype, device=x.device)
            abs_ = torch.empty((rows.m_cap, 2 * SF), dtype=x.dtype, device=x.device)
            ys = torch.empty((rows.m_cap, D), dtype=x.dtype, device=x.device)
            B.moe_grouped_fc1_swiglu(x, rows.offsets, rows.tile_expert, shared.w1, shared.w3,
                                     m_tile, rows.m_cap, hs, ab=abs_, workspace=ws,
                                     rows_used=rows.T)
            B.moe_grouped_fc2(hs, rows.offsets, rows.tile_expert, shared.w2, m_tile, rows.m_cap,
                              ys, workspace=ws)
            res["shared_h"], res["shared_ab"] = hs, abs_
        else:
            _, ys = B.moe_grouped_swiglu(x, rows.offsets, rows.tile_expert, shared.w1, shared.w3,
                                         shared.w2, m_tile, m_cap=rows.m_cap, workspace=ws,
                                         rows_used=rows.T)
        sh = ys[: x.shape[0]]
        res["shared"] = sh
    return res, y, sh


def moe_layer_masked(x: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor,
                     k: int, cap: int, wg: Optional[torch.Tensor] = None,
                     bias: Optional[torch.Tensor] = None, topk_idx: Optional[torch.Tensor] = None,
                     topk_w: Optional[torch.Tensor] = None,
                     shared: Optional[SharedExperts] = None, renorm: bool = False,
                     split_k: bool = True, shared_m_tile: int = 128) -> dict:
    """The layer on the masked (fixed-capacity) layout for decode: route -> masked
    permute (slabs of ``cap`` rows per expert) -> masked grouped SwiGLU [-> shared
    experts] -> combine. Slots past an expert's cap are dropped (bit 1 of dev_err)."""
    E = w1.shape[0]
    res = {}
    if topk_idx is None:
        topk_idx, topk_w, _ = B.moe_route(x, wg, k, bias=bias, renorm=renorm)
    res["topk_idx"], res["topk_w"] = topk_idx, topk_w
    p = B.moe_permute_masked(x, topk_idx, E, cap)
    res.update(p)
    ws = B.grouped_workspace(x.device) if split_k else None
    h, y = B.moe_grouped_swiglu_masked(p["x_masked"], p["counts"], w1, w3, w2, cap, workspace=ws)
    res["h"], res["y_perm"] = h, y
    sh = None
    if shared is not None:
        rows = DenseRows(x.shape[0], shared_m_tile, x.device)
        _, ys = B.moe_grouped_swiglu(x, rows.offsets, rows.tile_expert, shared.w1, shared.w3,
                                     shared.w2, shared_m_tile, m_cap=rows.m_cap, workspace=ws,
                                     rows_used=rows.T)
        sh = ys[: x.shape[0]]
        res["shared"] = sh
    res["out"] = B.moe_combine(y, p["dst_row"], topk_w, shared=sh, m_cap=p["m_cap"])
    return res


@dataclass
class MxWeights:
    """fc1's weights quantized once for the FP8 payload: e4m3 codes [E,F,D] of w1 and w3,
    and their E8M0 scales in the GEMM's k-step words (uint8 [D/128, E*F, 4]: word (s, r)
    holds row r's scales of values 128*s .. 128*s + 127)."""
    w1q: torch.Tensor
    w1s: torch.Tensor
    w3q: torch.Tensor
    w3s: torch.Tensor

    @staticmethod
    def quantize(w1: torch.Tensor, w3: torch.Tensor) -> "MxWeights":
        w1q, w1s = B.moe_quantize_mxfp8(w1, layout=B.MOE_MX_KSTEPS)
        w3q, w3s = B.moe_quantize_mxfp8(w3, layout=B.MOE_MX_KSTEPS)
        return MxWeights(w1q, w1s, w3q, w3s)


def moe_layer_mxfp8(x: torch.Tensor, mw: MxWeights, w2: torch.Tensor, k: int, m_tile: int,
                    wg: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                    topk_idx: Optional[torch.Tensor] = None,
                    topk_w: Optional[torch.Tensor] = None,
                    shared: Optional[SharedExperts] = None, renorm: bool = False,
                    split_k: bool = True) -> dict:
    """The layer with an FP8 payload (EP page, section 6 "DeepSeek-V3 量级的示例数字": the
    dispatch payload is FP8 e4m3 with scales, the combine stays bf16): route on the bf16 x -> MX-quantize x -> permute codes and scales ->
    fc1 on the scaled-FP8 MFMA -> fc2 (bf16) [-> shared experts, bf16] -> combine."""
    E = mw.w1q.shape[0]
    res = {}
    if topk_idx is None:
        topk_idx, topk_w, _ = B.moe_route(x, wg, k, bias=bias, renorm=renorm)
    res["topk_idx"], res["topk_w"] = topk_idx, topk_w
    xq, xs = B.moe_quantize_mxfp8(x)
    res["xq"], res["xs"] = xq, xs
    p = B.moe_permute_mxfp8(xq, xs, topk_idx, E, m_tile)
    res.update(p)
    m_cap = p["m_cap"]
    ws = B.grouped_workspace(x.device) if split_k else None
    h = B.moe_grouped_fc1_swiglu_mxfp8(p["xq_perm"], p["xs_perm"], p["offsets"], p["tile_expert"],
                                       mw.w1q, mw.w1s, mw.w3q, mw.w3s, m_tile, m_cap,
                                       workspace=ws, counts=p["counts"])
    y = torch.empty((m_cap, x.shape[1]), dtype=x.dtype, device=x.device)
    B.moe_grouped_fc2(h, p["offsets"], p["tile_expert"], w2, m_tile, m_cap, y, workspace=ws,
                      counts=p["counts"])
    res["h"], res["y_perm"] = h, y
    sh = None
    if shared is not None:
        rows = DenseRows(x.shape[0], m_tile, x.device)
        _, ys = B.moe_grouped_swiglu(x, rows.offsets, rows.tile_expert, shared.w1, shared.w3,
                                     shared.w2, m_tile, m_cap=rows.m_cap, workspace=ws,
                                     rows_used=rows.T)
        sh = ys[: x.shape[0]]
        res["shared"] = sh
    res["out"] = B.moe_combine(y, p["dst_row"], topk_w, shared=sh, m_cap=m_cap)
    return res


@dataclass
class Mx4Weights:
    """The experts' weights quantized once to MXFP4: codes (two a byte) w1q, w3q [E,F,D/2],
    w2q [E,D,F/2], and their E8M0 scales in the products' k-step words (w1s, w3s uint8
    [D/128, E*F, 4], w2s [F/128, E*D, 4])."""
    w1q: torch.Tensor
    w1s: torch.Tensor
    w3q: torch.Tensor
    w3s: torch.Tensor
    w2q: torch.Tensor
    w2s: torch.Tensor

    @staticmethod
    def quantize(w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor) -> "Mx4Weights":
        w1q, w1s = X.moe_quantize_mxfp4(w1, layout=B.MOE_MX_KSTEPS)
        w3q, w3s = X.moe_quantize_mxfp4(w3, layout=B.MOE_MX_KSTEPS)
        w2q, w2s = X.moe_quantize_mxfp4(w2, layout=B.MOE_MX_KSTEPS)
        return Mx4Weights(w1q, w1s, w3q, w3s, w2q, w2s)


def moe_layer_mxfp4(x: torch.Tensor, mw: Mx4Weights, k: int, m_tile: int,
                    wg: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                    topk_idx: Optional[torch.Tensor] = None,
                    topk_w: Optional[torch.Tensor] = None,
                    shared: Optional[SharedExperts] = None, renorm: bool = False,
                    split_k: bool = True) -> dict:
    """The layer (bf16 x) with 4-bit weights and 4-bit rows in both products: route on the bf16
    x -> quantize x -> permute codes and scales -> fc1 and fc2 on the scaled FP4 MFMA, h
    quantized between them [-> shared experts, bf16] -> combine."""
    E = mw.w1q.shape[0]
    res = {}
    if topk_idx is None:
        topk_idx, topk_w, _ = B.moe_route(x, wg, k, bias=bias, renorm=renorm)
    res["topk_idx"], res["topk_w"] = topk_idx, topk_w
    B._dtype(x, "x", torch.bfloat16)
    xq, xs = X.moe_quantize_mxfp4(x)
    res["xq"], res["xs"] = xq, xs
    p = X.moe_permute_mxfp4(xq, xs, topk_idx, E, m_tile)
    res.update(p)
    m_cap = p["m_cap"]
    ws = B.grouped_workspace(x.device) if split_k else None
    h = X.moe_grouped_fc1_swiglu_mxfp4(p["xq_perm"], p["xs_perm"], p["offsets"],
                                       p["tile_expert"], mw.w1q, mw.w1s, mw.w3q, mw.w3s, m_tile,
                                       m_cap, workspace=ws, counts=p["counts"])
    hq, hs = X.moe_quantize_mxfp4(h, layout=B.MOE_MX_KSTEPS)
    y = X.moe_grouped_fc2_mxfp4(hq, hs, p["offsets"], p["tile_expert"], mw.w2q, mw.w2s, m_tile,
                                m_cap, workspace=ws, counts=p["counts"])
    res["h"], res["y_perm"] = h, y
    sh = None
    if shared is not None:
        rows = DenseRows(x.shape[0], m_tile, x.device)
        _, ys = B.moe_grouped_swiglu(x, rows.offsets, rows.tile_expert, shared.w1, shared.w3,
                                     shared.w2, m_tile, m_cap=rows.m_cap, workspace=ws,
                                     rows_used=rows.T)
        sh = ys[: x.shape[0]]
        res["shared"] = sh
    res["out"] = B.moe_combine(y, p["dst_row"], topk_w, shared=sh, m_cap=m_cap)
    return res


def moe_layer_masked_mxfp4(x: torch.Tensor, mw: Mx4Weights, k: int, cap: int,
                           wg: Optional[torch.Tensor] = None,
                           bias: Optional[torch.Tensor] = None,
                           topk_idx: Optional[torch.Tensor] = None,
                           topk_w: Optional[torch.Tensor] = None,
                           shared: Optional[SharedExperts] = None, renorm: bool = False,
                           split_k: bool = True, shared_m_tile: int = 128) -> dict:
    """moe_layer_masked (bf16 x) with 4-bit expert weights: the rows stay bf16, the weights are
    streamed in 4 bits. ``split_k`` and ``shared_m_tile`` concern the shared experts."""
    E = mw.w1q.shape[0]
    res = {}
    if topk_idx is None:
        topk_idx, topk_w, _ = B.moe_route(x, wg, k, bias=bias, renorm=renorm)
    res["topk_idx"], res["topk_w"] = topk_idx, topk_w
    p = B.moe_permute_masked(x, topk_idx, E, cap)
    res.update(p)
    h, y = X.moe_grouped_swiglu_masked_mxfp4(p["x_masked"], p["counts"], mw.w1q, mw.w1s, mw.w3q,
                                             mw.w3s, mw.w2q, mw.w2s, cap)
    res["h"], res["y_perm"] = h, y
    sh = None
    if shared is not None:
        ws = B.grouped_workspace(x.device) if split_k else None
        rows = DenseRows(x.shape[0], shared_m_tile, x.device)
        _, ys = B.moe_grouped_swiglu(x, rows.offsets, rows.tile_expert, shared.w1, shared.w3,
                                     shared.w2, shared_m_tile, m_cap=rows.m_cap, workspace=ws,
                                     rows_used=rows.T)
        sh = ys[: x.shape[0]]
        res["shared"] = sh
    res["out"] = B.moe_combine(y, p["dst_row"], topk_w, shared=sh, m_cap=p["m_cap"])
    return res


def _experts_backward(dy, x_rows, ab, h, offsets, tile_expert, w1, w3, w2, m_tile, m_cap, ws,
                      rows_used=None, counts=None):
    """dgrad and wgrad of one grouped SwiGLU FFN over rows [0, m_cap) (section 5 of
    "Expert Parallelism (EP)": the m-grouped fc mirrors into an m-grouped dgrad and a
    k-grouped wgrad). Returns (dab, dX, dw1, dw3, dw2)."""
    F, D = w1.shape[1], w1.shape[2]
    ru, c = rows_used, counts
    dab = B.moe_grouped_dgrad_swiglu(dy, offsets, tile_expert, w2, ab, m_tile, m_cap,
                                     workspace=ws, rows_used=ru, counts=c)
    dX = B.moe_grouped_dgrad_fc1(dab, offsets, tile_expert, w1, w3, m_tile, m_cap, workspace=ws,
                                 rows_used=ru, counts=c)
    dw1, dw3 = B.moe_grouped_wgrad(dab, x_rows, offsets, m_tile, m_cap, NS=F, rows_used=ru,
                                   counts=c)
    dw2, _ = B.moe_grouped_wgrad(dy, h, offsets, m_tile, m_cap, NS=D, rows_used=ru, counts=c)
    return dab, dX, dw1, dw3, dw2


def _experts_backward_ckpt8(dout_rows, x_rows, codes, scales, offsets, tile_expert, w1, w3, w2,
                            m_tile, m_cap, ws, rows_used=None, counts=None, **weights):
    """_experts_backward from an 8-bit checkpoint, for the unweighted output gradient's rows;
    ``weights``: topk_w with src_row and dst_row. ``x_rows`` is called for the rows of x once
    they are needed. Returns (dab, dX, dw1, dw3, dw2, dtopk_w)."""
    F, D = w1.shape[1], w1.shape[2]
    ru, c = rows_used, counts
    dab, hw, dtw = X.moe_grouped_dgrad_swiglu_ckpt8(dout_rows, offsets, tile_expert, w2, codes,
                                                    scales, m_tile, m_cap, workspace=ws,
                                                    rows_used=ru, counts=c, **weights)
    dw2, _ = B.moe_grouped_wgrad(dout_rows, hw, offsets, m_tile, m_cap, NS=D, rows_used=ru,
                                 counts=c)
    del hw
    dX = B.moe_grouped_dgrad_fc1(dab, offsets, tile_expert, w1, w3, m_tile, m_cap, workspace=ws,
                                 rows_used=ru, counts=c)
    dw1, dw3 = B.moe_grouped_wgrad(dab, x_rows(), offsets, m_tile, m_cap, NS=F, rows_used=ru,
                                   counts=c)
    return dab, dX, dw1, dw3, dw2, dtw


def _layer_backward_ckpt8(fwd, dout, x, w1, w3, w2, m_tile, shared, split_k):
    """moe_layer_backward from ``moe_layer(save_for_backward="mxfp8")``: the output gradient
    and x are moved to the permuted rows by the forward's routing, the top-k weights are
    applied behind the dgrad of fc2."""
    E = w1.shape[0]
    m_cap, offs, te, counts = fwd["m_cap"], fwd["offsets"], fwd["tile_expert"], fwd["counts"]
    ws = B.grouped_workspace(x.device) if split_k else None
    rows = lambda t: B.moe_permute(t, fwd["topk_idx"], E, m_tile, m_cap)["x_perm"]  # noqa: E731
    res = {}
    res["dab"], dX, res["dw1"], res["dw3"], res["dw2"], res["dtopk_w"] = _experts_backward_ckpt8(
        rows(dout), lambda: rows(x), fwd["ab_codes"], fwd["ab_scales"], offs, te, w1, w3, w2,
        m_tile, m_cap, ws, counts=counts, src_row=fwd["src_row"], dst_row=fwd["dst_row"],
        topk_w=fwd["topk_w"])
    res["dx_perm"] = dX
    dxs = None
    if shared is not None:
        T = x.shape[0]
        sr = DenseRows(T, m_tile, x.device)
        _, dXs, res["dws1"], res["dws3"], res["dws2"], _ = _experts_backward_ckpt8(
            dout, lambda: x, fwd["shared_ab_codes"], fwd["shared_ab_scales"], sr.offsets,
            sr.tile_expert, shared.w1, shared.w3, shared.w2, m_tile, sr.m_cap, ws, rows_used=T)
        dxs = res["dx_shared"] = dXs[:T]
    res["dx"] = B.moe_combine(dX, fwd["dst_row"], None, shared=dxs, m_cap=m_cap)
    return res


def moe_layer_backward(fwd: dict, dout: torch.Tensor, x: torch.Tensor, w1: torch.Tensor,
                       w3: torch.Tensor, w2: torch.Tensor, m_tile: int,
                       shared: Optional[SharedExperts] = None, split_k: bool = True) -> dict:
    """Backward of ``moe_layer(..., save_for_backward=True)`` for the output gradient
    ``dout`` [T, D], as the mirror of each forward step ("Expert Parallelism (EP)",
    section 5): combine -> dispatch (moe_combine_backward), grouped SwiGLU -> dgrad +
    wgrad, permute -> unpermute (moe_combine without weights). Routing is taken as
    given; its weights get their gradient ``dtopk_w``. Weight gradients are float32
    (``dw1``, ``dw3`` [E,F,D], ``dw2`` [E,D,F]; for the shared experts ``dws1``, ``dws3``
    [1,S*Fs,D] and ``dws2`` [1,D,S*Fs], the concatenated layout of SharedExperts). After
    ``save_for_backward="mxfp8"`` the same from the 8-bit checkpoint, without ``dy_perm``."""
    if "ab_codes" in fwd:
        return _layer_backward_ckpt8(fwd, dout, x, w1, w3, w2, m_tile, shared, split_k)
    m_cap = fwd["m_cap"]
    offs, te = fwd["offsets"], fwd["tile_expert"]
    ws = B.grouped_workspace(x.device) if split_k else None
    res = {}
    dy, dtw = B.moe_combine_backward(dout, fwd["y_perm"], fwd["src_row"], offs, fwd["dst_row"],
                                     fwd["topk_w"], m_cap=m_cap)
    res["dy_perm"], res["dtopk_w"] = dy, dtw
    dab, dX, dw1, dw3, dw2 = _experts_backward(dy, fwd["x_perm"], fwd["ab"], fwd["h"], offs, te,
                                               w1, w3, w2, m_tile, m_cap, ws,
                                               counts=fwd["counts"])
    res.update(dab=dab, dx_perm=dX, dw1=dw1, dw3=dw3, dw2=dw2)
    dxs = None
    if shared is not None:
        T = x.shape[0]
        rows = DenseRows(T, m_tile, x.device)
        _, dXs, dws1, dws3, dws2 = _experts_backward(
            dout, x, fwd["shared_ab"], fwd["shared_h"], rows.offsets, rows.tile_expert,
            shared.w1, shared.w3, shared.w2, m_tile, rows.m_cap, ws, rows_used=T)
        dxs = dXs[:T]
        res.update(dx_shared=dxs, dws1=dws1, dws3=dws3, dws2=dws2)
    res["dx"] = B.moe_combine(dX, fwd["dst_row"], None, shared=dxs, m_cap=m_cap)
    return res


def moe_block(resid: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, k: int,
              m_tile: int, wg: torch.Tensor, x: Optional[torch.Tensor] = None,
              gamma_pre: Optional[torch.Tensor] = None,
              gamma_post: Optional[torch.Tensor] = None,
              gamma_next: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
              scale: float = 1.0, eps: float = 1e-6, bias: Optional[torch.Tensor] = None,
              shared: Optional[SharedExperts] = None, renorm: bool = False, split_k: bool = True,
              save_for_backward: Union[bool, str] = False) -> dict:
    """A residual block around the layer: x = norm(resid) with gain ``gamma_pre`` (or ``x`` given,
    as the block before left it in its x_next), the layer's route, permute and experts on x, and
    in place of its combine the block's border (moe_combine_norm): out = resid + scale * gate *
    norm(layer(x)) with gain ``gamma_post`` (no norm without), x_next = norm(out) with gain
    ``gamma_next``. Returns the layer's intermediates, out, x_next and with gamma_pre x.
    ``save_for_backward`` as in moe_layer, for moe_block_backward."""
    if (x is None) == (gamma_pre is None):
        raise ValueError("x or gamma_pre, one of the two")
    rstd = None
    if x is None:
        x, rstd = K.moe_norm(resid, gamma_pre, eps=eps)
    res, y, sh = _layer_rows(x, w1, w3, w2, k, m_tile, wg, bias, None, None, shared, renorm,
                             split_k, save_for_backward, want_logits=bool(save_for_backward))
    res.update(K.moe_combine_norm(resid, y, res["dst_row"], res["topk_w"], shared=sh, gate=gate,
                                  gamma_post=gamma_post, gamma_next=gamma_next, scale=scale,
                                  eps=eps, save=bool(save_for_backward)))
    if rstd is not None:
        res["x"], res["rstd_pre"] = x, rstd
    return res


def moe_block_backward(fwd: dict, dout: Optional[torch.Tensor], resid: torch.Tensor,
                       w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor, m_tile: int,
                       wg: torch.Tensor, x: Optional[torch.Tensor] = None,
                       dx_next: Optional[torch.Tensor] = None,
                       gamma_pre: Optional[torch.Tensor] = None,
                       gamma_post: Optional[torch.Tensor] = None,
                       gamma_next: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                       shared: Optional[SharedExperts] = None, renorm: bool = False,
                       split_k: bool = True,
                       dlogits_add: Optional[torch.Tensor] = None) -> dict:
    """Backward of ``moe_block(..., save_for_backward=...)`` with the same arguments, from the
    gradients of out (``dout``) and of x_next (``dx_next``), either None for zero. Returns the
    layer backward's results (``dx`` the whole gradient of x: experts, shared experts and
    router), the router's ``dlogits``, ``dwg`` and ``dbias``, ``dgate``, ``dgamma_post``,
    ``dgamma_next`` where those inputs were given, and the residual's gradient: with gamma_pre
    ``dresid`` is that of resid through both ways, and ``dgamma_pre`` is there; with x given it is
    the one beside x, and the block before takes it as its dout and dx as its dx_next.
    ``dlogits_add`` [T, E] float32: the gradient of a loss on the logits."""
    if gamma_pre is not None:
        x = fwd["x"]
    elif x is None:
        raise ValueError("x or gamma_pre, as in the forward")
    bb = K.moe_combine_norm_backward(dout, fwd["u"], out=fwd["out"], rstd_post=fwd.get("rstd_post"),
                                     rstd_next=fwd.get("rstd_next"), dx_next=dx_next, gate=gate,
                                     gamma_post=gamma_post, gamma_next=gamma_next, scale=scale)
    res = moe_layer_backward(fwd, bb.pop("du"), x, w1, w3, w2, m_tile, shared=shared,
                             split_k=split_k)
    res.update(K.moe_route_backward(res["dtopk_w"], fwd["topk_idx"], fwd["logits"], x, wg,
                                    renorm=renorm, dlogits_add=dlogits_add, dx_add=res["dx"]))
    res.update(bb)
    if gamma_next is not None and dx_next is None:   # nothing came through that norm
        res["dgamma_next"] = torch.zeros(gamma_next.shape, dtype=torch.float32, device=x.device)
    if gamma_pre is not None:
        res["dresid"], res["dgamma_pre"] = K.moe_norm_backward(res["dx"], resid, gamma_pre,
                                                               fwd["rstd_pre"],
                                                               dresid=bb["dresid"])
    return res


def moe_block_few(resid: torch.Tensor, weights, k: int, wg: torch.Tensor,
                  x: Optional[torch.Tensor] = None, gamma_pre: Optional[torch.Tensor] = None,
                  gamma_post: Optional[torch.Tensor] = None,
                  gamma_next: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, scale: float = 1.0, eps: float = 1e-6,
                  bias: Optional[torch.Tensor] = None, shared: Optional[SharedExperts] = None,
                  renorm: bool = False) -> dict:
    """moe_block for the at most 32 tokens of a decode step: the layer is moe_layer_few, or with
    ``weights`` an Mx4Weights moe_layer_few_mxfp4 (else ``weights`` is (w1, w3, w2)). Returns
    out, x_next, topk_idx and topk_w. From about 8 tokens over wide 4-bit experts
    moe_layer_masked_mxfp4 between moe_norm and moe_combine_norm (its out as ``shared``) is faster:
    8 experts of D = 4096, F = 14336, top-2, 32 tokens 167 us a layer against 251."""
    if (x is None) == (gamma_pre is None):
        raise ValueError("x or gamma_pre, one of the two")
    if x is None:
        x, _ = K.moe_norm(resid, gamma_pre, eps=eps)
    kw = dict(wg=wg, bias=bias, shared=shared, renorm=renorm)
    if isinstance(weights, Mx4Weights):
        res = K.moe_layer_few_mxfp4(x, weights, k, **kw)
    else:
        res = K.moe_layer_few(x, *weights, k, **kw)
    res.update(K.moe_combine_norm(resid, shared=res.pop("out"), gate=gate, gamma_post=gamma_post,
                                  gamma_next=gamma_next, scale=scale, eps=eps))
    return res
