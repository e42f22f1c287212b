"""Workloads of the block-scaled operators of the expert layer: 4-bit quantisation, the 4-bit
grouped products of prefill and decode, and the 8-bit checkpoint of fc1's pre-activations.

Every case names its operator in ``op``:

``quantize``  rows to 4-bit codes (E2M1) with one power-of-two scale per 32 values, and back;
``product``   one grouped product of 4-bit rows and 4-bit expert weights over contiguous
              segments: fc1 with silu(a)*b, or fc2;
``decode``    bf16 rows in fixed slabs per expert through 4-bit weights, fc1 and fc2;
``save``      fc1 of a training step that keeps its pre-activations in 8 bits (E4M3, one
              power-of-two scale per 32 values), and their values read back;
``use``       the backward of fc2 and the activation from such a checkpoint.

``own`` selects the library's kernels; otherwise ``run`` computes the same in elementary torch
operations in float32. Row layout and routing follow the library: expert e's rows are
[offsets[e], offsets[e+1]), padded to a multiple of ``mt`` with zero rows.
"""
import math

import torch

own = False

DEV = "cuda"
LUT4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the hidden rows of one decode batch on their way into a 4-bit product
        dict(name="quantize_decode_batch", op="quantize", R=64, C=4096, dtype="bf16", ksteps=False),
        # fc1's output of a 16384-token, top-4 batch before a 4-bit fc2, in the product's layout
        dict(name="quantize_prefill_hidden", op="quantize", R=69632, C=2048, dtype="bf16", ksteps=True),
        # the narrow experts of an expert-tensor-parallel shard: slots of other ranks are absent
        dict(name="fc1_etp_shard", op="product", fc=1, T=2025, k=8, E=32, D=7168, F=512, mt=128, skew=0.1, absent=0.05),
        # few wide experts, the largest product
        dict(name="fc1_dense_experts", op="product", fc=1, T=4096, k=2, E=8, D=4096, F=14336, mt=128, skew=0.05, absent=0.0),
        # many fine experts; F is not a multiple of 256
        dict(name="fc2_fine_experts", op="product", fc=2, T=8192, k=6, E=64, D=2048, F=1408, mt=128, skew=0.2, absent=0.0),
        # one user's next token
        dict(name="decode_one_token", op="decode", T=1, k=6, E=64, D=2048, F=1408, cap=16, skew=0.2),
        # 64 users over few wide experts: every expert is hit
        dict(name="decode_dense_experts", op="decode", T=64, k=2, E=8, D=4096, F=14336, cap=64, skew=0.05),
        # 128 users over many fine experts
        dict(name="decode_fine_experts", op="decode", T=128, k=6, E=64, D=2048, F=1408, cap=128, skew=0.2),
        # a short, odd fine-tuning batch
        dict(name="save_short_batch", op="save", T=389, k=2, E=8, D=512, F=1088, mt=64, skew=0.3, absent=0.0),
        # a training step's fc1 over many fine experts
        dict(name="save_fine_experts", op="save", T=8192, k=6, E=64, D=2048, F=1408, mt=128, skew=0.2, absent=0.0),
        dict(name="use_short_batch", op="use", T=389, k=2, E=8, D=512, F=1088, mt=64, skew=0.3, absent=0.05),
        dict(name="use_fine_experts", op="use", T=8192, k=6, E=64, D=2048, F=1408, mt=128, skew=0.2, absent=0.0),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "decode", "decode", "save", "use"])
    most = max(work(c)["flops"] for c in listed())
    while True:
        if op == "quantize":
            ksteps = rng.random() < 0.5
            c = dict(op=op, R=_log(rng, 1, 65536), C=_log(rng, 128, 16384, 128 if ksteps else 32), dtype=rng.choice(["bf16", "bf16", "f32"]), ksteps=ksteps)
            if c["R"] * c["C"] <= 69632 * 2048:
                return c
            continue
        E = _log(rng, 1, 128)
        c = dict(op=op, T=_log(rng, 1, 256 if op == "decode" else 16384), k=rng.randint(1, min(E, 8)), E=E, D=_log(rng, 128, 8192, 128),
                 F=_log(rng, 128, 14336, 64 if op in ("save", "use") else 128))
        if op == "decode":
            c["cap"] = 16 * rng.randint(1, 16)
            c["skew"] = rng.uniform(0.0, 0.6)
            if 3 * E * c["D"] * c["F"] > 2 * 3 * 8 * 4096 * 14336:
                continue
        else:
            c["mt"] = rng.choice([16, 32, 64, 128, 256])
            c["skew"] = rng.uniform(0.0, 0.4)
            c["absent"] = rng.choice([0.0, 0.0, 0.1])
            if op == "product":
                c["fc"] = rng.choice([1, 2])
            if E * c["D"] * c["F"] > 2 * 8 * 4096 * 14336:
                continue
            # the padded plain form costs E times the longest segment
            if work(c)["flops"] * (1.0 + 4.0 * c["skew"]) > most:
                continue
        return c


def work(case):
    """Bytes and operations of one pass: every input once, every output once."""
    op = case["op"]
    q4, q8 = 17.0 / 32.0, 33.0 / 32.0
    if op == "quantize":
        n, s = case["R"] * case["C"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (2 * s + 2 * q4), "flops": 4.0 * n}
    T, k, E, D, F = (case[x] for x in ("T", "k", "E", "D", "F"))
    n = T * k * (1.0 - case.get("absent", 0.0))
    hit = E * (1.0 - (1.0 - k / E) ** T)   # experts that some token takes
    if op == "product":
        if case["fc"] == 1:
            return {"bytes": hit * 2 * D * F * q4 + n * (D * q4 + 2 * F), "flops": 4.0 * n * D * F}
        return {"bytes": hit * D * F * q4 + n * (F * q4 + 2 * D), "flops": 2.0 * n * D * F}
    if op == "decode":
        n = min(n, hit * case["cap"])
        return {"bytes": hit * 3 * D * F * q4 + n * (4 * D + 4 * F), "flops": 6.0 * n * D * F}
    if op == "save":
        return {"bytes": hit * 4 * D * F + n * (2 * D + 2 * F + 2 * F * (2 * q8 + 2)), "flops": 4.0 * n * D * F}
    return {"bytes": hit * 2 * D * F + n * (2 * D + 2 * F * q8 + 6 * F), "flops": 2.0 * n * D * F}


# ---------------------------------------------------------------- inputs


def _pow2(x):
    """2^x of integers x in [-149, 127], exactly, in float32 (the power function may be off by an ulp)."""
    return ((x.long() + 1023) << 52).view(torch.float64).float()


def _block_exponent(v, mantissa, shift):
    """v [..., 32]: the smallest integer X >= -127 with max|v| <= mantissa * 2^(X + shift)."""
    m, e = torch.frexp(v.abs().amax(-1))
    x = torch.where(m <= mantissa, e - shift, e - shift + 1)
    return torch.where(m == 0, torch.full_like(x, -127), x.clamp(min=-127))


def _e2m1(a):
    """|v| / 2^X in [0, 6] rounded to {0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties to the even code."""
    return torch.where(a < 2, torch.round(a * 2) * 0.5, torch.where(a < 4, torch.round(a), torch.round(a * 0.5) * 2))


def _words(scales):
    """Scale rows [R, C/32] in k-step words [C/128, R, 4]."""
    R, nb = scales.shape
    return scales.view(R, nb // 4, 4).permute(1, 0, 2).contiguous()


def _to_mx4(x):
    """Rows x [R, C] float32: packed codes [R, C/2] (even element in the low half) and scale bytes [R, C/32]."""
    v = x.reshape(x.shape[0], -1, 32)
    X = _block_exponent(v, 0.75, 3)
    q = _e2m1(v.abs() * _pow2(-X[..., None]))
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q * 0.5 + 4)).to(torch.uint8)
    code = torch.where(v < 0, code | 8, code).reshape(x.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (X + 127).to(torch.uint8)


def _to_mx8(x):
    """Rows x [R, C] float32: E4M3 codes [R, C] and scale bytes [R, C/32]."""
    v = x.reshape(x.shape[0], -1, 32)
    X = _block_exponent(v, 0.875, 9)
    q = (v * _pow2(-X[..., None])).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(x.shape), (X + 127).to(torch.uint8)


def _mx4_weights(g, E, N, K):
    """Random weights [E, N, K] ~ N(0, 1/sqrt(K)) as codes [E, N, K/2] and k-step words [K/128, E*N, 4]."""
    codes, scales = [], []
    for _ in range(E):
        q, s = _to_mx4(torch.randn(N, K, device=DEV, generator=g) / math.sqrt(K))
        codes.append(q)
        scales.append(s)
    return torch.stack(codes), _words(torch.cat(scales))


def _route(case, g):
    """Top-k of random logits with a spread of ``skew`` between the experts, and the weights."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn(T, E, device=DEV, generator=g) + 2.0 * case["skew"] * torch.randn(E, device=DEV, generator=g)
    top, idx = torch.topk(logits, k, dim=1)
    w = torch.softmax(top, dim=1)
    if case.get("absent", 0.0) > 0:
        idx = torch.where(torch.rand(T, k, device=DEV, generator=g) < case["absent"], torch.full_like(idx, -1), idx)
    return idx, w


def _ranks(idx, E):
    """Each slot's stable rank in its expert's list, and the experts' counts."""
    flat = idx.reshape(-1)
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    first = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device=DEV)
    rank = rank - torch.cat([first, first.new_zeros(1)])[torch.where(flat < 0, E, flat)]
    return rank.reshape(idx.shape), counts


def _segments(case, g):
    """The permuted layout of random routing, as the library's permute writes it."""
    T, k, E, mt = case["T"], case["k"], case["E"], case["mt"]
    idx, w = _route(case, g)
    rank, counts = _ranks(idx, E)
    seg = -(-counts // mt) * mt
    offsets = torch.cat([seg.new_zeros(1), torch.cumsum(seg, 0)])
    m_cap = (T * k + min(E, T * k) * (mt - 1)) // mt * mt
    dst = torch.where(idx >= 0, offsets[idx.clamp(min=0)] + rank, torch.full_like(idx, -1))
    src = torch.full((m_cap + 1,), -1, dtype=torch.int32, device=DEV)   # absent slots go to the spare place
    src[torch.where(dst < 0, m_cap, dst).reshape(-1)] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    src = src[:m_cap].clone()
    tiles = torch.searchsorted(offsets[1:], torch.arange(0, m_cap, mt, device=DEV), right=True)
    tiles = torch.where(torch.arange(0, m_cap, mt, device=DEV) < offsets[-1], tiles, torch.full_like(tiles, -1))
    i32 = torch.int32
    return {"offsets": offsets.to(i32), "counts": counts.to(i32), "dst_row": dst.to(i32), "src_row": src, "topk_w": w,
            "tile_expert": tiles.to(i32), "m_cap": m_cap, "longest": max(1, int(seg.max()))}


def _segment_rows(s, g, K):
    """bf16 rows [m_cap, K] ~ N(0, 1) of the layout's tokens, zero in the pad rows."""
    x = torch.randn(s["m_cap"], K, device=DEV, generator=g)
    return torch.where(s["src_row"][:, None] >= 0, x, torch.zeros_like(x)).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        # hidden rows of different norms, some values far out
        x = torch.randn(case["R"], case["C"], device=DEV, generator=g)
        x = x * torch.exp(torch.randn(case["R"], 1, device=DEV, generator=g)) * torch.exp(0.5 * torch.randn(case["R"], case["C"], device=DEV, generator=g))
        return {"case": dict(case), "x": x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)}
    E, D, F = case["E"], case["D"], case["F"]
    if op == "decode":
        cap = case["cap"]
        idx, _ = _route(case, g)
        _, counts = _ranks(idx, E)
        s = {"case": dict(case), "counts": counts.clamp(max=cap).to(torch.int32)}
        s["x"] = torch.randn(E * cap, D, device=DEV, generator=g).to(torch.bfloat16)
        s["w1q"], s["w1s"] = _mx4_weights(g, E, F, D)
        s["w3q"], s["w3s"] = _mx4_weights(g, E, F, D)
        s["w2q"], s["w2s"] = _mx4_weights(g, E, D, F)
        # a server's activation buffers: rows past an expert's count stay as they are
        s["h"] = torch.zeros(E * cap, F, dtype=torch.bfloat16, device=DEV)
        s["y"] = torch.zeros(E * cap, D, dtype=torch.bfloat16, device=DEV)
        return s
    s = _segments(case, g)
    s["case"] = dict(case)
    m_cap = s["m_cap"]
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    if op == "product":
        K, N = (D, F) if case["fc"] == 1 else (F, D)
        s["aq"], rows = _to_mx4(_segment_rows(s, g, K).float())
        s["as"] = _words(rows)
        s["w1q"], s["w1s"] = _mx4_weights(g, E, N, K)
        if case["fc"] == 1:
            s["w3q"], s["w3s"] = _mx4_weights(g, E, N, K)
        s["out"] = torch.zeros(m_cap, N, **bf16)   # rows past the last segment stay as they are
    elif op == "save":
        s["x"] = _segment_rows(s, g, D)
        s["w1"] = (torch.randn(E, F, D, device=DEV, generator=g) / math.sqrt(D)).to(torch.bfloat16)
        s["w3"] = (torch.randn(E, F, D, device=DEV, generator=g) / math.sqrt(D)).to(torch.bfloat16)
        s["h"] = torch.zeros(m_cap, F, **bf16)
        s["ab_codes"] = torch.zeros(m_cap, 2 * F, dtype=torch.uint8, device=DEV)
        s["ab_scales"] = torch.zeros(m_cap, 2 * F // 32, dtype=torch.uint8, device=DEV)
    else:
        s["dout"] = _segment_rows(s, g, D)
        s["ab_codes"], s["ab_scales"] = _to_mx8(_segment_rows(s, g, 2 * F).float())
        s["w2"] = (torch.randn(E, D, F, device=DEV, generator=g) / math.sqrt(F)).to(torch.bfloat16)
        s["dab"] = torch.zeros(m_cap, 2 * F, **bf16)
        s["hw"] = torch.zeros(m_cap, F, **bf16)
    # the grouped calls' workspace: one 256 x 256 float32 tile per compute unit
    s["ws"] = torch.empty(torch.cuda.get_device_properties(0).multi_processor_count << 18, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- one pass


def _library():
    import routing_permute_grouped_amd
    return routing_permute_grouped_amd


def run(s):
    op = s["case"]["op"]
    return {"quantize": _quantize, "product": _product, "decode": _decode, "save": _save, "use": _use}[op](s)


def _from_mx4(codes, scales):
    """Values [..., C] in float32 of codes [..., C/2] and scale rows [..., C/32]."""
    lut = torch.tensor(LUT4 + tuple(-v for v in LUT4), device=codes.device)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1)
    v = v.reshape(*scales.shape, 32) * _pow2(scales.long() - 127)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _from_mx8(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().reshape(*scales.shape, 32)
    return (v * _pow2(scales.long() - 127)[..., None]).reshape(codes.shape)


def _rows_of(words):
    """k-step words [C/128, R, 4] as scale rows [R, C/32]."""
    return words.permute(1, 0, 2).reshape(words.shape[1], -1)


def _silu(a):
    return a / (1 + torch.exp(-a))


def _batched(s, rows, weights):
    """rows [m_cap, K] times the transposed weights [E, N, K] of each row's expert, [m_cap, N], zero past
    the last segment: one batched product over the segments, padded to the longest."""
    start, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = start[:, None] + torch.arange(s["longest"], device=rows.device)
    padded = rows[torch.where(at < end[:, None], at, torch.zeros_like(at))]
    out = torch.bmm(padded, weights.transpose(1, 2))
    r = torch.arange(s["m_cap"], device=rows.device)
    e = torch.searchsorted(end, r, right=True).clamp(max=end.numel() - 1)
    got = out[e, (r - start[e]).clamp(max=s["longest"] - 1)]
    return torch.where(r[:, None] < end[-1], got, torch.zeros_like(got))


def _quantize(s):
    x, c = s["x"], s["case"]
    if own:
        rpg = _library()
        layout = rpg.MOE_MX_KSTEPS if c["ksteps"] else rpg.MOE_MX_ROWS
        q, scales = rpg.moe_quantize_mxfp4(x, layout=layout)
        return rpg.moe_dequantize_mxfp4(q, scales, layout=layout, dtype=x.dtype)
    v = x.float().reshape(c["R"], -1, 32)
    X = _block_exponent(v, 0.75, 3)[..., None]
    q = _e2m1(v.abs() * _pow2(-X)) * _pow2(X)
    return torch.where(v < 0, -q, q).reshape(x.shape).to(x.dtype)


def _product(s):
    c = s["case"]
    if own:
        rpg = _library()
        if c["fc"] == 1:
            return rpg.moe_grouped_fc1_swiglu_mxfp4(s["aq"], s["as"], s["offsets"], s["tile_expert"], s["w1q"], s["w1s"], s["w3q"], s["w3s"],
                                                    c["mt"], h=s["out"], workspace=s["ws"], counts=s["counts"])
        return rpg.moe_grouped_fc2_mxfp4(s["aq"], s["as"], s["offsets"], s["tile_expert"], s["w1q"], s["w1s"], c["mt"], y_perm=s["out"],
                                         workspace=s["ws"], counts=s["counts"])
    x = _from_mx4(s["aq"], _rows_of(s["as"]))
    a = _batched(s, x, _from_mx4(s["w1q"], _rows_of(s["w1s"]).reshape(*s["w1q"].shape[:2], -1)))
    if c["fc"] == 1:
        a = _silu(a) * _batched(s, x, _from_mx4(s["w3q"], _rows_of(s["w3s"]).reshape(*s["w3q"].shape[:2], -1)))
    return a.to(torch.bfloat16)


def _decode(s):
    c = s["case"]
    E, cap = c["E"], c["cap"]
    if own:
        rpg = _library()
        return rpg.moe_grouped_swiglu_masked_mxfp4(s["x"], s["counts"], s["w1q"], s["w1s"], s["w3q"], s["w3s"], s["w2q"], s["w2s"], cap,
                                                   h=s["h"], y=s["y"])
    x = s["x"].float().reshape(E, cap, -1)
    w = [_from_mx4(s[n + "q"], _rows_of(s[n + "s"]).reshape(*s[n + "q"].shape[:2], -1)) for n in ("w1", "w3", "w2")]
    there = (torch.arange(cap, device=x.device) < s["counts"][:, None])[..., None]
    h = _silu(torch.bmm(x, w[0].transpose(1, 2))) * torch.bmm(x, w[1].transpose(1, 2))
    h = torch.where(there, h, torch.zeros_like(h))
    y = torch.bmm(h, w[2].transpose(1, 2))
    return h.reshape(E * cap, -1).to(torch.bfloat16), y.reshape(E * cap, -1).to(torch.bfloat16)


def _save(s):
    c = s["case"]
    if own:
        rpg = _library()
        rpg.moe_grouped_fc1_swiglu_ckpt8(s["x"], s["offsets"], s["tile_expert"], s["w1"], s["w3"], c["mt"], h=s["h"], ab_codes=s["ab_codes"],
                                         ab_scales=s["ab_scales"], workspace=s["ws"], counts=s["counts"])
        return s["h"], rpg.moe_dequantize_mxfp8(s["ab_codes"], s["ab_scales"])
    x = s["x"].float()
    a, b = _batched(s, x, s["w1"].float()), _batched(s, x, s["w3"].float())
    h = _silu(a) * b
    v = torch.cat([a, b], 1).reshape(s["m_cap"], -1, 32)
    X = _block_exponent(v, 0.875, 9)[..., None]
    v = v * _pow2(-X)
    # E4M3: 3 fraction bits, subnormal below 2^-6
    step = _pow2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 4)
    v = torch.round(v / step) * step * _pow2(X)
    return h.to(torch.bfloat16), v.reshape(s["m_cap"], -1).to(torch.bfloat16)


def _use(s):
    c = s["case"]
    if own:
        rpg = _library()
        return rpg.moe_grouped_dgrad_swiglu_ckpt8(s["dout"], s["offsets"], s["tile_expert"], s["w2"], s["ab_codes"], s["ab_scales"], c["mt"],
                                                  src_row=s["src_row"], dst_row=s["dst_row"], topk_w=s["topk_w"], dab=s["dab"], hw=s["hw"],
                                                  workspace=s["ws"], counts=s["counts"])
    F = c["F"]
    u = _batched(s, s["dout"].float(), s["w2"].float().transpose(1, 2))
    ab = _from_mx8(s["ab_codes"], s["ab_scales"])
    a, b = ab[:, :F], ab[:, F:]
    sg = 1 / (1 + torch.exp(-a))
    src = s["src_row"].long()
    w = torch.where(src >= 0, s["topk_w"].reshape(-1)[src.clamp(min=0)], torch.zeros((), device=a.device))[:, None]
    h = a * sg * b
    dab = torch.cat([w * u * b * (sg * (1 + a * (1 - sg))), w * u * (a * sg)], 1)
    dots = (u * h).sum(1)
    dst = s["dst_row"].long()
    dtw = torch.where(dst >= 0, dots[dst.clamp(min=0)], torch.zeros((), device=a.device))
    return dab.to(torch.bfloat16), (w * h).to(torch.bfloat16), dtw


# ---------------------------------------------------------------- the definition in 64 bits


def _power(x):
    """2^x of integer-valued x in [-300, 300] in float64, from a table of exact powers."""
    return torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=x.device)[x.long() + 300]


def _value4(codes, scales):
    """The same values from sign, exponent and fraction of each code, in float64."""
    nib = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.uint8, device=codes.device)
    nib[..., 0::2] = codes % 16
    nib[..., 1::2] = codes // 16
    sign = 1.0 - 2.0 * (nib // 8).double()
    ex, fr = ((nib // 2) % 4).double(), (nib % 2).double()
    mag = torch.where(ex == 0, 0.5 * fr, _power(ex - 1) * (1 + 0.5 * fr))
    return sign * mag * _power(scales.double() - 127).repeat_interleave(32, -1)


def _value8(codes, scales):
    sign = 1.0 - 2.0 * (codes // 128).double()
    ex, fr = ((codes // 8) % 16).double(), (codes % 8).double()
    mag = torch.where(ex == 0, fr * 2.0 ** -9, _power(ex - 7) * (1 + fr / 8))
    return sign * mag * _power(scales.double() - 127).repeat_interleave(32, -1)


def _nearest(v, grid, largest):
    """Values of each 32-wide block on ``grid`` (ascending, code order) times the block's power of two:
    the nearest, ties to the even code."""
    blocks = v.reshape(v.shape[0], -1, 32)
    amax = blocks.abs().amax(-1, keepdim=True)
    X = torch.ceil(torch.log2(amax / largest).clamp(min=-200))
    X = torch.where(amax > largest * _power(X), X + 1, X)
    X = torch.where(amax <= largest * _power(X - 1), X - 1, X).clamp(min=-127)
    scale = _power(X)
    a = (blocks.abs() / scale).contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = a - grid[lo], grid[hi] - a
    take = torch.where(down == up, torch.where(hi % 2 == 0, hi, lo), torch.where(up < down, hi, lo))
    return (torch.sign(blocks) * grid[take] * scale).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        grid = torch.tensor(LUT4, dtype=torch.float64, device=DEV)
        rows = max(1, (1 << 24) // case["C"])
        return torch.cat([_nearest(p.double(), grid, 6.0) for p in s["x"].split(rows)])
    E, D, F = case["E"], case["D"], case["F"]

    def weight4(name, e):
        q = s[name + "q"][e]
        per = q.shape[0]
        scale = s[name + "s"][:, e * per:(e + 1) * per]
        return _value4(q, torch.cat([scale[i] for i in range(scale.shape[0])], 1))

    f64 = dict(dtype=torch.float64, device=DEV)
    if op == "decode":
        cap, counts = case["cap"], s["counts"].tolist()
        h, y = torch.zeros(E * cap, F, **f64), torch.zeros(E * cap, D, **f64)
        for e in range(E):
            if counts[e]:
                rows = slice(e * cap, e * cap + counts[e])
                x = s["x"][rows].double()
                a, b = x @ weight4("w1", e).T, x @ weight4("w3", e).T
                h[rows] = a * torch.sigmoid(a) * b
                y[rows] = h[rows] @ weight4("w2", e).T
        return h, y
    ends = s["offsets"].tolist()
    m_cap = s["m_cap"]
    if op == "product":
        out = torch.zeros(m_cap, F if case["fc"] == 1 else D, **f64)
        row_scales = torch.cat([s["as"][i] for i in range(s["as"].shape[0])], 1)
        for e in range(E):
            rows = slice(ends[e], ends[e + 1])
            if ends[e + 1] > ends[e]:
                x = _value4(s["aq"][rows], row_scales[rows])
                a = x @ weight4("w1", e).T
                out[rows] = a * torch.sigmoid(a) * (x @ weight4("w3", e).T) if case["fc"] == 1 else a
        return out
    if op == "save":
        codes = torch.arange(127, dtype=torch.uint8, device=DEV)
        ex, fr = (codes // 8).double(), (codes % 8).double()
        grid = torch.where(ex == 0, fr * 2.0 ** -9, _power(ex - 7) * (1 + fr / 8))
        h, ab = torch.zeros(m_cap, F, **f64), torch.zeros(m_cap, 2 * F, **f64)
        for e in range(E):
            rows = slice(ends[e], ends[e + 1])
            if ends[e + 1] > ends[e]:
                x = s["x"][rows].double()
                a, b = x @ s["w1"][e].double().T, x @ s["w3"][e].double().T
                h[rows] = a * torch.sigmoid(a) * b
                ab[rows] = _nearest(torch.cat([a, b], 1), grid, 448.0)
        return h, ab
    dab, hw = torch.zeros(m_cap, 2 * F, **f64), torch.zeros(m_cap, F, **f64)
    dtw = torch.zeros(case["T"] * case["k"], **f64)
    tw = s["topk_w"].double().reshape(-1)
    for e in range(E):
        rows = slice(ends[e], ends[e + 1])
        if ends[e + 1] > ends[e]:
            u = s["dout"][rows].double() @ s["w2"][e].double()
            ab = _value8(s["ab_codes"][rows], s["ab_scales"][rows])
            a, b = ab[:, :F], ab[:, F:]
            sg = torch.sigmoid(a)
            src = s["src_row"][rows].long()
            w = torch.where(src >= 0, tw[src.clamp(min=0)], 0.0)[:, None]
            h = a * sg * b
            dab[rows, :F] = w * u * b * (sg + a * sg * (1 - sg))
            dab[rows, F:] = w * u * a * sg
            hw[rows] = w * h
            dtw[src[src >= 0]] = (u * h).sum(1)[src >= 0]
    return dab, hw, dtw.reshape(case["T"], case["k"])
