"""GPU tests of the tiled grouped GEMMs on segments that end in whole row blocks of pad rows:
with counts, pad rows are not read (they hold NaN here) and give exact zeros, and the token
rows keep the bits they have beside zero pad rows."""
import numpy as np
import pytest
import torch

import routing_permute_grouped_amd as rpg
from oracle import moe_oracle as orc
from oracle import mx_oracle as mx
from tests import _parity as P
from tests.test_gpu_mxfp4 import bf16

pytestmark = pytest.mark.gpu

# segment lengths and tokens; the blocks of 128 or 256 rows behind the tokens hold none
SEGMENTS = {
    "one_row": ([512], [1]),
    "some": ([512, 256, 0, 768], [100, 0, 0, 300]),
    "half_blocks": ([256, 256], [100, 30]),
    "two_stage_kernel": ([2560], [130]),          # past the ring's row blocks
    "many_experts": ([256] * 65, [3] * 64 + [0]),  # past the ring's experts
}
CALLS = ["fc1", "fc1_ab", "fc2", "fc1_mxfp8", "dgrad_swiglu", "dgrad_fc1", "fc1_mxfp4", "fc2_mxfp4",
         "save", "use"]
MT = 256


def outputs(call, lens, counts, bad, D=384, F=320):
    rng = np.random.default_rng(31)
    E, M = len(lens), sum(lens)
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    te = P.to_dev(np.repeat(np.arange(E), [n // MT for n in lens]).astype(np.int32))
    pad = np.ones(M, dtype=bool)
    for e, c in enumerate(counts):
        pad[offs[e]:offs[e] + c] = False
    do, dc = P.to_dev(offs), P.to_dev(np.array(counts, dtype=np.int32))
    K, N = (F, D) if call.startswith("fc2") else (2 * F, D) if call == "dgrad_fc1" else (D, F)
    if call == "fc2_mxfp4":
        K = 384
    x = rng.standard_normal((M, K))
    x[pad] = np.nan if bad else 0.0
    xd = P.to_dev(bf16(x))

    def weight(*shape):
        return bf16(rng.standard_normal(shape) / 16)

    def empty(cols):
        return P.poison(torch.empty((M, cols), dtype=torch.bfloat16, device="cuda"))

    seg = (do, te)
    if call in ("fc1", "fc1_ab"):
        h, ab = empty(F), empty(2 * F) if call == "fc1_ab" else None
        rpg.moe_grouped_fc1_swiglu(xd, *seg, P.to_dev(weight(E, F, D)), P.to_dev(weight(E, F, D)), MT, M, h,
                                   ab=ab, counts=dc)
        out = [h] + ([ab] if ab is not None else [])
    elif call == "fc2":
        out = [empty(D)]
        rpg.moe_grouped_fc2(xd, *seg, P.to_dev(weight(E, D, F)), MT, M, out[0], counts=dc)
    elif call == "fc1_mxfp8":
        q, s = rpg.moe_quantize_mxfp8(xd, layout=rpg.MOE_MX_KSTEPS)
        w = [t for _ in range(2) for t in rpg.moe_quantize_mxfp8(P.to_dev(weight(E, F, D)), layout=rpg.MOE_MX_KSTEPS)]
        out = [rpg.moe_grouped_fc1_swiglu_mxfp8(q, s, *seg, *w, MT, M, h=empty(F), counts=dc)]
    elif call in ("fc1_mxfp4", "fc2_mxfp4"):
        q, s = rpg.moe_quantize_mxfp4(xd, layout=rpg.MOE_MX_KSTEPS)
        w = [t for _ in range(2 if call[2] == "1" else 1)
             for t in rpg.moe_quantize_mxfp4(P.to_dev(weight(E, N, K)), layout=rpg.MOE_MX_KSTEPS)]
        if call[2] == "1":
            out = [rpg.moe_grouped_fc1_swiglu_mxfp4(q, s, *seg, *w, MT, M, h=empty(N), counts=dc)]
        else:
            out = [rpg.moe_grouped_fc2_mxfp4(q, s, *seg, *w, MT, M, y_perm=empty(N), counts=dc)]
    elif call == "dgrad_swiglu":
        ab = rng.standard_normal((M, 2 * F))
        ab[pad] = np.nan if bad else 0.0
        out = [rpg.moe_grouped_dgrad_swiglu(xd, *seg, P.to_dev(weight(E, D, F)), P.to_dev(bf16(ab)), MT, M,
                                            dab=empty(2 * F), counts=dc)]
    elif call == "dgrad_fc1":
        out = [rpg.moe_grouped_dgrad_fc1(xd, *seg, P.to_dev(weight(E, F, D)), P.to_dev(weight(E, F, D)), MT, M,
                                         dx_perm=empty(D), counts=dc)]
    elif call == "save":
        q = torch.full((M, 2 * F), 0x7F, dtype=torch.uint8, device="cuda")
        s = torch.full((M, F // 16), 255, dtype=torch.uint8, device="cuda")
        h, q, s = rpg.moe_grouped_fc1_swiglu_ckpt8(xd, *seg, P.to_dev(weight(E, F, D)), P.to_dev(weight(E, F, D)),
                                                   MT, M, h=empty(F), ab_codes=q, ab_scales=s, counts=dc)
        out = [h, q, s]
    else:
        q, s = mx.mx8_quantize(rng.standard_normal((M, 2 * F)))
        q[pad], s[pad] = (0x7F, 255) if bad else (0, 0)
        src = np.where(pad, -1, np.cumsum(~pad) - 1).astype(np.int32)
        T = int((~pad).sum())
        tw = rng.random((T, 1)).astype(np.float32)
        dst = np.flatnonzero(~pad).astype(np.int32).reshape(T, 1)
        out = rpg.moe_grouped_dgrad_swiglu_ckpt8(
            xd, *seg, P.to_dev(weight(E, D, F)), P.to_dev(q), P.to_dev(s), MT, M, src_row=P.to_dev(src),
            dst_row=P.to_dev(dst), topk_w=P.to_dev(tw), dab=empty(2 * F), hw=empty(F), counts=dc)
    torch.cuda.synchronize()
    return [P.to_host(o) for o in out], pad


@pytest.mark.parametrize("name", list(SEGMENTS))
@pytest.mark.parametrize("call", CALLS)
def test_row_blocks_of_pad_rows_are_not_read(call, name):
    lens, counts = SEGMENTS[name]
    P.log(f"[segments] {call} {name}")
    ref, _ = outputs(call, lens, counts, bad=False)
    got, pad = outputs(call, lens, counts, bad=True)
    for a, b in zip(got, ref):
        np.testing.assert_array_equal(a.view(np.uint8), b.view(np.uint8))
        if a.shape[0] == pad.size:
            assert not np.any(orc.values64(a[pad]) if a.dtype == np.uint16 else a[pad])
    assert np.any(got[0].view(np.uint8))
