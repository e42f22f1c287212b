"""The block-scaled calls refuse scales whose shape says that they are not in the layout the call
reads: scale rows and k-step words hold the same number of bytes, and words over other rows
have another stride. Tensors are on the CPU, so a call that takes its arguments ends at the
check for the GPU."""
import pytest
import torch

import routing_permute_grouped_amd as rpg

ROWS, KSTEPS = rpg.MOE_MX_ROWS, rpg.MOE_MX_KSTEPS
BF, I32 = torch.bfloat16, torch.int32
E, D, F, M, MT, T, K2 = 2, 256, 384, 64, 16, 8, 2


def z(*shape, dt=torch.uint8):
    return torch.zeros(shape, dtype=dt)


SEG = (z(E + 1, dt=I32), z(M // MT, dt=I32))
CNT = z(E, dt=I32)
W1Q, W1S = z(E, F, D // 2), z(D // 128, E * F, 4)
W2Q, W2S = z(E, D, F // 2), z(F // 128, E * D, 4)


def fc1(xs=None, w1s=W1S, w3s=W1S, rows=M, m_cap=None):
    xs = z(D // 128, M, 4) if xs is None else xs
    return rpg.moe_grouped_fc1_swiglu_mxfp4(z(rows, D // 2), xs, *SEG, W1Q, w1s, W1Q, w3s, MT, m_cap)


def fc2(hs=None, w2s=W2S):
    hs = z(F // 128, M, 4) if hs is None else hs
    return rpg.moe_grouped_fc2_mxfp4(z(M, F // 2), hs, *SEG, W2Q, w2s, MT)


def masked(w1s=W1S, w3s=W1S, w2s=W2S):
    return rpg.moe_grouped_swiglu_masked_mxfp4(z(E * 16, D, dt=BF), CNT, W1Q, w1s, W1Q, w3s, W2Q, w2s, 16)


def permute(xs, **out):
    return rpg.moe_permute_mxfp4(z(T, D // 2), xs, z(T, K2, dt=I32), E, MT, M, out=out)


REFUSED = [
    # scale rows, the quantisation's default, where words are read
    ("xs", lambda: fc1(xs=z(M, D // 32))),
    ("w1s", lambda: fc1(w1s=z(E, F, D // 32))),
    ("w3s", lambda: fc1(w3s=z(E * F, D // 32))),
    ("hs", lambda: fc2(hs=z(M, F // 32))),
    ("w2s", lambda: fc2(w2s=z(E, D, F // 32))),
    ("w1s", lambda: masked(w1s=z(E, F, D // 32))),
    ("w3s", lambda: masked(w3s=z(E, F, D // 32))),
    ("w2s", lambda: masked(w2s=z(E, D, F // 32))),
    ("scales", lambda: rpg.moe_dequantize_mxfp4(z(M, D // 2), z(M, D // 32), layout=KSTEPS)),
    ("scales", lambda: rpg.moe_dequantize_mxfp8(z(M, D), z(M, D // 32), layout=KSTEPS)),
    ("scales", lambda: rpg.moe_quantize_mxfp4(z(M, D, dt=BF), scales=z(M, D // 32), layout=KSTEPS)),
    ("xs_perm", lambda: permute(z(T, D // 32), xs_perm=z(M, D // 32))),
    # words over more rows: another stride
    ("xs", lambda: fc1(xs=z(D // 128, 2 * M, 4))),
    ("xs", lambda: fc1(xs=z(D // 128, 2 * M, 4), rows=2 * M, m_cap=M)),
    ("w1s", lambda: fc1(w1s=z(D // 128, 2 * E * F, 4))),
    ("xs_perm", lambda: permute(z(T, D // 32), xs_perm=z(D // 128, 2 * M, 4))),
    ("scales", lambda: rpg.moe_dequantize_mxfp4(z(M, D // 2), z(D // 128, 2 * M, 4), layout=KSTEPS)),
    ("scales", lambda: rpg.moe_quantize_mxfp4(z(M, D, dt=BF), scales=z(D // 128, 2 * M, 4), layout=KSTEPS)),
    # words over other k-steps
    ("w2s", lambda: fc2(w2s=z(D // 128, E * F, 4))),
    # words where scale rows are read
    ("scales", lambda: rpg.moe_dequantize_mxfp4(z(M, D // 2), z(D // 128, M, 4))),
    ("scales", lambda: rpg.moe_dequantize_mxfp8(z(M, D), z(D // 128, M, 4))),
    ("scales", lambda: rpg.moe_quantize_mxfp4(z(M, D, dt=BF), scales=z(D // 128, M, 4))),
    ("xs", lambda: permute(z(D // 128, T, 4))),
    # scale rows of other widths
    ("scales", lambda: rpg.moe_dequantize_mxfp4(z(M, D // 2), z(M, D // 16))),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_scales_of_another_layout_are_refused(i):
    name, call = REFUSED[i]
    with pytest.raises(ValueError, match=rf"^{name}: shape"):
        call()


TAKEN = [
    lambda: fc1(),
    lambda: fc2(),
    lambda: masked(),
    lambda: permute(z(T, D // 32)),
    lambda: permute(z(T, D // 32), xs_perm=z(D // 128, M, 4)),
    # a flat buffer has no shape to tell a layout by; it may be larger
    lambda: fc1(xs=z(M * D // 32), w1s=z(E * F * D // 32 + 64)),
    lambda: rpg.moe_quantize_mxfp4(z(M, D, dt=BF), scales=z(M * D), layout=KSTEPS),
    lambda: rpg.moe_dequantize_mxfp4(z(M, D // 2), z(M * D), layout=KSTEPS),
    # the expert axis apart: the same bytes
    lambda: fc1(w1s=z(D // 128, E, F, 4)),
    # more scale rows than codes: the first ones are read
    lambda: rpg.moe_dequantize_mxfp4(z(M, D // 2), z(2 * M, D // 32)),
    lambda: rpg.moe_quantize_mxfp4(z(2, M, D, dt=BF), scales=z(2, M, D // 32)),
    # of one row, or of one step of 128 values, both layouts are the same bytes
    lambda: rpg.moe_dequantize_mxfp4(z(1, D // 2), z(1, D // 32), layout=KSTEPS),
    lambda: rpg.moe_dequantize_mxfp4(z(1, D // 2), z(D // 128, 1, 4)),
    lambda: rpg.moe_dequantize_mxfp4(z(M, 64), z(M, 4), layout=KSTEPS),
    lambda: rpg.moe_dequantize_mxfp4(z(M, 64), z(1, M, 4)),
]


@pytest.mark.parametrize("i", range(len(TAKEN)))
def test_scales_of_the_layout_are_taken(i):
    with pytest.raises(ValueError, match="must live on the GPU"):
        TAKEN[i]()
