"""Host-side checks of the calls in include/moe_mx.h: every declared symbol is exported and
bound, and bad arguments are rejected before the GPU is touched. No call here reaches a
kernel launch."""
import os
import re

import pytest
import torch

import routing_permute_grouped_amd as rpg

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "moe_mx.h")
MOE_OK, MOE_EINVAL, MOE_ESHAPE, MOE_ECAPACITY, MOE_EWORKSPACE = 0, 1, 2, 3, 4
FAKE = 0x10000   # aligned, non-null; never dereferenced because every call is rejected
lib = rpg.lib


def test_header_symbols_are_bound_and_exported():
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^(?![\s/*#])[^\n(]*?\b(moe_[a-z_0-9]+)\(", text, re.M)))
    assert names == sorted(n for n, _, _ in rpg.MX_SIGNATURES)
    assert all(hasattr(lib, n) and hasattr(rpg, n) for n in names)


def quantize(dt=1, x=FAKE, R=4, C=128, q=FAKE, s=FAKE, layout=0):
    return lib.moe_quantize_mxfp4(dt, x, R, C, q, s, layout, None)


def dequantize4(dt=1, x=FAKE, R=4, C=128, q=FAKE, s=FAKE, layout=0):
    return lib.moe_dequantize_mxfp4(dt, q, s, R, C, layout, x, None)


def dequantize8(dt=1, x=FAKE, R=4, C=128, q=FAKE, s=FAKE, layout=0):
    return lib.moe_dequantize_mxfp8(dt, q, s, R, C, layout, x, None)


@pytest.mark.parametrize("call", [quantize, dequantize4, dequantize8])
@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), MOE_EINVAL), (dict(x=None), MOE_EINVAL), (dict(x=FAKE + 8), MOE_EINVAL),
    (dict(q=FAKE + 4), MOE_EINVAL), (dict(s=None), MOE_EINVAL), (dict(layout=2), MOE_EINVAL),
    (dict(s=FAKE + 1, layout=1), MOE_EINVAL), (dict(R=0), MOE_ESHAPE), (dict(C=48), MOE_ESHAPE),
    (dict(C=0), MOE_ESHAPE), (dict(C=96, layout=1), MOE_ESHAPE), (dict(C=65568), MOE_ESHAPE),
    (dict(R=(1 << 31) + 1), MOE_ESHAPE),
])
def test_row_calls_validate(call, kw, code):
    assert call(**kw) == code


def permute(xq=FAKE, T=64, D=128, E=8, k=2, mt=16, m_cap=None, ws_bytes=1 << 20, err=FAKE):
    if m_cap is None:
        m_cap = max(rpg.moe_capacity(T, k, E, mt), mt)
    return lib.moe_permute_mxfp4(xq, FAKE, FAKE, T, D, E, k, mt, m_cap, FAKE, FAKE, FAKE, FAKE,
                                 FAKE, FAKE, FAKE, FAKE, ws_bytes, err, None)


@pytest.mark.parametrize("kw,code", [
    (dict(xq=FAKE + 8), MOE_EINVAL), (dict(err=None), MOE_EINVAL), (dict(D=192), MOE_ESHAPE),
    (dict(T=0), MOE_ESHAPE), (dict(k=9), MOE_ESHAPE), (dict(mt=48), MOE_ESHAPE),
    (dict(m_cap=16), MOE_ECAPACITY), (dict(ws_bytes=3), MOE_EWORKSPACE),
])
def test_permute_validation(kw, code):
    assert permute(**kw) == code


def fc1(xq=FAKE, xs=FAKE, offs=FAKE, counts=None, te=FAKE, E=8, D=256, F=320, mt=16, m_cap=1024,
        w1q=FAKE, h=FAKE, ws=None, wsb=0):
    return lib.moe_grouped_fc1_swiglu_mxfp4(xq, xs, offs, counts, te, E, D, F, mt, m_cap, w1q,
                                            FAKE, FAKE, FAKE, h, ws, wsb, None)


def fc2(xq=FAKE, xs=FAKE, offs=FAKE, counts=None, te=FAKE, E=8, D=256, F=320, mt=16, m_cap=1024,
        w1q=FAKE, h=FAKE, ws=None, wsb=0):   # D and F change places
    return lib.moe_grouped_fc2_mxfp4(xq, xs, offs, counts, te, E, F, D, mt, m_cap, w1q, FAKE, h,
                                     ws, wsb, None)


@pytest.mark.parametrize("call", [fc1, fc2])
@pytest.mark.parametrize("kw,code", [
    (dict(xq=None), MOE_EINVAL), (dict(xs=FAKE + 8), MOE_EINVAL), (dict(offs=None), MOE_EINVAL),
    (dict(counts=FAKE + 2), MOE_EINVAL), (dict(te=None), MOE_EINVAL),
    (dict(w1q=FAKE + 8), MOE_EINVAL), (dict(h=None), MOE_EINVAL),
    (dict(ws=FAKE + 8, wsb=1 << 20), MOE_EINVAL), (dict(E=0), MOE_ESHAPE),
    (dict(E=1025), MOE_ESHAPE), (dict(D=192), MOE_ESHAPE), (dict(F=100), MOE_ESHAPE),
    (dict(D=65536, F=32768), MOE_ESHAPE), (dict(mt=8), MOE_ESHAPE), (dict(m_cap=0), MOE_ECAPACITY),
    (dict(m_cap=1032), MOE_ECAPACITY), (dict(m_cap=1 << 31), MOE_ECAPACITY),
])
def test_products_validate(call, kw, code):
    assert call(**kw) == code


def masked(x=FAKE, counts=FAKE, E=8, D=256, F=384, cap=16, w=FAKE, ws=FAKE, y=FAKE):
    return lib.moe_grouped_swiglu_masked_mxfp4(x, counts, E, D, F, cap, w, ws, FAKE, FAKE, FAKE,
                                               FAKE, FAKE, y, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=FAKE + 2), MOE_EINVAL), (dict(counts=None), MOE_EINVAL), (dict(w=None), MOE_EINVAL),
    (dict(ws=FAKE + 1), MOE_EINVAL), (dict(y=None), MOE_EINVAL), (dict(D=192), MOE_ESHAPE),
    (dict(F=448), MOE_ESHAPE), (dict(E=2000), MOE_ESHAPE), (dict(D=65536, F=32768), MOE_ESHAPE),
    (dict(cap=0), MOE_ECAPACITY), (dict(cap=24), MOE_ECAPACITY), (dict(cap=65552), MOE_ECAPACITY),
])
def test_masked_validation(kw, code):
    assert masked(**kw) == code


def save(x=FAKE, offs=FAKE, E=8, D=256, F=320, mt=16, m_cap=1024, w=FAKE, h=FAKE, q=FAKE, s=FAKE,
         ws=None, wsb=0):
    return lib.moe_grouped_fc1_swiglu_ckpt8(x, offs, None, FAKE, E, D, F, mt, m_cap, w, FAKE, h, q,
                                            s, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), MOE_EINVAL), (dict(w=FAKE + 4), MOE_EINVAL), (dict(h=None), MOE_EINVAL),
    (dict(q=FAKE + 8), MOE_EINVAL), (dict(s=None), MOE_EINVAL), (dict(s=FAKE + 2), MOE_EINVAL),
    (dict(offs=FAKE + 1), MOE_EINVAL),
    (dict(ws=FAKE + 8, wsb=1), MOE_EINVAL), (dict(D=100), MOE_ESHAPE), (dict(F=96), MOE_ESHAPE),
    (dict(E=0), MOE_ESHAPE), (dict(m_cap=1000), MOE_ECAPACITY),
])
def test_save_validation(kw, code):
    assert save(**kw) == code


def use(d=FAKE, offs=FAKE, E=8, D=256, F=320, mt=16, m_cap=1024, w2=FAKE, q=FAKE, s=FAKE, src=FAKE,
        dst=FAKE, tw=FAKE, T=64, k=2, dab=FAKE, hw=FAKE, dtw=FAKE, scr=FAKE, scrb=1 << 20):
    return lib.moe_grouped_dgrad_swiglu_ckpt8(d, offs, None, FAKE, E, D, F, mt, m_cap, w2, q, s,
                                              src, dst, tw, T, k, dab, hw, dtw, scr, scrb, None, 0,
                                              None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=None), MOE_EINVAL), (dict(q=FAKE + 4), MOE_EINVAL), (dict(s=None), MOE_EINVAL),
    (dict(hw=None), MOE_EINVAL), (dict(dab=FAKE + 8), MOE_EINVAL), (dict(src=None), MOE_EINVAL),
    (dict(scr=None), MOE_EINVAL), (dict(dst=None), MOE_EINVAL), (dict(tw=None), MOE_EINVAL),
    (dict(F=100), MOE_ESHAPE), (dict(T=0), MOE_ESHAPE), (dict(k=33), MOE_ESHAPE),
    (dict(m_cap=1000), MOE_ECAPACITY), (dict(scrb=1024 * 4 * 5 - 1), MOE_EWORKSPACE),
])
def test_use_validation(kw, code):
    assert use(**kw) == code


def test_scratch_bytes():
    assert rpg.moe_ckpt8_scratch_bytes(320, 1024) == 1024 * 4 * 5
    assert rpg.moe_ckpt8_scratch_bytes(100, 1024) == 0
    assert rpg.moe_ckpt8_scratch_bytes(320, 0) == 0


# The binding's own refusals: types and sizes that the C ABI cannot see. Tensors are on the
# CPU, and the first check that fails names its argument before any pointer is taken.
def z(*shape, dt=torch.uint8):
    return torch.zeros(shape, dtype=dt)


BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32


def test_binding_refuses_wrong_types_and_sizes():
    E, D, F, M, mt = 2, 256, 128, 64, 16
    offs, te, cnt = z(E + 1, dt=I32), z(M // mt, dt=I32), z(E, dt=I32)
    w1q, w1s = z(E, F, D // 2), z(D // 128, E * F, 4)
    w2q, w2s = z(E, D, F // 2), z(F // 128, E * D, 4)
    xq, xs = z(M, D // 2), z(D // 128, M, 4)
    bad = [
        (TypeError, "x", lambda: rpg.moe_quantize_mxfp4(z(4, 64, dt=torch.float16))),
        (ValueError, "x", lambda: rpg.moe_quantize_mxfp4(z(0, 64, dt=BF))),
        (ValueError, "scales", lambda: rpg.moe_quantize_mxfp4(z(4, 64, dt=BF), scales=z(4, 1))),
        (TypeError, "q", lambda: rpg.moe_dequantize_mxfp4(z(4, 64, dt=I32), z(4, 4))),
        (ValueError, "scales", lambda: rpg.moe_dequantize_mxfp8(z(4, 64), z(4, 1))),
        (TypeError, "dtype", lambda: rpg.moe_dequantize_mxfp8(z(4, 64), z(4, 2), dtype=torch.float16)),
        (ValueError, "out", lambda: rpg.moe_dequantize_mxfp4(z(4, 64), z(4, 4), out=z(4, 64, dt=BF))),
        (ValueError, "xs", lambda: rpg.moe_permute_mxfp4(z(8, 64), z(8, 2), z(8, 2, dt=I32), 4, 16)),
        (TypeError, "topk_idx", lambda: rpg.moe_permute_mxfp4(z(8, 64), z(8, 4), z(8, 2, dt=torch.int64), 4, 16)),
        (ValueError, "capacity", lambda: rpg.moe_permute_mxfp4(z(8, 64), z(8, 4), z(8, 2, dt=I32), 4, 17)),
        (ValueError, "w3q", lambda: rpg.moe_grouped_fc1_swiglu_mxfp4(xq, xs, offs, te, w1q, w1s, z(E, F, D), w1s, mt)),
        (ValueError, "w1s", lambda: rpg.moe_grouped_fc1_swiglu_mxfp4(xq, xs, offs, te, w1q, z(1), w1q, w1s, mt)),
        (ValueError, "xs", lambda: rpg.moe_grouped_fc1_swiglu_mxfp4(xq, z(9), offs, te, w1q, w1s, w1q, w1s, mt)),
        (TypeError, "h", lambda: rpg.moe_grouped_fc1_swiglu_mxfp4(xq, xs, offs, te, w1q, w1s, w1q, w1s, mt, h=z(M, F, dt=F32))),
        (ValueError, "hq", lambda: rpg.moe_grouped_fc2_mxfp4(xq, xs, offs, te, w2q, w2s, mt)),
        (TypeError, "offsets", lambda: rpg.moe_grouped_fc2_mxfp4(z(M, F // 2), z(1, M, 4), z(E + 1, dt=torch.int64), te, w2q, w2s, mt)),
        (TypeError, "x_masked", lambda: rpg.moe_grouped_swiglu_masked_mxfp4(z(E * 16, D, dt=F32), cnt, w1q, w1s, w1q, w1s, w2q, w2s, 16)),
        (ValueError, "x_masked", lambda: rpg.moe_grouped_swiglu_masked_mxfp4(z(16, D, dt=BF), cnt, w1q, w1s, w1q, w1s, w2q, w2s, 16)),
        (ValueError, "w2q", lambda: rpg.moe_grouped_swiglu_masked_mxfp4(z(E * 16, D, dt=BF), cnt, w1q, w1s, w1q, w1s, w1q, w1s, 16)),
    ]
    w1, w2 = z(E, F, D, dt=BF), z(E, D, F, dt=BF)
    codes, scales = z(M, 2 * F), z(M, F // 16)
    x = z(M, D, dt=BF)
    tw, dst, src = z(8, 2, dt=F32), z(8, 2, dt=I32), z(M, dt=I32)
    sv, us = rpg.moe_grouped_fc1_swiglu_ckpt8, rpg.moe_grouped_dgrad_swiglu_ckpt8
    bad += [
        (TypeError, "x_perm", lambda: sv(z(M, D, dt=F32), offs, te, w1, w1, mt)),
        (TypeError, "w1", lambda: sv(x, offs, te, w1.float(), w1, mt)),
        (ValueError, "ab_scales", lambda: sv(x, offs, te, w1, w1, mt, ab_scales=z(M, 1))),
        (ValueError, "rows_used", lambda: sv(x, offs, te, w1, w1, mt, rows_used=M + 1)),
        (ValueError, "ab_codes", lambda: us(x, offs, te, w2, z(M, F), scales, mt)),
        (ValueError, "src_row", lambda: us(x, offs, te, w2, codes, scales, mt, topk_w=tw)),
        (ValueError, "dst_row", lambda: us(x, offs, te, w2, codes, scales, mt, topk_w=tw, src_row=src, dst_row=z(8, 3, dt=I32))),
        (TypeError, "topk_w", lambda: us(x, offs, te, w2, codes, scales, mt, topk_w=tw.double(), src_row=src, dst_row=dst)),
        (ValueError, "scratch", lambda: us(x, offs, te, w2, codes, scales, mt, topk_w=tw, src_row=src, dst_row=dst, scratch=z(8))),
        (ValueError, "dtopk_w", lambda: us(x, offs, te, w2, codes, scales, mt, dtopk_w=tw)),
        # everything fits, but the tensors are not on a GPU
        (ValueError, "GPU", lambda: us(x, offs, te, w2, codes, scales, mt)),
        (ValueError, "GPU", lambda: sv(x, offs, te, w1, w1, mt)),
        (ValueError, "GPU", lambda: rpg.moe_quantize_mxfp4(z(4, 64, dt=BF))),
    ]
    for kind, word, call in bad:
        with pytest.raises(kind, match=word):
            call()


def test_layer_refuses_an_unknown_checkpoint():
    with pytest.raises(ValueError, match="save_for_backward"):
        rpg.moe_layer(z(4, 64, dt=BF), z(2, 64, 64, dt=BF), z(2, 64, 64, dt=BF),
                      z(2, 64, 64, dt=BF), 1, 16, save_for_backward="fp4")
