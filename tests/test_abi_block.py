"""Host-side checks of the calls in include/moe_block.h: every declared symbol is exported and
bound, and bad arguments are rejected before the GPU is touched. No call here reaches a
kernel launch."""
import os
import re

import pytest
import torch

import routing_permute_grouped_amd as rpg

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "moe_block.h")
MOE_OK, MOE_EINVAL, MOE_ESHAPE, MOE_ECAPACITY, MOE_EWORKSPACE = 0, 1, 2, 3, 4
FAKE = 0x10000   # aligned, non-null; never dereferenced because every call is rejected
lib = rpg.lib


def test_header_symbols_are_bound_and_exported():
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^(?![\s/*#])[^\n(]*?\b(moe_[a-z_0-9]+)\(", text, re.M)))
    assert names == sorted(n for n, _, _ in rpg.BLOCK_SIGNATURES)
    assert all(hasattr(lib, n) and hasattr(rpg, n) for n in names)


def few(dt=1, x=FAKE, wg=FAKE, bias=FAKE, T=4, D=128, F=128, E=8, k=2, w1=FAKE, w2=FAKE, Fs=64, ws1=FAKE,
        ws2=FAKE, idx=FAKE, w=FAKE, out=FAKE, ws=FAKE, n=1 << 30):
    return lib.moe_layer_few(dt, x, wg, bias, T, D, F, E, k, 0, w1, FAKE, w2, Fs, ws1, FAKE, ws2, idx, w, out, ws, n, None)


def few4(dt=1, x=FAKE, wg=FAKE, bias=FAKE, T=4, D=128, F=128, E=8, k=2, w1=FAKE, w2=FAKE, Fs=64, ws1=FAKE,
         ws2=FAKE, idx=FAKE, w=FAKE, out=FAKE, ws=FAKE, n=1 << 30, s1=FAKE):
    return lib.moe_layer_few_mxfp4(x, wg, bias, T, D, F, E, k, 0, w1, s1, FAKE, FAKE, w2, FAKE, Fs, ws1, FAKE, ws2, idx, w, out,
                                   ws, n, None)


@pytest.mark.parametrize("call", [few, few4])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), MOE_EINVAL), (dict(x=FAKE + 8), MOE_EINVAL), (dict(wg=FAKE + 4), MOE_EINVAL), (dict(bias=FAKE + 2), MOE_EINVAL),
    (dict(w1=None), MOE_EINVAL), (dict(w2=FAKE + 8), MOE_EINVAL), (dict(ws1=None), MOE_EINVAL), (dict(ws2=FAKE + 2), MOE_EINVAL),
    (dict(idx=None), MOE_EINVAL), (dict(w=FAKE + 1), MOE_EINVAL), (dict(out=None), MOE_EINVAL), (dict(ws=None), MOE_EINVAL),
    (dict(ws=FAKE + 4), MOE_EINVAL), (dict(T=0), MOE_ESHAPE), (dict(T=33), MOE_ESHAPE), (dict(D=96), MOE_ESHAPE),
    (dict(F=0), MOE_ESHAPE), (dict(F=65600), MOE_ESHAPE), (dict(Fs=-64), MOE_ESHAPE), (dict(Fs=100), MOE_ESHAPE),
    (dict(E=0), MOE_ESHAPE), (dict(E=1025), MOE_ESHAPE), (dict(k=0), MOE_ESHAPE), (dict(k=9), MOE_ESHAPE),
    (dict(E=64, k=33), MOE_ESHAPE), (dict(n=4 * 2 * 128 * 2 + 4 * 64 * 2 - 1), MOE_EWORKSPACE),
])
def test_few_validates(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(D=192), MOE_ESHAPE), (dict(F=64), MOE_ESHAPE), (dict(s1=None), MOE_EINVAL), (dict(s1=FAKE + 2), MOE_EINVAL),
])
def test_few_4bit_validates(kw, code):
    assert few4(**kw) == code


def test_few_dtype():
    assert few(dt=2) == MOE_EINVAL


def test_few_workspace_bytes():
    n = rpg.moe_layer_few_workspace_bytes
    assert n(torch.bfloat16, 3, 2, 128, 64) == (3 * 2 * 128 + 3 * 64) * 2 + 3 * 1024 * 4   # h, hs, logits
    assert n(torch.float32, 3, 2, 128) == 3 * 2 * 128 * 4 + 3 * 1024 * 4
    assert n(torch.float32, 33, 2, 128) == n(torch.float32, 1, 2, 100) == n(torch.float32, 1, 33, 128) == 0


def cpu_layer(T=4, D=128, F=128, E=8, dt=torch.bfloat16):
    z = lambda *s: torch.zeros(*s, dtype=dt)  # noqa: E731
    return dict(x=z(T, D), w1=z(E, F, D), w3=z(E, F, D), w2=z(E, D, F), k=2, wg=z(E, D))


@pytest.mark.parametrize("change,exc,text", [
    (dict(x=torch.zeros(33, 128, dtype=torch.bfloat16)), ValueError, "33 tokens"),
    (dict(x=torch.zeros(0, 128, dtype=torch.bfloat16)), ValueError, "0 tokens"),
    (dict(x=torch.zeros(4, 64, dtype=torch.bfloat16)), ValueError, "x: shape"),
    (dict(x=torch.zeros(4, 128, dtype=torch.float16)), TypeError, "x: dtype"),
    (dict(w3=torch.zeros(8, 128, 64, dtype=torch.bfloat16)), ValueError, "w3: shape"),
    (dict(w2=torch.zeros(8, 128, 128)), TypeError, "w2: dtype"),
    (dict(wg=None), ValueError, "wg, or topk_idx"),
    (dict(wg=torch.zeros(7, 128, dtype=torch.bfloat16)), ValueError, "wg: shape"),
    (dict(bias=torch.zeros(8, dtype=torch.bfloat16)), TypeError, "bias: dtype"),
    (dict(topk_idx=torch.zeros(4, 2, dtype=torch.int32)), ValueError, "topk_w: missing"),
    (dict(topk_idx=torch.zeros(4, 2, dtype=torch.int64), topk_w=torch.zeros(4, 2)), TypeError, "topk_idx: dtype"),
    (dict(topk_idx=torch.zeros(4, 3, dtype=torch.int32), topk_w=torch.zeros(4, 2)), ValueError, "topk_idx: shape"),
    (dict(out=torch.zeros(4, 128)), TypeError, "out: dtype"),
    (dict(out=torch.zeros(5, 128, dtype=torch.bfloat16)), ValueError, "out: shape"),
    (dict(shared=rpg.SharedExperts(torch.zeros(2, 64, 128, dtype=torch.bfloat16), torch.zeros(2, 64, 128, dtype=torch.bfloat16),
                                   torch.zeros(2, 128, 64, dtype=torch.bfloat16))), ValueError, "shared.w1: shape"),
    (dict(), ValueError, "must live on the GPU"),
])
def test_few_python_checks(change, exc, text):
    kw = {**cpu_layer(), **change}
    with pytest.raises(exc, match=text):
        rpg.moe_layer_few(**kw)


def norm(dt=1, r=FAKE, gamma=FAKE, eps=1e-6, T=4, D=128, x=FAKE, rstd=FAKE):
    return lib.moe_norm(dt, r, gamma, eps, T, D, x, rstd, None)


def norm_bwd(dt=1, r=FAKE, gamma=FAKE, T=4, D=128, x=FAKE, rstd=FAKE, dresid=None, dgamma=FAKE, ws=FAKE, n=1 << 30):
    return lib.moe_norm_backward(dt, FAKE, r, gamma, rstd, dresid, T, D, x, dgamma, ws, n, None)


@pytest.mark.parametrize("call", [norm, norm_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), MOE_EINVAL), (dict(r=None), MOE_EINVAL), (dict(gamma=FAKE + 8), MOE_EINVAL), (dict(x=None), MOE_EINVAL),
    (dict(rstd=FAKE + 1), MOE_EINVAL), (dict(T=0), MOE_ESHAPE), (dict(D=96), MOE_ESHAPE), (dict(D=16448), MOE_ESHAPE),
])
def test_norm_validates(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("eps", [0.0, -1.0, float("nan"), float("inf")])
def test_norm_eps(eps):
    assert norm(eps=eps) == combine(eps=eps) == MOE_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(rstd=None), MOE_EINVAL), (dict(dresid=FAKE + 4), MOE_EINVAL), (dict(dgamma=FAKE + 2), MOE_EINVAL), (dict(ws=None), MOE_EINVAL),
    (dict(n=2 * 128 * 4 - 1), MOE_EWORKSPACE),
])
def test_norm_backward_validates(kw, code):
    assert norm_bwd(**kw) == code


def combine(dt=1, resid=FAKE, y=FAKE, dst=FAKE, w=FAKE, shared=None, gate=None, gp=FAKE, gn=FAKE, scale=1.0, eps=1e-6, T=4, D=128, k=2, m_cap=64,
            out=FAKE, xn=FAKE, u=None, rp=None, rn=None):
    return lib.moe_combine_norm(dt, resid, y, dst, w, shared, gate, gp, gn, scale, eps, T, D, k, m_cap, out, xn, u, rp, rn, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=5), MOE_EINVAL), (dict(resid=None), MOE_EINVAL), (dict(out=FAKE + 2), MOE_EINVAL), (dict(y=None), MOE_EINVAL),
    (dict(y=FAKE + 8), MOE_EINVAL), (dict(dst=None), MOE_EINVAL), (dict(w=FAKE + 2), MOE_EINVAL), (dict(shared=FAKE + 4), MOE_EINVAL),
    (dict(gate=FAKE + 1), MOE_EINVAL), (dict(gp=FAKE + 8), MOE_EINVAL), (dict(gn=FAKE + 8), MOE_EINVAL), (dict(xn=None), MOE_EINVAL),
    (dict(u=FAKE + 8), MOE_EINVAL), (dict(rp=FAKE + 1), MOE_EINVAL), (dict(rn=FAKE + 3), MOE_EINVAL), (dict(scale=float("inf")), MOE_EINVAL),
    (dict(T=0), MOE_ESHAPE), (dict(D=100), MOE_ESHAPE), (dict(D=32768), MOE_ESHAPE), (dict(k=0), MOE_ESHAPE), (dict(k=33), MOE_ESHAPE),
    (dict(m_cap=0), MOE_ECAPACITY), (dict(m_cap=1 << 31), MOE_ECAPACITY),
])
def test_combine_norm_validates(kw, code):
    assert combine(**kw) == code


@pytest.mark.parametrize("kw", [dict(gp=None, rp=FAKE), dict(gn=None, xn=None, rn=FAKE), dict(gn=None), dict(gp=None, gn=None, xn=None, rp=FAKE)])
def test_combine_norm_refuses_results_of_a_norm_it_does_not_take(kw):
    # sizes that are refused as well: a call that passes these checks launches nothing here
    assert combine(T=0, gp=None, gn=None, xn=None) == combine(T=0, rp=FAKE, rn=FAKE) == MOE_ESHAPE
    assert combine(T=0, **kw) == MOE_EINVAL


def combine_bwd(dt=1, dout=FAKE, dx=FAKE, u=FAKE, out=FAKE, gate=None, gp=FAKE, gn=FAKE, rp=FAKE, rn=FAKE, scale=1.0, T=4, D=128, du=FAKE, dr=FAKE,
                dgate=None, dgp=FAKE, dgn=FAKE, ws=FAKE, n=1 << 30):
    return lib.moe_combine_norm_backward(dt, dout, dx, u, out, gate, gp, gn, rp, rn, scale, T, D, du, dr, dgate, dgp, dgn, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), MOE_EINVAL), (dict(dout=None, dx=None), MOE_EINVAL), (dict(dout=FAKE + 8), MOE_EINVAL), (dict(out=None), MOE_EINVAL),
    (dict(gn=None), MOE_EINVAL), (dict(rn=None), MOE_EINVAL), (dict(rp=None), MOE_EINVAL), (dict(gp=None), MOE_EINVAL), (dict(u=None), MOE_EINVAL),
    (dict(gp=None, dgp=None, u=None, dgate=FAKE), MOE_EINVAL), (dict(dx=None), MOE_EINVAL), (dict(du=None), MOE_EINVAL),
    (dict(dr=FAKE + 8), MOE_EINVAL), (dict(dgn=FAKE + 2), MOE_EINVAL), (dict(ws=FAKE + 8), MOE_EINVAL), (dict(scale=float("nan")), MOE_EINVAL),
    (dict(T=-1), MOE_ESHAPE), (dict(D=0), MOE_ESHAPE), (dict(n=16), MOE_EWORKSPACE),
])
def test_combine_norm_backward_validates(kw, code):
    assert combine_bwd(**kw) == code


def route_bwd(dt=1, dw=FAKE, idx=FAKE, lg=FAKE, x=FAKE, wg=FAKE, dla=None, dxa=None, T=4, D=128, E=8, k=2, dl=FAKE, dx=FAKE, dwg=FAKE, db=FAKE,
              ws=FAKE, n=1 << 30):
    return lib.moe_route_backward(dt, dw, idx, lg, x, wg, dla, dxa, T, D, E, k, 0, dl, dx, dwg, db, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), MOE_EINVAL), (dict(dw=None), MOE_EINVAL), (dict(idx=FAKE + 2), MOE_EINVAL), (dict(lg=None), MOE_EINVAL), (dict(x=None), MOE_EINVAL),
    (dict(wg=None), MOE_EINVAL), (dict(x=FAKE + 8), MOE_EINVAL), (dict(dla=FAKE + 1), MOE_EINVAL), (dict(dxa=FAKE + 8), MOE_EINVAL),
    (dict(dl=None), MOE_EINVAL), (dict(dx=FAKE + 2), MOE_EINVAL), (dict(dwg=FAKE + 4), MOE_EINVAL), (dict(db=FAKE + 1), MOE_EINVAL),
    (dict(ws=None), MOE_EINVAL), (dict(T=0), MOE_ESHAPE), (dict(D=65600), MOE_ESHAPE), (dict(D=32), MOE_ESHAPE), (dict(E=0), MOE_ESHAPE),
    (dict(E=1025), MOE_ESHAPE), (dict(k=0), MOE_ESHAPE), (dict(k=9), MOE_ESHAPE), (dict(E=64, k=33), MOE_ESHAPE), (dict(n=64), MOE_EWORKSPACE),
])
def test_route_backward_validates(kw, code):
    assert route_bwd(**kw) == code


def test_workspace_bytes_of_bad_sizes():
    assert rpg.moe_norm_workspace_bytes(0, 128) == rpg.moe_norm_workspace_bytes(4, 100) == rpg.moe_norm_workspace_bytes(4, 32768) == 0
    n = rpg.moe_route_backward_workspace_bytes
    assert n(torch.bfloat16, 0, 128, 8) == n(torch.bfloat16, 4, 100, 8) == n(torch.float32, 4, 128, 1025) == 0
    assert rpg.moe_norm_workspace_bytes(4, 128) > 0 and n(torch.bfloat16, 4, 128, 8) > 0


BF = torch.bfloat16


def z(*s, dt=BF):
    return torch.zeros(*s, dtype=dt)


@pytest.mark.parametrize("call,exc,text", [
    (lambda: rpg.moe_norm(z(4, 128, dt=torch.float16), z(128)), TypeError, "r: dtype"),
    (lambda: rpg.moe_norm(z(4, 128), z(64)), ValueError, "gamma: shape"),
    (lambda: rpg.moe_norm(z(4, 128), z(128, dt=torch.float32)), TypeError, "gamma: dtype"),
    (lambda: rpg.moe_norm(z(128), z(128)), ValueError, "r: 1-d"),
    (lambda: rpg.moe_norm(z(4, 128), z(128)), ValueError, "must live on the GPU"),
    (lambda: rpg.moe_norm_backward(z(4, 64), z(4, 128), z(128), z(4, dt=torch.float32)), ValueError, "dx: shape"),
    (lambda: rpg.moe_norm_backward(z(4, 128), z(4, 128), z(128), z(5, dt=torch.float32)), ValueError, "rstd: shape"),
    (lambda: rpg.moe_norm_backward(z(4, 128), z(4, 128), z(128), z(4)), TypeError, "rstd: dtype"),
    (lambda: rpg.moe_combine_norm(z(4, 128)), ValueError, "y_perm with dst_row, or shared"),
    (lambda: rpg.moe_combine_norm(z(4, 128), z(9, 128)), ValueError, "dst_row: missing"),
    (lambda: rpg.moe_combine_norm(z(4, 128), z(9, 64), z(4, 2, dt=torch.int32)), ValueError, "y_perm: shape"),
    (lambda: rpg.moe_combine_norm(z(4, 128), z(9, 128), z(5, 2, dt=torch.int32)), ValueError, "dst_row: shape"),
    (lambda: rpg.moe_combine_norm(z(4, 128), z(9, 128), z(4, 2, dt=torch.int32), z(4, 3, dt=torch.float32)), ValueError, "topk_w: shape"),
    (lambda: rpg.moe_combine_norm(z(4, 128), shared=z(4, 128), topk_w=z(4, 3, dt=torch.float32)), ValueError, "without y_perm"),
    (lambda: rpg.moe_combine_norm(z(4, 128), shared=z(4, 128), gate=z(4)), TypeError, "gate: dtype"),
    (lambda: rpg.moe_combine_norm(z(4, 128), shared=z(4, 128), gamma_next=z(64)), ValueError, "gamma_next: shape"),
    (lambda: rpg.moe_combine_norm_backward(None, z(4, 128)), ValueError, "dout or dx_next"),
    (lambda: rpg.moe_combine_norm_backward(z(4, 128), None, gamma_post=z(128), rstd_post=z(4, dt=torch.float32)), ValueError, "u: needed"),
    (lambda: rpg.moe_combine_norm_backward(z(4, 128), z(4, 128), gamma_post=z(128)), ValueError, "needs rstd_post"),
    (lambda: rpg.moe_combine_norm_backward(z(4, 128), z(4, 128), dx_next=z(4, 128)), ValueError, "dx_next: needs"),
    (lambda: rpg.moe_combine_norm_backward(z(4, 128), z(3, 128)), ValueError, "u: shape"),
    (lambda: rpg.moe_route_backward(z(4, 2), z(4, 2, dt=torch.int32), z(4, 8, dt=torch.float32), z(4, 128), z(8, 128)), TypeError, "dtopk_w: dtype"),
    (lambda: rpg.moe_route_backward(z(4, 2, dt=torch.float32), z(4, 2, dt=torch.int64), z(4, 8, dt=torch.float32), z(4, 128), z(8, 128)), TypeError,
     "topk_idx: dtype"),
    (lambda: rpg.moe_route_backward(z(4, 2, dt=torch.float32), z(4, 2, dt=torch.int32), z(4, 9, dt=torch.float32), z(4, 128), z(8, 128)), ValueError,
     "logits: shape"),
    (lambda: rpg.moe_route_backward(z(4, 2, dt=torch.float32), z(4, 2, dt=torch.int32), z(4, 8, dt=torch.float32), z(4, 128), z(8, 64)), ValueError,
     "wg: shape"),
    (lambda: rpg.moe_block(z(4, 128), z(8, 128, 128), z(8, 128, 128), z(8, 128, 128), 2, 16, z(8, 128)), ValueError, "x or gamma_pre"),
    (lambda: rpg.moe_block_few(z(4, 128), (z(8, 128, 128),) * 3, 2, z(8, 128), x=z(4, 128), gamma_pre=z(128)), ValueError, "x or gamma_pre"),
])
def test_python_checks(call, exc, text):
    with pytest.raises(exc, match=text):
        call()
