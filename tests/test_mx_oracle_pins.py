"""The block-scaled oracle against things other than itself: torch's e4m3 conversion, plain
searches, finite differences, autograd in float64."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import moe_oracle as orc
from oracle import mx_oracle as mx


def test_mx4_codes_are_the_nearest_by_plain_search():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 64)) * 10.0 ** rng.uniform(-6, 6, (40, 1))
    x[0] = 0.0
    x[1, :32] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4) * np.tile([1, -1], 16)
    q, s = mx.mx4_quantize(x)
    v = mx.mx4_values(q, s)
    grid = sorted({c * t for c in mx.E2M1 for t in (1, -1)})
    for r in range(40):
        for b in range(2):
            blk = x[r, 32 * b:32 * b + 32]
            amax = np.abs(blk).max()
            X = -127
            while amax > 6.0 * 2.0 ** X:
                X += 1
            assert s[r, b] == X + 127
            for i, t in enumerate(blk):
                best = min(abs(t / 2.0 ** X - g) for g in grid)
                assert abs(t / 2.0 ** X - v[r, 32 * b + i] / 2.0 ** X) == best
    # ties: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    np.testing.assert_array_equal(np.abs(v[1, :32:4]), [0, 1, 1, 2, 2, 4, 4, 6])


def test_mx4_nibble_order_sign_and_special_blocks():
    x = np.zeros((1, 128))
    x[0, 0], x[0, 1], x[0, 2] = 6.0, -0.5, -0.0
    x[0, 40], x[0, 70], x[0, 100] = np.nan, np.inf, -2.0 ** -140
    q, s = mx.mx4_quantize(x)
    assert q[0, 0] == 7 | (9 << 4) and q[0, 1] == 8
    assert list(s[0]) == [127, 255, 255, 0]
    assert not q[0, 16:48].any()
    v = mx.mx4_values(q, s)
    assert np.isnan(v[0, 32:96]).all() and np.isfinite(v[0, :32]).all()


def test_mx8_values_against_torch():
    codes = np.tile(np.arange(256, dtype=np.uint8), (3, 1))
    scales = np.repeat(np.array([[0], [127], [140]], dtype=np.uint8), 8, axis=1)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(mx.mx8_values(codes, scales), t * 2.0 ** (scales[:, :1] - 127.0))


def test_words_round_trip():
    s = np.arange(5 * 12, dtype=np.uint8).reshape(5, 12)
    w = mx.words_of(s)
    assert w.shape == (3, 5, 4) and w[1, 2, 3] == s[2, 7]
    np.testing.assert_array_equal(mx.rows_of(w), s)


def test_exact_inputs_make_the_4bit_layer_the_bf16_layer():
    # weights on the E2M1 grid, one power of two each; the product itself then matches the
    # plain SwiGLU of the same numbers
    rng = np.random.default_rng(3)
    w = rng.choice(mx.E2M1, size=(2, 64, 128)) * rng.choice([-0.25, 0.25], size=(2, 64, 128))
    w[..., ::32] = 1.5   # the block's maximum fixes the scale
    x = rng.choice(mx.E2M1, size=(9, 128))
    x[..., ::32] = 6.0
    q, s = mx.quantize_weights(w)
    np.testing.assert_array_equal(mx.mx4_values(q, s), w)
    np.testing.assert_array_equal(mx.mx4_values(*mx.mx4_quantize(x)), x)
    h = mx.fc1(x, w[0], w[1])[0]
    t = torch.from_numpy
    a, b = t(x) @ t(w[0]).T, t(x) @ t(w[1]).T
    np.testing.assert_allclose(h, (torch.nn.functional.silu(a) * b).numpy(), rtol=1e-12)


def test_ckpt8_rows_against_differences_and_autograd():
    rng = np.random.default_rng(4)
    n, D, F = 3, 5, 4
    dout, w2 = rng.standard_normal((n, D)), rng.standard_normal((D, F))
    a, b, w = rng.standard_normal((n, F)), rng.standard_normal((n, F)), rng.random(n)

    def loss(a, b, w, w2):   # <dout, weighted fc2 of silu(a) * b>
        return ((w[:, None] * ((orc.silu(a) * b) @ w2.T)) * dout).sum()

    da, db, hw, dw = mx.ckpt8_rows(dout, w2, a, b, w)
    dw2 = dout.T @ hw
    eps = 1e-6
    for args, grad in (((a, 0), da), ((b, 1), db), ((w, 2), dw), ((w2, 3), dw2)):
        v, pos = args
        for at in np.ndindex(v.shape):
            hi, lo = [a, b, w, w2], [a, b, w, w2]
            hi[pos], lo[pos] = v.copy(), v.copy()
            hi[pos][at] += eps
            lo[pos][at] -= eps
            # central difference: error O(eps^2) + rounding 1e-16 / eps
            assert abs((loss(*hi) - loss(*lo)) / (2 * eps) - grad[at]) < 1e-7
    ta, tb, tw = (torch.from_numpy(v).requires_grad_() for v in (a, b, w))
    L = (tw[:, None] * ((torch.nn.functional.silu(ta) * tb) @ torch.from_numpy(w2).T)
         * torch.from_numpy(dout)).sum()
    L.backward()
    for t, g in ((ta, da), (tb, db), (tw, dw)):
        np.testing.assert_allclose(t.grad.numpy(), g, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("shared", [0, 2])
def test_ckpt8_backward_is_near_the_bf16_checkpoints(shared):
    # the same gradients up to the checkpoint's rounding (half a step, 2^-4 relative, each
    # value on its own): averaged over rows and columns far below that
    cfg = W.shrink(W.preset("fine64_shared2_bf16"), T=48, D=128, F=64, E=4, k=2, n_shared=shared,
                   F_shared=64, m_tile=16)
    inp = W.generate(cfg, seed=1)
    dout = W.f32_to_bf16_bits(np.random.default_rng(5).standard_normal((48, 128)).astype(np.float32))
    r8 = mx.backward_ckpt8(inp, dout, cfg.k, cfg.m_tile)
    r16 = orc.backward(inp, dout, cfg.k, cfg.m_tile, "bf16")
    if shared:   # one expert with its intermediate dimensions side by side
        r16["dws1"] = np.concatenate(list(r16["dws1"]), axis=0)
        r16["dws2"] = np.concatenate(list(r16["dws2"]), axis=1)
    for n in ("dx", "dw1", "dw3", "dw2", "dtopk_w") + (("dws1", "dws2") if shared else ()):
        a = np.asarray(r8[n])
        assert np.linalg.norm(a - r16[n]) <= 2.0 ** -4 * np.linalg.norm(r16[n]), n
