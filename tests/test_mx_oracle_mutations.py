"""Plant plausible mistakes in the block-scaled oracle (on the CPU) and check that a pin of
test_mx_oracle_pins.py catches each."""
import numpy as np
import pytest

from oracle import moe_oracle as orc
from oracle import mx_oracle as mx
from tests import test_mx_oracle_pins as pins

_quantize, _values, _rows8 = mx.mx4_quantize, mx.mx4_values, mx.ckpt8_rows


def _scale_from_the_exponent_alone(x):   # X = floor(log2 max) - 2: values past 6 * 2^X saturate
    q, s = _quantize(x)
    amax = np.abs(np.nan_to_num(orc.values64(x), nan=0.0, posinf=0.0)).reshape(len(x), -1, 32).max(2)
    X = np.where(amax > 0, np.maximum(np.frexp(amax)[1] - 3, -127), -127)
    return q, np.where(s == 255, 255, X + 127).astype(np.uint8)


def _scale_one_too_large(x):
    q, s = _quantize(x)
    return q, np.where((s > 0) & (s < 254), s + 1, s).astype(np.uint8)


def _ties_away_from_zero(x):
    v = orc.values64(x)
    return _quantize(np.nextafter(v, np.copysign(np.inf, v)) if np.isfinite(v).all() else v)


def _high_half_first(x):
    q, s = _quantize(x)
    return (q << 4) | (q >> 4), s


def _zeros_lose_their_sign(x):
    return _quantize(orc.values64(x) + 0.0)


def _special_blocks_keep_codes(x):
    q, s = _quantize(x)
    c = _quantize(np.nan_to_num(orc.values64(x), nan=1.0, posinf=6.0))[0]
    return np.where(np.repeat(s == 255, 16, axis=1), c, q), s


def _values_without_sign(q, s):
    return np.abs(_values(q, s))


def _words_of_neighbouring_rows(s):
    return np.ascontiguousarray(s.reshape(s.shape[0], 4, -1).transpose(2, 0, 1))


def _wgrad_rows_unweighted(dout, w2e, a, b, w):
    da, db, _, dw = _rows8(dout, w2e, a, b, w)
    return da, db, orc.silu(a) * b, dw


def _weight_gradient_weighted(dout, w2e, a, b, w):
    da, db, hw, dw = _rows8(dout, w2e, a, b, w)
    return da, db, hw, dw * np.asarray(w)


def _gradients_unweighted(dout, w2e, a, b, w):
    _, _, hw, dw = _rows8(dout, w2e, a, b, w)
    da, db, _, _ = _rows8(dout, w2e, a, b, np.ones_like(w))
    return da, db, hw, dw


def _silu_grad_is_the_sigmoid(dout, w2e, a, b, w):
    u, w_ = dout @ w2e, np.asarray(w)[:, None]
    _, db, hw, dw = _rows8(dout, w2e, a, b, w)
    return w_ * u * b / (1.0 + np.exp(-a)), db, hw, dw


def _swapped(dout, w2e, a, b, w):
    da, db, hw, dw = _rows8(dout, w2e, a, b, w)
    return db, da, hw, dw


CASES = [
    ("mx4_quantize", _scale_from_the_exponent_alone, pins.test_mx4_codes_are_the_nearest_by_plain_search),
    ("mx4_quantize", _scale_one_too_large, pins.test_mx4_codes_are_the_nearest_by_plain_search),
    ("mx4_quantize", _ties_away_from_zero, pins.test_mx4_codes_are_the_nearest_by_plain_search),
    ("mx4_quantize", _high_half_first, pins.test_mx4_nibble_order_sign_and_special_blocks),
    ("mx4_quantize", _zeros_lose_their_sign, pins.test_mx4_nibble_order_sign_and_special_blocks),
    ("mx4_quantize", _special_blocks_keep_codes, pins.test_mx4_nibble_order_sign_and_special_blocks),
    ("mx4_values", _values_without_sign, pins.test_exact_inputs_make_the_4bit_layer_the_bf16_layer),
    ("words_of", _words_of_neighbouring_rows, pins.test_words_round_trip),
    ("ckpt8_rows", _wgrad_rows_unweighted, pins.test_ckpt8_rows_against_differences_and_autograd),
    ("ckpt8_rows", _weight_gradient_weighted, pins.test_ckpt8_rows_against_differences_and_autograd),
    ("ckpt8_rows", _gradients_unweighted, pins.test_ckpt8_rows_against_differences_and_autograd),
    ("ckpt8_rows", _silu_grad_is_the_sigmoid, pins.test_ckpt8_rows_against_differences_and_autograd),
    ("ckpt8_rows", _swapped, pins.test_ckpt8_rows_against_differences_and_autograd),
]


@pytest.mark.parametrize("name,mutant,pin", CASES, ids=[c[1].__name__.strip("_") for c in CASES])
def test_a_pin_catches(monkeypatch, name, mutant, pin):
    pin()
    monkeypatch.setattr(mx, name, mutant)
    with pytest.raises(AssertionError):
        pin()
