"""GPU tests of how exact the few-token layer is in float32. A sum of n products in a chain whose partial sums
grow as sqrt(i / n) is off by u sqrt(n / 6) of its size, u = 2^-24 (every add by u / sqrt(3) of its partial
sum, at random). The layer's sums over k are chains of 256 products and one of their sums (and of the at most
16 waves' and the slots'), so with N(K) = 256 + K / 256 + 64:
    a, b:  u sqrt(N(D) / 6)        h = silu(a) b: both of them, silu's slope below 1.1
    out:   u sqrt(N(k F + Fs) / 6) beside h's
Held to 1.5 times that, over all of out. One chain of D = 4544 products would be off by 2.2 times as much."""
import math

import pytest
import torch

from tests.test_gpu_few import Layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bound(k, D, F, Fs):
    n = lambda K: U * math.sqrt((256 + K / 256 + 64) / 6)  # noqa: E731
    return 1.5 * math.hypot(1.1 * math.sqrt(2) * n(D), n(k * F + Fs))


@pytest.mark.parametrize("T,k,E,D,F,Fs", [(8, 4, 32, 4544, 256, 256), (20, 1, 31, 1856, 1024, 1728), (15, 6, 69, 1344, 2624, 0), (14, 5, 44, 6976, 832, 128),
                                          (8, 4, 8, 1856, 8192, 0), (16, 2, 8, 4096, 4096, 0), (32, 2, 4, 4096, 2048, 0), (1, 1, 1, 16384, 64, 0), (1, 2, 4, 64, 16384, 0)])
def test_as_exact_as_short_chains(T, k, E, D, F, Fs):
    lay = Layer(41, E, D, F, Fs, "f32")
    x = lay.x(42, T)
    r = lay.run(x, k, wg=lay.wg, bias=lay.bias)
    idx, w = r["topk_idx"].long(), r["topk_w"].double()
    ref = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for e in range(E):
        tok, slot = (idx == e).nonzero(as_tuple=True)
        if tok.numel():
            ref.index_add_(0, tok, w[tok, slot][:, None] * lay.ffn(x[tok], lay.w1[e], lay.w3[e], lay.w2[e])[0])
    if Fs:
        ref += lay.ffn(x, lay.shared.w1[0], lay.shared.w3[0], lay.shared.w2[0])[0]
    err = float((r["out"].double() - ref).norm() / ref.norm())
    print(f"{err:.2e} of {bound(k, D, F, Fs):.2e}", flush=True)
    assert err <= bound(k, D, F, Fs)
    lay.check(x, r)
