"""The bound that the GPU test of the router's weight gradient past 2^31 elements holds it to, on the CPU:
a gradient of zeros and one that lacks a single token both lie outside it."""
import pytest
import torch

from tests import _block_ref as R


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("E,k", [(4, 2), (70, 4)])
def test_a_missing_token_is_outside_the_bound_of_dwg(E, k, seed):
    T, D = 4, 4096
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    logits, x, wg = rn(T, E), rn(T, D).bfloat16(), (rn(E, D) / D ** 0.5).bfloat16()
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    want = R.route_backward(rn(T, k), idx, logits, x, wg)
    ref, tol = want["dwg"]
    R.within(ref, ref, tol)
    with pytest.raises(AssertionError):
        R.within(torch.zeros_like(ref), ref, tol)
    dl = want["dlogits"][0]
    for t in range(T):
        part = ref - dl[t][:, None] * x[t].double()
        with pytest.raises(AssertionError):
            R.within(part, ref, tol)
        # and in nearly every element, so that a wrong piece of a row shows too
        assert float(((part - ref).abs() > tol).double().mean()) > 0.9
