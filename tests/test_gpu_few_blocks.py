"""GPU tests of the few-token layer on 4-bit blocks whose scales lie at the ends of E8M0: 255 is NaN and
reaches what reads it and nothing else; the smallest ones hold their values."""
import pytest
import torch

import routing_permute_grouped_amd as rpg
from tests.test_gpu_few import BF16, F32, Layer, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 20])
def test_a_nan_block_stays_with_its_expert_and_its_column(T):
    """Experts 0 to 3; a block of expert 1's w1 is NaN, and one of row 40 of expert 2's w2."""
    lay = Layer(91, 4, 256, 256, 0, "mx4")
    x = lay.x(92, T)
    idx = torch.stack([torch.arange(T) % 4, (torch.arange(T) + 1) % 4], 1).to(torch.int32).cuda()
    w = torch.full((T, 2), 0.5, device="cuda")
    clean = lay.run(x, 2, topk_idx=idx, topk_w=w)["out"]
    lay.mw.w1s[1, 1 * 256 + 7, 2] = 255     # words [D/128, E*F, 4]
    lay.mw.w2s[0, 2 * 256 + 40, 1] = 255    # words [F/128, E*D, 4]
    out = lay.run(x, 2, topk_idx=idx, topk_w=w)["out"]
    one, two = (idx == 1).any(1), (idx == 2).any(1)
    assert bool(torch.isnan(out[one]).all())
    assert bool(torch.isnan(out[two][:, 40]).all())
    keep = [c for c in range(256) if c != 40]
    assert torch.equal(out[~one][:, keep], clean[~one][:, keep])
    assert torch.equal(out[~one & ~two], clean[~one & ~two])


@pytest.mark.parametrize("byte", [0, 1, 64, 190])
def test_scales_far_out(byte):
    """Every block of w2 at one scale: its values are exact in float32 and the bound is relative."""
    lay = Layer(93, 3, 128, 128, 0, "mx4")
    lay.mw.w2s.fill_(byte)
    lay.w2 = rpg.moe_dequantize_mxfp4(lay.mw.w2q, lay.mw.w2s, layout=rpg.MOE_MX_KSTEPS, dtype=F32)
    big = lay.x(94, 5)
    # rows large enough that the smallest scale's results are normal numbers of bf16
    x = (big.float() * (64.0 if byte < 2 else 1.0)).to(BF16)
    lay.check(x, lay.run(x, 2, wg=lay.wg))
