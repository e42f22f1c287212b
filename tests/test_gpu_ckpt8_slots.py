"""GPU test of the checkpoint's backward with more slots than a launch has threads for at eight a
slot: the entry point takes T * k up to 2^30, and most slots may have no row."""
import torch

import pytest

import routing_permute_grouped_amd as rpg

pytestmark = pytest.mark.gpu


def test_two_to_the_29_slots_and_more():
    T, k, D, F, mt, rows = (1 << 24) + 1, 32, 64, 128, 16, 48
    i32 = dict(dtype=torch.int32, device="cuda")
    b = dict(dtype=torch.bfloat16, device="cuda")
    torch.manual_seed(0)
    n = T * k
    # the rows belong to the first and the last slots and to some on both sides of 2^29
    slots = torch.cat([torch.arange(16), torch.arange((1 << 29) - 8, (1 << 29) + 8), torch.arange(n - 16, n)])
    src = slots.to(**i32)
    dst = torch.full((n,), -1, **i32)
    dst[slots.cuda()] = torch.arange(rows, **i32)
    tw = torch.full((n,), 0.5, device="cuda")
    x, w2 = torch.randn((rows, D), **b), torch.randn((1, D, F), **b) / 8
    w1, w3 = torch.randn((1, F, D), **b) / 8, torch.randn((1, F, D), **b) / 8
    offs, te = torch.tensor([0, rows], **i32), torch.zeros(rows // mt, **i32)
    _, q, s = rpg.moe_grouped_fc1_swiglu_ckpt8(x, offs, te, w1, w3, mt)
    dtw = torch.full((T, k), float("nan"), device="cuda")
    _, _, got = rpg.moe_grouped_dgrad_swiglu_ckpt8(x, offs, te, w2, q, s, mt, src_row=src, dst_row=dst.view(T, k),
                                                   topk_w=tw.view(T, k), dtopk_w=dtw)
    # the same rows with a slot each
    few = torch.arange(rows, **i32)
    _, _, ref = rpg.moe_grouped_dgrad_swiglu_ckpt8(x, offs, te, w2, q, s, mt, src_row=few, dst_row=few.view(rows, 1),
                                                   topk_w=torch.full((rows, 1), 0.5, device="cuda"))
    torch.cuda.synchronize()
    flat = got.view(-1)
    assert torch.equal(flat[slots.cuda()], ref.view(-1)) and ref.abs().max() > 0
    flat[slots.cuda()] = 0.0
    assert not flat.any()
