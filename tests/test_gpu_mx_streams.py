"""GPU tests of the block-scaled calls on a stream of their own (``stream``): what the call
allocates belongs to that stream. Memory of the current stream's pool may belong to a tensor
that was freed while work queued there still uses it, and nothing orders the call behind it."""
import numpy as np
import pytest
import torch

import routing_permute_grouped_amd as rpg
from tests import _parity as P
from tests.test_gpu_mxfp4 import bf16

pytestmark = pytest.mark.gpu

E, D, F, MT, T, K = 4, 256, 384, 64, 200, 2
KSTEPS = rpg.MOE_MX_KSTEPS


def make_call(name):
    """call(**kw) -> the call's own tensors, by name."""
    rng = np.random.default_rng(41)
    dev = lambda a: P.to_dev(bf16(a))  # noqa: E731
    x = dev(rng.standard_normal((T, D)))
    idx = P.to_dev(np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32))
    w1, w3 = (dev(rng.standard_normal((E, F, D)) / 16) for _ in range(2))
    w2 = dev(rng.standard_normal((E, D, F)) / 16)
    p = rpg.moe_permute(x, idx, E, MT)
    seg, m_cap, cnt = (p["offsets"], p["tile_expert"]), p["m_cap"], p["counts"]
    w1q, w3q, w2q = (rpg.moe_quantize_mxfp4(w, layout=KSTEPS) for w in (w1, w3, w2))
    xq, xs = rpg.moe_quantize_mxfp4(x)
    p4 = rpg.moe_permute_mxfp4(xq, xs, idx, E, MT)
    hq = rpg.moe_quantize_mxfp4(dev(rng.standard_normal((m_cap, F))), layout=KSTEPS)
    x8 = rpg.moe_quantize_mxfp8(x)
    masked = rpg.moe_permute_masked(x, idx, E, 128)
    ckpt = rpg.moe_grouped_fc1_swiglu_ckpt8(p["x_perm"], *seg, w1, w3, MT, counts=cnt)
    tw = torch.rand((T, K), device="cuda")
    used = int(p["offsets"][-1])

    def rows(names, out):   # rows behind the last segment are nobody's
        return {n: t[:used] if t.shape[0] == m_cap else t for n, t in zip(names, out)}

    def permute4(**kw):
        o = rpg.moe_permute_mxfp4(xq, xs, idx, E, MT, **kw)
        return {n: o[n] for n in ("counts", "offsets", "dst_row", "src_row", "tile_expert", "dev_err")} | {
            "xq_perm": o["xq_perm"][:used], "xs_perm": o["xs_perm"][:, :used]}

    def slabs(**kw):
        h, y = rpg.moe_grouped_swiglu_masked_mxfp4(masked["x_masked"], masked["counts"], *w1q, *w3q, *w2q, 128, **kw)
        n = int(masked["counts"][0])
        return {"h": h[:n], "y": y[:n]}

    return {
        "quantize": lambda **kw: dict(zip("qs", rpg.moe_quantize_mxfp4(x, layout=KSTEPS, **kw))),
        "values4": lambda **kw: {"out": rpg.moe_dequantize_mxfp4(xq, xs, **kw)},
        "values8": lambda **kw: {"out": rpg.moe_dequantize_mxfp8(*x8, **kw)},
        "permute": permute4,
        "fc1": lambda **kw: rows(["h"], [rpg.moe_grouped_fc1_swiglu_mxfp4(
            p4["xq_perm"], p4["xs_perm"], *seg, *w1q, *w3q, MT, counts=cnt, **kw)]),
        "fc2": lambda **kw: rows(["y"], [rpg.moe_grouped_fc2_mxfp4(*hq, *seg, *w2q, MT, counts=cnt, **kw)]),
        "masked": slabs,
        "save": lambda **kw: rows(["h", "codes", "scales"], rpg.moe_grouped_fc1_swiglu_ckpt8(
            p["x_perm"], *seg, w1, w3, MT, counts=cnt, **kw)),
        "use": lambda **kw: rows(["dab", "hw", "dtopk_w"], rpg.moe_grouped_dgrad_swiglu_ckpt8(
            p["x_perm"], *seg, w2, ckpt[1], ckpt[2], MT, src_row=p["src_row"], dst_row=p["dst_row"],
            topk_w=tw, counts=cnt, **kw)),
    }[name]


CALLS = ["quantize", "values4", "values8", "permute", "fc1", "fc2", "masked", "save", "use"]


def storages(out):
    return [(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in out.values()]


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_another_stream_takes_no_memory_of_this_one(name):
    P.log(f"[streams] {name}")
    call = make_call(name)
    ref = {n: t.clone() for n, t in call().items()}
    sizes = [n for _, n in storages(call())]
    if name == "use":
        sizes.append(rpg.moe_ckpt8_scratch_bytes(F, rpg.moe_capacity(T, K, E, MT)))
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        # blocks of this stream's, free again while their fills still wait behind the delay
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF) for n in sizes for _ in range(3)]
        ranges = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
        del blocks
        got = call(stream=stream)
        for at, n in storages(got):
            assert not any(lo < at + n and at < hi for lo, hi in ranges)
        torch.cuda.synchronize()
        for n, t in ref.items():
            assert torch.equal(got[n].view(torch.uint8), t.view(torch.uint8)), n


@pytest.mark.parametrize("name", CALLS)
def test_results_on_another_stream_outlive_their_use_here(name):
    call = make_call(name)
    side = torch.cuda.Stream()
    first = call(stream=side)
    side.synchronize()
    torch.cuda._sleep(50_000_000)
    copies = {n: t.clone() for n, t in first.items()}   # wait behind the delay
    held = [at for at, _ in storages(first)]
    del first
    second = call(stream=side)
    assert not set(held) & {at for at, _ in storages(second)}
    torch.cuda.synchronize()
    for n, t in second.items():
        assert torch.equal(copies[n].view(torch.uint8), t.view(torch.uint8)), n


def test_the_default_stream_by_its_handle():
    call = make_call("use")
    ref = call()
    torch.cuda.synchronize()
    got = call(stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    for n, t in ref.items():
        assert torch.equal(got[n].view(torch.uint8), t.view(torch.uint8)), n


@pytest.mark.parametrize("name", ["quantize", "fc1", "use"])
def test_a_call_on_a_capturing_stream(name):
    call = make_call(name)
    ref = {n: t.clone() for n, t in call().items()}
    side = torch.cuda.Stream()
    call(stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call(stream=side)
    for _ in range(3):
        for t in got.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        for n, t in ref.items():
            assert torch.equal(got[n].contiguous().view(torch.uint8), t.view(torch.uint8)), n
