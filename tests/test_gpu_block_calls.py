"""The norm's and the 4-bit products' calls from outside: their launches and labels, what they allocate, and a
captured block."""
import pytest
import torch

import moe_inputs as mi
import serving_router_gate_gb300 as moe
from serving_router_gate_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu

T = 11


def _layer(w4=64):
    cfg = mi.MoEConfig("calls", T=T, H=512, I=256, E=16, k=3, renorm=True, n_shared=1, I_shared=256, shared_gate=True)
    inp = mi.make_inputs(cfg)
    d = {n: (v.cuda().contiguous() if isinstance(v, torch.Tensor) else v) for n, v in inp.items()}
    W1s, W2s = mi.shared_concat(d["W1s"], d["W2s"])
    g = torch.Generator(device="cuda").manual_seed(5)
    w = (1.0 + 0.1 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
    layer = MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, cfg.renorm, 16, W1s=W1s, W2s=W2s, shared_gate_w=d["w_s"], w4=w4,
                     norm_w=w, **({} if w4 else dict(fp8=True, act8=True)))
    return layer, d["x"], torch.randn(T, 512, generator=g, device="cuda")


def test_launch_events_follow_the_block():
    layer, x, res = _layer()
    want_res = res.clone()
    want = layer.block(x, want_res).clone()
    mine = res.clone()
    n = moe.moe_get_launch_count()
    layer.block(x, mine)
    n = moe.moe_get_launch_count() - n
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(n + 1)]
    for e in evs:
        e.record()
    torch.cuda.synchronize()
    mine = res.clone()
    moe.moe_launch_events_arm(evs)
    try:
        out = layer.block(x, mine).clone()
        moe.moe_launch_events_mark()
        labels = moe.moe_launch_events_used()
    finally:
        moe.moe_launch_events_arm(None)
    torch.cuda.synchronize()
    assert len(labels) == n + 1 and labels[0] == "add_rmsnorm", labels
    assert labels[-4:] == ["w4_fc1", "w4_fc2", "w4_combine", "mark"], labels
    assert all(evs[i].elapsed_time(evs[i + 1]) > 0.0 for i in range(n))
    # without overlap between the kernels: the same results
    assert torch.equal(out, want) and torch.equal(mine, want_res)


@pytest.mark.parametrize("w4", [64, 0])
def test_calls_allocate_nothing_on_the_device(w4):
    layer, x, res = _layer(w4)
    q = torch.empty(64, 256, dtype=torch.uint8, device="cuda")
    s = torch.empty(64, 8, dtype=torch.bfloat16, device="cuda")
    w, y = torch.randn(64, 512, device="cuda").to(torch.bfloat16), torch.empty(T, 64, dtype=torch.bfloat16, device="cuda")

    def calls():
        layer.block(x, res)
        moe.moe_quantize_w4_rows(w, q, s)
        moe.moe_matvec_w4(x, q, s, y)
    calls()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        calls()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


@pytest.mark.parametrize("w4", [64, 0])
def test_a_captured_block_is_the_eager_one(w4):
    layer, x, res = _layer(w4)
    want_res = res.clone()
    want = layer.block(x, want_res).clone()
    mine = res.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.block(x, mine)
    for _ in range(2):
        mine.copy_(res)
        layer.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(mine, want_res)
