"""Expert-parallel layers on 4-bit experts, the ranks one after the other on one GPU.

Tolerance (derived before the first run): the partials and the one-GPU output are rounded to bf16 once each (2^-8
relative); an h whose sum is added in another order may round to its neighbour, which moves a product by at most
2^-7 of its size, far less in the 2-norm: 2^-7 of the partials' and the output's 2-norms together."""
import pytest
import torch

import moe_inputs as mi
import serving_router_gate_gb300 as moe
from serving_router_gate_gb300.expert_parallel import EPMoELayer, PeerReduction
from serving_router_gate_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu


def _case(T=9, H=256, I=128, E=16, k=4, I_sh=1408):
    cfg = mi.MoEConfig("ep_w4", T=T, H=H, I=I, E=E, k=k, renorm=True, n_shared=1, I_shared=I_sh, shared_gate=True)
    inp = mi.make_inputs(cfg)
    d = {n: (v.cuda().contiguous() if isinstance(v, torch.Tensor) else v) for n, v in inp.items()}
    W1s, W2s = mi.shared_concat(d["W1s"], d["W2s"])
    return cfg, d, dict(W1s=W1s.contiguous(), W2s=W2s.contiguous(), shared_gate_w=d["w_s"])


@pytest.mark.parametrize("w4", [32, 128])
@pytest.mark.parametrize("world", [2, 8])
def test_partials_sum_to_the_one_gpu_layer(world, w4):
    # 1408 shared columns: over 2 ranks slices of 704 and over 8 of 176 would cut groups of 128
    cfg, d, shared = _case()
    full = MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, True, cfg.T, w4=w4, **shared).forward(d["x"]).double()
    acc, size = torch.zeros_like(full), full.norm()
    for r in range(world):
        rank = EPMoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, True, cfg.T, world, r, w4=w4, **shared)
        part = rank.forward(d["x"]).double()
        assert moe.moe_get_device_status(rank.layer.ws) == 0
        acc, size = acc + part, size + part.norm()
    assert (acc - full).norm() <= 2.0 ** -7 * size


def _norm_case(T=9):
    cfg, d, shared = _case(T)
    g = torch.Generator(device="cuda").manual_seed(3)
    norm = dict(norm_w=(1.0 + 0.2 * torch.randn(cfg.H, generator=g, device="cuda")).to(torch.bfloat16), norm_eps=1e-5)
    return cfg, d, dict(w4=64, **shared, **norm), torch.randn(T, cfg.H, generator=g, device="cuda") * 3.0


def test_block_of_the_ranks_is_the_norm_then_the_layer():
    cfg, d, options, residual = _norm_case()
    r0 = residual.clone()
    full = MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, True, cfg.T, **options).block(d["x"], r0).double()
    acc, size = torch.zeros_like(full), full.norm()
    for r in range(2):
        rank = EPMoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, True, cfg.T, 2, r, **options)
        mine = residual.clone()
        part = rank.block(d["x"], mine).double()
        assert torch.equal(mine, r0)                      # the stream, replicated
        acc, size = acc + part, size + part.norm()
    assert (acc - full).norm() <= 2.0 ** -7 * size
    rank = EPMoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, True, cfg.T, 2, 0, w4=64)
    with pytest.raises(ValueError):
        rank.block(d["x"], residual)                      # no norm


def test_block_through_the_peer_reduction():
    cfg, d, options, residual = _norm_case()
    r0 = residual.clone()
    full = MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, True, cfg.T, **options).block(d["x"], r0).double()
    reds = PeerReduction.local_set(cfg.T, cfg.H, 2, "cuda")
    ranks = [EPMoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, True, cfg.T, 2, r, peer=reds[r], **options)
             for r in range(2)]
    with pytest.raises(ValueError):                       # refused before the epoch advances
        EPMoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, True, cfg.T, 2, 0, peer=reds[0], w4=64).block(d["x"], residual)
    for step in range(3):
        mine = [residual.clone() for _ in ranks]
        for rank, m in zip(ranks, mine):                  # every partial and flag before the first reduction
            rank.write_block_partial(d["x"], m)
        outs = [rank.peer.reduce() for rank in ranks]
        torch.cuda.synchronize()
        assert all(torch.equal(m, r0) for m in mine)
        assert torch.equal(outs[0], outs[1])
        parts = [rank.peer.slots[rank.peer.epoch % 2, :cfg.T].double() for rank in ranks]
        size = full.norm() + sum(p.norm() for p in parts)
        assert (outs[0].double() - full).norm() <= 2.0 ** -7 * size
        assert all(moe.moe_get_device_status(rank.peer.ws) == 0 for rank in ranks)
