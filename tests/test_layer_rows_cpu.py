"""MoELayer.expert_forward takes token rows that are E4M3 already only where the layer's own rows would be such."""
import pytest
import torch

from serving_router_gate_gb300 import layer as L

CALLS = ("moe_forward", "moe_forward_fp8", "moe_forward_nvfp4", "moe_forward_w4", "moe_forward_w8a8",
         "moe_forward_w8a8_rows")


def _layer(monkeypatch, on_input=False, fp8=False, act8=False, fp4=False, w4=0):
    """A layer of 4 tokens without weights, and the names of the library calls that it makes."""
    made = []
    for n in CALLS:
        monkeypatch.setattr(L, n, lambda *a, _n=n, **k: made.append(_n))
    la = object.__new__(L.MoELayer)
    la.on_input, la.fp8, la.act8, la.fp4, la.w4, la.k, la.I_sh = on_input, fp8, act8, fp4, w4, 2, 0
    for n in ("topk_ids", "topk_w", "slot_ids", "counts", "offsets", "perm_src", "pair_row", "x_perm", "out"):
        setattr(la, n, torch.zeros(8))
    for n in ("W1", "W2", "W1s", "W2s", "W1q", "s1", "W2q", "s2", "W1sq", "s1s", "W2sq", "s2s", "gate", "ws", "W1sf",
              "W1sw4"):
        setattr(la, n, None)
    la.W1f = la.W2f = (None,) * 3
    la.W1w4 = la.W2w4 = (None,) * 2
    return la, made


@pytest.mark.parametrize("kw", [dict(), dict(fp8=True), dict(fp4=True), dict(w4=64),
                                dict(fp8=True, act8=True, on_input=True)])
def test_rows_in_e4m3_are_refused_by_other_formats(monkeypatch, kw):
    # (with the weights on the input the rows are those of x_perm: the token rows' codes are not weighted)
    la, made = _layer(monkeypatch, **kw)
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        la.expert_forward(x, x_q=torch.zeros(4, 8, dtype=torch.uint8), x_scale=torch.ones(4))
    assert made == []
    la.expert_forward(x)
    assert len(made) == 1 and made[0] != "moe_forward_w8a8_rows"


def test_rows_in_e4m3_reach_the_e4m3_experts(monkeypatch):
    la, made = _layer(monkeypatch, fp8=True, act8=True)
    la.expert_forward(torch.zeros(4, 8), x_q=torch.zeros(4, 8, dtype=torch.uint8), x_scale=torch.ones(4))
    assert made == ["moe_forward_w8a8_rows"]
