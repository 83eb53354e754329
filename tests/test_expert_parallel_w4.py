"""Expert-parallel layers on 4-bit weights: every rank's slice of the shared experts is whole groups of the format."""
import pytest
import torch

from serving_router_gate_gb300 import expert_parallel as ep


@pytest.mark.parametrize("world", [1, 2, 3, 5, 8, 16])
@pytest.mark.parametrize("w4", [32, 64, 128])
def test_shared_slices_are_whole_groups(w4, world, monkeypatch):
    # 5632 shared columns over 8 ranks: slices of 704 would cut a group of 128 in two
    E, H, I, I_sh = 16, 128, 64, 5632
    built = []

    class Layer:
        def __init__(self, Wg, W1, W2, k, renorm, max_T, **options):
            built.append(options)

    monkeypatch.setattr(ep, "MoELayer", Layer)
    W1s, W2s = torch.arange(2 * I_sh, dtype=torch.float32)[:, None], torch.arange(I_sh, dtype=torch.float32)[None, :]
    for rank in range(world):
        ep.EPMoELayer(torch.zeros(E, H), torch.zeros(E, 2 * I, H), torch.zeros(E, H, I), 2, True, 4, world, rank,
                      W1s=W1s, W2s=W2s, w4=w4)
    cols = []
    for o in built:
        assert o["w4"] == w4
        if o["W2s"] is None:
            continue
        w = o["W2s"].shape[1]
        assert w % w4 == 0 and w % 64 == 0
        c = o["W2s"][0]
        assert int(c[0]) % w4 == 0
        assert torch.equal(o["W1s"][:, 0], torch.cat([c, c + I_sh]))
        cols.append(c)
    assert torch.equal(torch.cat(cols), W2s[0])


def test_a_shared_size_that_is_no_whole_number_of_groups_is_refused():
    with pytest.raises(ValueError):
        ep.ep_shared_shard(torch.zeros(2 * 192, 1), torch.zeros(1, 192), 2, 0, unit=128)
