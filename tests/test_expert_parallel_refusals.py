"""A call of an expert-parallel rank that its layer refuses (a residual of another type, tensors of another device) leaves
the peer reduction's epoch and flags as they were: the next call is the other ranks' next one."""
import pytest
import torch

from serving_router_gate_gb300 import expert_parallel as ep


class Refuses:
    """A layer that refuses a residual of one row too few, and any x of odd rows in forward."""

    def check_block(self):
        pass

    def block(self, x, residual, stream=None, out=None):
        if residual.shape != x.shape:
            raise ValueError("residual has another shape")
        out.copy_(x + residual)

    def forward(self, x, stream=None, out=None):
        if x.shape[0] % 2:
            raise ValueError("odd")
        out.copy_(x)


def _rank():
    red = object.__new__(ep.PeerReduction)
    red.max_T, red.H, red.world, red.rank, red.epoch = 4, 8, 1, 0, 0
    red.slots = torch.zeros(2, 4, 8)
    flags = []
    red.signal = lambda stream=None: flags.append(red.epoch)
    rank = object.__new__(ep.EPMoELayer)
    rank.layer, rank.peer = Refuses(), red
    return rank, flags


def test_a_refused_block_does_not_advance_the_epoch():
    rank, flags = _rank()
    x, r = torch.ones(4, 8), torch.ones(4, 8)
    rank.write_block_partial(x, r)
    assert flags == [1] and rank.peer.epoch == 1
    with pytest.raises(ValueError):
        rank.write_block_partial(x, r[:3])
    assert flags == [1] and rank.peer.epoch == 1
    rank.write_block_partial(x, r)
    assert flags == [1, 2] and torch.equal(rank.peer.slots[0], x + r)


def test_a_refused_forward_does_not_advance_the_epoch():
    rank, flags = _rank()
    with pytest.raises(ValueError):
        rank.write_partial(torch.ones(3, 8))
    assert flags == [] and rank.peer.epoch == 0
    rank.write_partial(torch.ones(2, 8))
    assert flags == [1]
