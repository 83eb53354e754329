"""moe_forward_w4 on routing tables that are wrong or extreme: bad entries are dropped and flagged and touch nothing
else, whatever the token rows hold."""
import pytest
import torch

import serving_router_gate_gb300 as moe

from test_gpu_w4 import _experts

pytestmark = pytest.mark.gpu

X, OFFSETS, PERM_SRC, PAIR_ROW, OUT, WS = 0, 1, 2, 7, 14, 15


def _run(args):
    out = torch.full_like(args[OUT], float("nan"))
    moe.moe_forward_w4(*args[:OUT], out, args[WS])
    status = moe.moe_get_device_status(args[WS])
    return out, status


def _same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))


@pytest.mark.parametrize("first", [0.5, float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("T,E,k", [(6, 16, 4), (40, 4, 2)])  # pieces of eight rows, of sixteen
@pytest.mark.parametrize("group", [32, 128])
def test_bad_perm_src_entries_are_dropped_and_flagged(T, E, k, group, first):
    args = list(_experts(T, 256, 128, E, k, group, seed=20))
    args[X] = args[X].clone()
    args[X][0] = first
    good = args[PERM_SRC].clone()
    rows = int(args[OFFSETS][-1])
    # rows of tokens other than 0, in slots that others share, each with an entry out of range
    picks = [r for r in range(rows) if int(good[r]) // k != 0][1::5][:6]
    values = [-1, T * k, -7, 2 ** 31 - 1, -2 ** 31, T * k + 1]
    bad = good.clone()
    dropped = args[PAIR_ROW].clone()
    for r, v in zip(picks, values):
        bad[r] = v
        dropped.reshape(-1)[int(good[r])] = -1
    without = list(args)
    without[PAIR_ROW] = dropped
    want, status = _run(without)
    assert status == 0
    args[PERM_SRC] = bad
    got, status = _run(args)
    assert status == moe.MOE_ERR_DEVICE_BOUNDS
    assert _same(got, want)
    assert torch.isfinite(got[1:].float()).all()


def test_bad_pair_row_entries_leave_the_other_pairs():
    args = list(_experts(6, 256, 128, 16, 4, 64, seed=21))
    dropped, bad = args[PAIR_ROW].clone(), args[PAIR_ROW].clone()
    for i, (t, j, v) in enumerate([(0, 0, 24), (2, 1, -2), (2, 3, 2 ** 31 - 1), (5, 2, -2 ** 31)]):
        bad[t, j], dropped[t, j] = v, -1
    args[PAIR_ROW] = dropped
    want, status = _run(args)
    assert status == 0
    args[PAIR_ROW] = bad
    got, status = _run(args)
    assert status == moe.MOE_ERR_DEVICE_BOUNDS
    assert torch.equal(got, want)


@pytest.mark.parametrize("make", [
    lambda off, cap: [0, cap] * (len(off) // 2) + [cap],            # slots that overlap, over and over
    lambda off, cap: [-1] + off[1:],
    lambda off, cap: [-2 ** 31] + off[1:],
    lambda off, cap: off[:-1] + [cap + 1],
    lambda off, cap: off[:-1] + [2 ** 31 - 1],
    lambda off, cap: off[:3] + [off[2] - 1] + off[4:],
    lambda off, cap: [cap] + [0] * (len(off) - 1),
    lambda off, cap: [2 ** 31 - 1] + [-2 ** 31] * (len(off) - 1)])
@pytest.mark.parametrize("E", [8, 500, 1024])
def test_bad_offsets_are_flagged_and_no_routed_row_is_computed(E, make):
    args = list(_experts(6, 128, 64, E, 4, 64, I_sh=64, gated=True, seed=22))
    args[WS][moe.MOE_WS_HEADER_BYTES:] = 0               # routed outputs that nothing writes read as zeros
    alone = list(args)
    alone[PAIR_ROW] = torch.full_like(args[PAIR_ROW], -1)
    want, status = _run(alone)                            # the shared expert alone
    assert status == 0
    args[WS][moe.MOE_WS_HEADER_BYTES:] = 0
    off = make(args[OFFSETS].tolist(), 24)
    assert len(off) == E + 1
    args[OFFSETS] = torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
    got, status = _run(args)
    assert status == moe.MOE_ERR_DEVICE_BOUNDS
    assert torch.equal(got, want)
