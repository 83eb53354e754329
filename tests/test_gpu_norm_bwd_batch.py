"""A row's gradient does not depend on the rows beside it: the same bits from a long batch and from its pieces, at every
layout of a row (16 and 32 columns a thread, dstream in shared memory and beside it)."""
import pytest
import torch

import serving_router_gate_gb300 as moe

import bwd_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [512, 1408, 2560, 2816, 3584, 4096, 4608, 5120, 6144, 7168, 8200, 12288])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("ln", [False, True])
def test_every_row_of_a_batch_and_of_its_pieces(H, f32, stream, ln):
    T = 6001
    g = torch.Generator("cuda").manual_seed(H)
    new = lambda std, dt: (torch.randn(T, H, generator=g, device="cuda") * std).to(dt)  # noqa: E731
    rt = torch.float32 if f32 else torch.bfloat16
    r, dy = new(3.0, rt) + 0.5, new(0.01, torch.bfloat16)
    ds = new(0.01, rt) if stream else None
    w = ref.rnd(H, seed=1)

    def run(lo, hi, dr):
        a = (dy[lo:hi], r[lo:hi], w, 1e-5, None if ds is None else ds[lo:hi], dr[lo:hi], None, None)
        moe.moe_add_layernorm_bwd(*a, None, None) if ln else moe.moe_add_rmsnorm_bwd(*a, None)

    whole, parts = torch.empty_like(r), torch.empty_like(r)
    run(0, T, whole)
    lo = 0
    for n in (1, 3, 32, 300, 777, 1408, T):
        run(lo, min(T, lo + n), parts)
        lo = min(T, lo + n)
    assert lo == T and torch.equal(parts, whole)
