"""Refusals of the layer norm's and the gradients' entry points: every call here fails validation on the host (or has
nothing to do), so no pointer is dereferenced and no CUDA call is made."""
import pytest
import torch

import serving_router_gate_gb300 as moe

FAKE = 0x1000
ODD = 0x1008   # not 16-byte aligned
INVALID, UNSUPPORTED, WORKSPACE, OK = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE,
                                       moe.MOE_OK)
NEED = moe.moe_workspace_size_bwd(64)


def _ln(x=FAKE, res=FAKE, f32=0, w=FAKE, b=FAKE, eps=1e-5, T=4, H=64, ro=FAKE, y=FAKE, q=None, scale=None):
    return moe._lib.moe_add_layernorm(x, res, f32, w, b, eps, T, H, ro, y, q, scale, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(f32=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(H=60), UNSUPPORTED), (dict(H=16392), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(res=None), INVALID), (dict(ro=None, y=None), INVALID),
    (dict(q=FAKE), INVALID), (dict(scale=FAKE), INVALID), (dict(x=ODD), INVALID), (dict(res=ODD), INVALID),
    (dict(w=ODD), INVALID), (dict(b=ODD), INVALID), (dict(ro=ODD), INVALID), (dict(y=ODD), INVALID),
    (dict(q=FAKE + 4, scale=FAKE), INVALID), (dict(q=FAKE, scale=FAKE + 2), INVALID), (dict(T=0, x=None, w=None), OK)])
def test_layernorm_refusals(kw, want):
    assert _ln(**kw) == want


def _norm_bwd(ln, dy=FAKE, r=FAKE, f32=0, w=FAKE, eps=1e-5, T=4, H=64, ds=None, dr=FAKE, dx=None, dw=FAKE, db=None,
              ws=FAKE, wsb=NEED):
    if ln:
        return moe._lib.moe_add_layernorm_bwd(dy, r, f32, w, eps, T, H, ds, dr, dx, dw, db, ws, wsb, None)
    return moe._lib.moe_add_rmsnorm_bwd(dy, r, f32, w, eps, T, H, ds, dr, dx, dw, ws, wsb, None)


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(f32=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(H=60), UNSUPPORTED), (dict(H=16392), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(dy=None), INVALID), (dict(r=None), INVALID), (dict(w=None), INVALID),
    (dict(dr=None, dw=None), INVALID), (dict(dy=ODD), INVALID), (dict(r=ODD), INVALID), (dict(w=ODD), INVALID),
    (dict(ds=ODD), INVALID), (dict(dr=ODD), INVALID), (dict(dx=ODD), INVALID), (dict(dw=ODD), INVALID),
    (dict(ws=ODD), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=NEED - 1), WORKSPACE),
    (dict(T=0, dy=None, r=None, w=None, dr=None, dw=None, ws=None), OK)])
def test_norm_bwd_refusals(ln, kw, want):
    assert _norm_bwd(ln, **kw) == want


def test_layernorm_bwd_refuses_a_bad_bias_gradient():
    assert _norm_bwd(True, db=ODD) == INVALID
    assert _norm_bwd(True, dr=None, dw=None, db=FAKE, ws=None) == WORKSPACE


def _fin(dout=FAKE, y=FAKE, cap=8, pr=FAKE, w=FAKE, T=4, k=2, H=64, ysh=FAKE, x=FAKE, gw=FAKE, dy=FAKE, dw=FAKE, dysh=FAKE,
         dz=FAKE, dgw=FAKE, ws=FAKE, wsb=NEED):
    return moe._lib.moe_finalize_bwd(dout, y, cap, pr, w, T, k, H, ysh, x, gw, dy, dw, dysh, dz, dgw, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(H=0), INVALID), (dict(cap=-1), INVALID),
    (dict(H=72), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(cap=1 << 31), UNSUPPORTED),
    (dict(T=1 << 62), UNSUPPORTED), (dict(T=(1 << 63) // 2 + 1), UNSUPPORTED),
    (dict(dout=None), INVALID), (dict(y=None), INVALID), (dict(pr=None), INVALID), (dict(dy=None), INVALID),
    (dict(w=None), INVALID),                                   # a weight's gradient without weights
    (dict(gw=None), INVALID), (dict(ysh=None), INVALID), (dict(x=None), INVALID), (dict(dysh=None), INVALID),
    (dict(dz=None), INVALID),
    (dict(dout=ODD), INVALID), (dict(y=ODD), INVALID), (dict(pr=FAKE + 2), INVALID), (dict(w=FAKE + 2), INVALID),
    (dict(ysh=ODD), INVALID), (dict(x=ODD), INVALID), (dict(gw=ODD), INVALID), (dict(dy=ODD), INVALID),
    (dict(dw=FAKE + 2), INVALID), (dict(dysh=ODD), INVALID), (dict(dz=FAKE + 2), INVALID), (dict(dgw=ODD), INVALID),
    (dict(ws=ODD), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=NEED - 1), WORKSPACE),
    (dict(dgw=None, wsb=255), WORKSPACE), (dict(T=0, dout=None, y=None, pr=None, dy=None, dgw=None, ws=None), OK)])
def test_finalize_bwd_refusals(kw, want):
    assert _fin(**kw) == want


def _perm(dxp=FAKE, cap=8, pr=FAKE, w=FAKE, x=FAKE, add=FAKE, f32=0, dz=FAKE, gw=FAKE, T=4, k=2, H=64, dx=FAKE, dw=FAKE,
          ws=FAKE, wsb=256):
    return moe._lib.moe_permute_bwd(dxp, cap, pr, w, x, add, f32, dz, gw, T, k, H, dx, dw, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(H=0), INVALID), (dict(cap=-1), INVALID), (dict(f32=2), INVALID),
    (dict(H=72), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(cap=1 << 31), UNSUPPORTED),
    (dict(T=1 << 62), UNSUPPORTED), (dict(dxp=None), INVALID), (dict(pr=None), INVALID), (dict(dx=None), INVALID),
    (dict(w=None), INVALID), (dict(x=None), INVALID), (dict(dz=None), INVALID), (dict(gw=None), INVALID),
    (dict(dxp=ODD), INVALID), (dict(pr=FAKE + 2), INVALID), (dict(w=FAKE + 2), INVALID), (dict(x=ODD), INVALID),
    (dict(add=ODD), INVALID), (dict(dz=FAKE + 2), INVALID), (dict(gw=ODD), INVALID), (dict(dx=ODD), INVALID),
    (dict(dw=FAKE + 2), INVALID), (dict(ws=ODD), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=255), WORKSPACE),
    (dict(T=0, dxp=None, pr=None, dx=None), OK)])
def test_permute_bwd_refusals(kw, want):
    assert _perm(**kw) == want


def _route(ids=FAKE, w=FAKE, dw=FAKE, logits=FAKE, T=4, E=8, k=2, renorm=0, out=FAKE, ws=FAKE, wsb=256):
    return moe._lib.moe_route_bwd(ids, w, dw, logits, T, E, k, renorm, out, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(renorm=2), INVALID),
    (dict(E=513), UNSUPPORTED), (dict(E=64, k=33), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(T=1 << 62), UNSUPPORTED), (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(dw=None), INVALID),
    (dict(logits=None), INVALID), (dict(out=None), INVALID), (dict(ids=FAKE + 2), INVALID), (dict(w=FAKE + 2), INVALID),
    (dict(dw=FAKE + 2), INVALID), (dict(logits=ODD), INVALID), (dict(out=ODD), INVALID), (dict(ws=ODD), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=255), WORKSPACE), (dict(T=0, ids=None, out=None), OK)])
def test_route_bwd_refusals(kw, want):
    assert _route(**kw) == want


def test_workspace():
    assert NEED >= 256 + 2 * 4 * 64
    assert moe.moe_workspace_size_bwd(16384) <= 4096 + 2560 * 16384
    for bad in (0, -8, 60, 1 << 21):
        assert moe._lib.moe_workspace_size_bwd(bad) == 0
    with pytest.raises(moe.MoEError):
        moe.moe_workspace_size_bwd(60)


def test_binding_refuses_what_is_no_cuda_tensor():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    f, i = torch.zeros(2, 2), torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: moe.moe_add_layernorm(x, x, w, w, 1e-5, x, x),
                 lambda: moe.moe_add_rmsnorm_bwd(x, x, w, 1e-5, None, x, None, None, None),
                 lambda: moe.moe_add_layernorm_bwd(x, x, w, 1e-5, None, x, None, None, None, None),
                 lambda: moe.moe_finalize_bwd(x, x, i, f, None, None, None, x, f, None, None, None, None),
                 lambda: moe.moe_permute_bwd(x, i, None, None, None, None, None, x, None, None),
                 lambda: moe.moe_route_bwd(i, f, f, None, True, f, None)):
        with pytest.raises(ValueError):
            call()
