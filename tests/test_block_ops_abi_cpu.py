"""Refusals of the norm's and the 4-bit products' entry points: every call here fails validation on the host (or has
nothing to do), so no pointer is dereferenced and no CUDA call is made."""

import pytest
import torch

import serving_router_gate_gb300 as moe

FAKE = 0x1000
ODD = 0x1008   # not 16-byte aligned
INVALID, UNSUPPORTED, WORKSPACE, OK = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE,
                                       moe.MOE_OK)


def _norm(x=FAKE, res=FAKE, f32=0, w=FAKE, eps=1e-6, T=4, H=64, ro=FAKE, y=FAKE, q=None, scale=None):
    return moe._lib.moe_add_rmsnorm(x, res, f32, w, eps, T, H, ro, y, q, scale, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(f32=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(H=60), UNSUPPORTED), (dict(H=16392), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(res=None), INVALID),  # a stream output without a stream
    (dict(ro=None, y=None), INVALID), (dict(q=FAKE), INVALID), (dict(scale=FAKE), INVALID),
    (dict(x=ODD), INVALID), (dict(res=ODD), INVALID), (dict(w=ODD), INVALID), (dict(ro=ODD), INVALID),
    (dict(y=ODD), INVALID), (dict(q=FAKE + 4, scale=FAKE), INVALID), (dict(q=FAKE, scale=FAKE + 2), INVALID),
    (dict(T=0, x=None, w=None), OK)])
def test_norm_refusals(kw, want):
    assert _norm(**kw) == want


def _matvec(x=FAKE, q=FAKE, s=FAKE, M=2, N=8, K=256, group=64, y=FAKE):
    return moe._lib.moe_matvec_w4(x, q, s, M, N, K, group, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(group=0), INVALID),
    (dict(group=48), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=256), UNSUPPORTED),
    (dict(K=96), UNSUPPORTED), (dict(K=1 << 21), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(y=None), INVALID),
    (dict(x=ODD), INVALID), (dict(q=ODD), INVALID), (dict(s=FAKE + 1), INVALID), (dict(y=FAKE + 1), INVALID),
    (dict(M=0, x=None, q=None, s=None, y=None), OK)])
def test_matvec_refusals(kw, want):
    assert _matvec(**kw) == want


def test_matvec_work_that_its_kernel_could_not_count():
    # ceil(M / 8) ceil(N / 32) ceil(K / 128) pieces of work, below 2^31 - 2^20
    assert _matvec(M=1 << 30, N=1 << 30, K=1 << 20, group=128) == UNSUPPORTED
    assert _matvec(M=8 * 2048, N=32 * 1024, K=128 * 1024) == UNSUPPORTED      # 2^31
    assert _matvec(M=8 * 2047, N=32 * 1024, K=128 * 1024) == UNSUPPORTED      # 2^31 - 2^20
    assert _matvec(M=8 * 2047, N=32 * 1024, K=128 * 1024, y=None) == UNSUPPORTED
    assert _matvec(M=8 * 2046, N=32 * 1024, K=128 * 1024, y=None) == INVALID  # counted; refused for y


def _quant(w=FAKE, rows=2, K=256, group=64, q=FAKE, s=FAKE):
    return moe._lib.moe_quantize_w4_rows(w, rows, K, group, q, s, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(group=-32), INVALID), (dict(group=100), UNSUPPORTED),
    (dict(K=200), UNSUPPORTED), (dict(w=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(w=ODD), INVALID), (dict(q=FAKE + 2), INVALID), (dict(s=FAKE + 1), INVALID), (dict(rows=0), OK)])
def test_quantise_refusals(kw, want):
    assert _quant(**kw) == want


def _forward(x=FAKE, off=FAKE, S=8, P=8, src=FAKE, w1=FAKE, s1=FAKE, w2=FAKE, s2=FAKE, H=256, I=128, group=64, pr=FAKE,
             tw=FAKE, T=4, k=2, sh=(None, None, None, None), I_sh=0, gate=None, out=FAKE, ws=FAKE, wsb=1 << 30):
    return moe._lib.moe_forward_w4(x, off, S, P, src, w1, s1, w2, s2, H, I, group, pr, tw, T, k, *sh, I_sh, gate, out,
                                   ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(S=0), INVALID), (dict(k=0), INVALID), (dict(P=-1), INVALID),
    (dict(group=0), INVALID), (dict(I_sh=-64), INVALID),
    (dict(H=200), UNSUPPORTED), (dict(I=100), UNSUPPORTED), (dict(I=192, group=128), UNSUPPORTED),
    (dict(group=16), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(S=1025), UNSUPPORTED),
    (dict(I_sh=64, group=128), UNSUPPORTED), (dict(P=1 << 31), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(off=None), INVALID), (dict(src=None), INVALID), (dict(w1=None), INVALID),
    (dict(s2=None), INVALID), (dict(pr=None), INVALID), (dict(out=None), INVALID),
    (dict(I_sh=64), INVALID),                      # a shared size without shared weights
    (dict(gate=FAKE), INVALID),                    # a gate without a shared expert
    (dict(x=ODD), INVALID), (dict(w1=ODD), INVALID), (dict(out=ODD), INVALID), (dict(s1=FAKE + 1), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=300), WORKSPACE), (dict(T=0, x=None, off=None), OK)])
def test_forward_w4_refusals(kw, want):
    assert _forward(**kw) == want


def test_forward_w4_work_that_its_kernels_could_not_count():
    big = dict(H=16384, I=8192, group=128)
    assert _forward(T=1 << 20, k=1, P=1 << 20, **big) == UNSUPPORTED
    assert _forward(T=1 << 20, k=1, P=8, I_sh=16384, sh=(FAKE,) * 4, **big) == UNSUPPORTED
    assert _forward(T=1 << 10, k=1, P=1 << 10, wsb=300, **big) == WORKSPACE   # counted; the workspace is too small


def test_forward_w4_workspace():
    n = moe.moe_workspace_size_w4(32, 2048, 1408, 6, 5632)
    assert n >= 256 + 32 * 6 * (1408 * 2 + 2048 * 4) + 32 * (5632 * 2 + 2048 * 4)
    assert _forward(T=32, k=6, P=192, H=2048, I=1408, I_sh=5632, sh=(FAKE,) * 4, wsb=n - 1) == WORKSPACE
    assert moe.moe_workspace_size_w4(0, 64, 64, 1) > 0
    for bad in ((-1, 64, 64, 1, 0), (1, 100, 64, 1, 0), (1, 64, 60, 1, 0), (1, 64, 64, 0, 0), (1, 64, 64, 33, 0),
                (1, 64, 64, 1, 65)):
        assert moe._lib.moe_workspace_size_w4(*bad) == 0
    with pytest.raises(moe.MoEError):
        moe.moe_workspace_size_w4(1, 100, 64, 1)


def _rows(xq=FAKE, xs=FAKE, T=4, H=256, I=128, s1=FAKE, x=FAKE, sh=(None,) * 4, I_sh=0, gate=None, wsb=1 << 30):
    return moe._lib.moe_forward_w8a8_rows(xq, xs, FAKE, 8, 8, FAKE, s1, FAKE, FAKE, H, I, FAKE, FAKE, T, 2, x, *sh,
                                          I_sh, gate, FAKE, FAKE, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(xq=None), INVALID), (dict(xs=None), INVALID), (dict(xq=ODD), INVALID), (dict(xs=FAKE + 2), INVALID),
    (dict(s1=None), INVALID), (dict(T=-1), INVALID), (dict(H=100), UNSUPPORTED), (dict(I_sh=64), INVALID),
    (dict(gate=FAKE), INVALID), (dict(x=None, I_sh=64, sh=(FAKE,) * 4, gate=FAKE), INVALID),
    (dict(wsb=300), WORKSPACE), (dict(T=0, xq=None, xs=None), OK)])
def test_w8a8_rows_refusals(kw, want):
    assert _rows(**kw) == want


def test_binding_refuses_what_is_no_cuda_tensor():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(x, x, w, 1e-6, x, x)
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_matvec_w4(x, q, s, torch.zeros(2, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.moe_quantize_w4_rows(torch.zeros(8, 64, dtype=torch.bfloat16), q, s)
