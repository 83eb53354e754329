"""The layer norm and its gradient on rows of little or no variance far from zero, whose values have full mantissas, so
that no binary32 sum of them is exact.

Tolerances: a sum of a row has no chain of more than 64 additions, so the mean that is taken first is off by at most
2^-18 A, A the row's largest absolute value; the deviations' own sum leaves 2^-18 of that.  So with k = 2^-18 A rstd the
normalised values are off by 2^-18 k beside what a row about zero has (2^-16 of the terms' absolute values, as in
tests/bwd_ref.py), and the variance, of which up to (2^-18 A)^2 is taken off again, by 2^-18 of that: 2^-18 k^2 of itself,
and up to 4 times that where a row's parts are joined.  All of it lies within 2^-16 K of the terms, K = 1 + k + 4 k^2.
Without the second sum the normalised values would be off by k: 1 to 300 times as much."""
import pytest
import torch

import serving_router_gate_gb300 as moe

import bwd_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-5
TERM = 2.0 ** -16
WIDTHS = [8, 72, 264, 520, 1000, 1408, 2048, 4096, 5000, 5640, 6144, 7168, 8192, 12288, 16384]
VALUES = [100.3, -1234.567, 10000.3, 77777.7]


def _rows(H, seed):
    """(x, residual): four rows of one value, two of little variance far from zero, one about zero, fp32 residual."""
    x = torch.zeros(7, H, dtype=torch.bfloat16, device="cuda")
    res = torch.zeros(7, H, device="cuda")
    res[:4] = torch.tensor(VALUES, device="cuda")[:, None]
    res[4], res[5] = 10000.3, -333.3
    x[4], x[5], x[6] = ref.rnd(H, seed=seed, std=0.02), ref.rnd(H, seed=seed + 1, std=0.003), ref.rnd(H, seed=seed + 2)
    return x, res


def _vec(H, seed):
    w = (1.0 + 0.3 * ref.rnd(H, seed=seed, dtype=torch.float32)).to(torch.bfloat16)
    return w, ref.rnd(H, seed=seed + 1)


def _norm(r):
    """Deviations, rstd and K of the rows r (float64)."""
    d = r - r.mean(1, keepdim=True)
    d = torch.where(r.amax(1, keepdim=True) == r.amin(1, keepdim=True), 0.0, d)
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    k = 2.0 ** -18 * r.abs().amax(1, keepdim=True) * rstd
    return d, rstd, 1.0 + k + 4.0 * k * k


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("q8", [False, True])
def test_layernorm_of_rows_far_from_zero(H, q8):
    x, res = _rows(H, 3)
    w, b = _vec(H, 7)
    ro, y = torch.empty_like(res), torch.empty_like(x)
    q = torch.empty(x.shape, dtype=torch.uint8, device="cuda") if q8 else None
    sc = torch.empty(x.shape[0], device="cuda") if q8 else None
    moe.moe_add_layernorm(x, res, w, b, EPS, ro, y, q, sc)
    r = res + x.float()
    assert torch.equal(ro, r)
    d, rstd, K = _norm(r.double())
    want = d * rstd * w.double() + b.double()
    tol = TERM * (K * ((d * rstd).abs() + 1.0) * w.double().abs() + b.double().abs())
    ref.inside(y, want, tol + ref.BF * (want.abs() + tol), "y")
    assert all(torch.equal(y[t], b) for t in range(4))      # rows of one value: the bias itself
    if q8:
        val = q.view(torch.float8_e4m3fn).double() * sc.double()[:, None]
        ref.inside(val, want, 2.0 ** -4 * (want.abs() + tol) + 2.0 ** -10 * sc.double()[:, None] + tol, "E4M3 values")


def _bf16_rows(H, seed):
    """Rows of one value, and of one value but for a few columns a bf16 step apart; one row about zero."""
    r = torch.zeros(7, H, device="cuda")
    r[:4] = torch.tensor(VALUES, device="cuda")[:, None]
    r[4], r[5], r[6] = 10000.3, -333.3, ref.rnd(H, seed=seed + 2)
    r = r.to(torch.bfloat16)
    r.view(torch.int16)[4, ::3] += 1
    r.view(torch.int16)[5, H // 2] += 1
    return r


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("stream", [False, True])
def test_gradients_of_rows_far_from_zero(H, f32, stream):
    """A bf16 stream: the sums of rows of one value are exact.  Elsewhere the mean is off by its last rounding and one
    more, 2^-23 A at most, which is 2^-16 of 2^-7 A rstd in the normalised values."""
    x, res = _rows(H, 3)
    r = res + x.float() if f32 else _bf16_rows(H, 3)
    w, _ = _vec(H, 7)
    dy = ref.rnd(7, H, seed=11, std=0.01)
    ds = ref.rnd(7, H, seed=12, std=0.01, dtype=r.dtype) if stream else None
    dr, dx = torch.empty_like(r), torch.empty_like(dy)
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.zeros(moe.moe_workspace_size_bwd(H), dtype=torch.uint8, device="cuda")
    moe.moe_add_layernorm_bwd(dy, r, w, EPS, ds, dr, dx, dw, db, ws)
    d, rstd, K = _norm(r.double())
    if not f32:
        A = r.double().abs().amax(1, keepdim=True)
        K = torch.where((d == 0.0).all(1, keepdim=True), 1.0, 1.0 + 2.0 ** -7 * A * rstd)
    g = dy.double() * w.double()
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    want = rstd * (g - mean(g) - d * rstd * rstd * mean(g * d))
    amag = mean((g * d).abs()) + mean(g.abs()) / rstd
    mag = rstd * K * (g.abs() + mean(g.abs()) + (d.abs() + 1.0 / rstd) * rstd * rstd * amag)
    if stream:
        want, mag = want + ds.double(), mag + ds.double().abs()
    tol = TERM * mag
    rnd = ref.BF * (want.abs() + tol)
    ref.inside(dr, want, tol + (0.0 if f32 else rnd), "dr")
    ref.inside(dx, want, tol + rnd, "dx")
    xh = d * rstd
    wmag = (dy.double().abs() * K * (xh.abs() + 1.0)).sum(0)
    ref.inside(dw, (dy.double() * xh).sum(0), (TERM + 129 * ref.U) * wmag, "dweight")
    ref.inside(db, dy.double().sum(0), 129 * ref.U * dy.double().abs().sum(0), "dbias")
