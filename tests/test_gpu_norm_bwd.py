"""moe_add_layernorm and the two norms' gradients against the 64-bit formulas of tests/bwd_ref.py.

Tolerances (derived there): a row's binary32 sums are off by at most 2^-18 of the absolute values summed, everything made
of them by at most 2^-16 of its terms' absolute values; a column sum over T rows has chains of at most T / 128 + 128
additions; one more rounding for each output's type."""
import pytest
import torch

import serving_router_gate_gb300 as moe

import bwd_ref as ref
from block_ops_ref import act_exponent

pytestmark = pytest.mark.gpu

EPS = 1e-5
TERM = 2.0 ** -16


def _inputs(T, H, f32, seed=0, mean=0.5):
    r = ref.rnd(T, H, seed=seed, std=3.0, dtype=torch.float32) + mean
    r[:, H // 2] *= 50.0
    w = (1.0 + 0.3 * ref.rnd(H, seed=seed + 1, dtype=torch.float32)).to(torch.bfloat16)
    return (r if f32 else r.to(torch.bfloat16)), w, ref.rnd(H, seed=seed + 2), ref.rnd(T, H, seed=seed + 3, std=0.01)


def _bwd(ln, dy, r, w, dstream, dr, dx, dw, db, ws, eps=EPS, stream=None):
    if ln:
        moe.moe_add_layernorm_bwd(dy, r, w, eps, dstream, dr, dx, dw, db, ws, stream)
    else:
        moe.moe_add_rmsnorm_bwd(dy, r, w, eps, dstream, dr, dx, dw, ws, stream)


def _ws(H):
    ws = torch.full((moe.moe_workspace_size_bwd(H),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    return ws


def _run(ln, dy, r, w, dstream, eps=EPS):
    H = dy.shape[1]
    dr, dx = torch.empty_like(r), torch.empty_like(dy)
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda") if ln else None
    _bwd(ln, dy, r, w, dstream, dr, dx, dw, db, _ws(H), eps)
    return dr, dx, dw, db


def _check(ln, dy, r, w, dstream, got, eps=EPS):
    dr, dx, dw, db = got
    T = dy.shape[0]
    want, mag, wd, wmag, bd, bmag = ref.norm_bwd(dy, r, w, eps, dstream, ln)
    tol = TERM * mag + 1e-37
    rnd = ref.BF * (want.abs() + tol)
    ref.inside(dr, want, tol + (0.0 if r.dtype == torch.float32 else rnd), "dr")
    ref.inside(dx, want, tol + rnd, "dx")
    chain = (T / 128 + 128) * ref.U
    ref.inside(dw, wd, (TERM + chain) * wmag + 1e-37, "dweight")
    if db is not None:
        ref.inside(db, bd, chain * bmag + 1e-37, "dbias")


@pytest.mark.parametrize("H", [8, 64, 72, 504, 512, 520, 1024, 1032, 1408, 2048, 2056, 4096, 5000, 7168, 8200, 16384])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ln", [False, True])
def test_bwd_widths(H, f32, ln):
    r, w, _, dy = _inputs(5, H, f32)
    _check(ln, dy, r, w, None, _run(ln, dy, r, w, None))


@pytest.mark.parametrize("T", [1, 2, 3, 7, 151, 153, 305, 1217, 4999])
@pytest.mark.parametrize("H", [128, 512, 2048, 7168])
@pytest.mark.parametrize("ln", [False, True])
def test_bwd_row_counts_with_a_streams_gradient(T, H, ln):
    f32 = T % 2 == 0
    r, w, _, dy = _inputs(T, H, f32, seed=1)
    ds = ref.rnd(T, H, seed=9, std=0.01, dtype=r.dtype)
    _check(ln, dy, r, w, ds, _run(ln, dy, r, w, ds))


@pytest.mark.parametrize("H", [200, 1024, 2048, 5120, 7168])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ln", [False, True])
def test_bwd_many_rows_an_sm(H, f32, ln):
    r, w, _, dy = _inputs(7001, H, f32, seed=13)
    _check(ln, dy, r, w, None, _run(ln, dy, r, w, None))


@pytest.mark.parametrize("T, H", [(3600, 3584), (2400, 5632), (310, 9728), (310, 12288), (310, 13312), (310, 16384)])
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ln", [False, True])
def test_bwd_wide_rows(T, H, stream, f32, ln):
    """With a stream's gradient and without: the widest leave it no room in shared memory."""
    r, w, _, dy = _inputs(T, H, f32, seed=14)
    ds = ref.rnd(T, H, seed=15, std=0.01, dtype=r.dtype) if stream else None
    _check(ln, dy, r, w, ds, _run(ln, dy, r, w, ds))


@pytest.mark.parametrize("H", [520, 1024, 2048, 5000, 7168, 8200, 16384])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", ["first", "last", "ramp"])
def test_bwd_parts_of_a_row_far_from_each_other(H, f32, kind):
    """The layer norm's means of a row's parts are joined to the row's."""
    r, w, _, dy = _inputs(7, H, True, seed=16)
    col = torch.arange(H, device="cuda")
    r = r + {"first": 500.0 * (col < 512), "last": 500.0 * (col >= H - 8), "ramp": 0.25 * col}[kind]
    r = r if f32 else r.to(torch.bfloat16)
    _check(True, dy, r, w, None, _run(True, dy, r, w, None))


@pytest.mark.parametrize("H", [64, 2048, 7168])
@pytest.mark.parametrize("f32", [False, True])
def test_bwd_rows_of_one_value(H, f32):
    """No variance at all: the deviations are 0 and rstd is 1 / sqrt(eps)."""
    r = torch.full((5, H), 3.25, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    _, w, _, dy = _inputs(5, H, f32, seed=17)
    _check(True, dy, r, w, None, _run(True, dy, r, w, None))


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("H", [256, 1024, 7168])
def test_bwd_in_place(ln, f32, H):
    r, w, _, dy = _inputs(333, H, f32, seed=2)
    ds = ref.rnd(333, H, seed=4, std=0.01, dtype=r.dtype)
    want = _run(ln, dy, r, w, ds)
    ws, dw = _ws(H), torch.empty(H, device="cuda")
    db = torch.empty(H, device="cuda") if ln else None
    d2, dy2, r2 = ds.clone(), dy.clone(), r.clone()
    _bwd(ln, dy2, r, w, d2, d2, dy2, dw, db, ws)             # dr over dstream, dx over dy
    _bwd(ln, dy, r2, w, ds, r2, None, None, None, None)      # dr over r
    assert torch.equal(d2, want[0]) and torch.equal(dy2, want[1]) and torch.equal(dw, want[2])
    assert torch.equal(r2, want[0])


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("T", [1, 3, 400])
def test_bwd_single_outputs_and_repeats(T, ln):
    r, w, _, dy = _inputs(T, 640, False, seed=3)
    want = _run(ln, dy, r, w, None)
    ws = _ws(640)
    for i in range(4 if ln else 3):
        one = [None] * 4
        one[i] = torch.full_like(want[i], 7.0)
        _bwd(ln, dy, r, w, None, *one, ws)
        assert torch.equal(one[i], want[i])


@pytest.mark.parametrize("H", [512, 2048, 7168])
@pytest.mark.parametrize("ln", [False, True])
def test_bwd_rows_do_not_depend_on_the_batch(H, ln):
    r, w, _, dy = _inputs(3001, H, False, seed=6)
    big = _run(ln, dy, r, w, None)
    for t in (0, 1, 1999, 3000):
        one = _run(ln, dy[t:t + 1], r[t:t + 1], w, None)
        assert torch.equal(one[0][0], big[0][t]) and torch.equal(one[1][0], big[1][t])


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("H", [264, 2048])
def test_bwd_special_rows(ln, H):
    r, w, _, dy = _inputs(8, H, True, seed=5)
    r[0] = 0.0                                   # eps alone under the root
    r[1] = 7.0                                   # equal values: no variance
    r[2] = 1e-30
    r[3] = 3.0 * torch.sign(r[3]) * 1e10          # large, its squares still finite
    dy[4] = 0.0
    _check(ln, dy, r, w, None, _run(ln, dy, r, w, None))
    dr = _run(ln, dy, r, w, None)[0]
    assert not dr[4].any()
    r[5, 3] = float("inf")
    r[6, 7] = float("nan")
    got = _run(ln, dy, r, w, None)
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(got[0][keep], dr[keep])    # a bad row stays in its row
    assert torch.isnan(got[0][6]).all() and torch.isnan(got[2]).all()


def test_layernorm_bwd_far_from_zero():
    r, w, _, dy = _inputs(33, 1408, True, seed=7, mean=3e4)
    r[:, 704] = 3e4
    _check(True, dy, r, w, None, _run(True, dy, r, w, None))


@pytest.mark.parametrize("ln", [False, True])
def test_bwd_against_differences(ln):
    """The directional derivative of sum(y * dy) along v, from the 64-bit norm at r + h v and r - h v."""
    r, w, b, dy = _inputs(3, 192, True, seed=8)
    ds = torch.zeros_like(r)
    dr, _, dw, db = _run(ln, dy, r, w, ds)
    v, h = ref.rnd(3, 192, seed=11, dtype=torch.float64), 1e-4
    f = lambda rr, ww, bb: float((ref.norm(rr, ww, bb, EPS, ln)[0] * dy.double()).sum())  # noqa: E731
    R, W, B = r.double(), w.double(), b.double()
    # third-order terms: (h |v| / std)^2 of the first, below 2^-20; the gradient's own error as in _check
    num = (f(R + h * v, W, B) - f(R - h * v, W, B)) / (2 * h)
    mag = ref.norm_bwd(dy, r, w, EPS, None, ln)[1]
    assert abs(num - float((dr.double() * v).sum())) <= 2 * TERM * float((mag * v.abs()).sum())
    vw = ref.rnd(192, seed=12, dtype=torch.float64)
    num = (f(R, W + h * vw, B) - f(R, W - h * vw, B)) / (2 * h)
    assert abs(num - float((dw.double() * vw).sum())) <= TERM * float((ref.norm_bwd(dy, r, w, EPS, None, ln)[3] * vw.abs()).sum())
    if ln:
        num = (f(R, W, B + h * vw) - f(R, W, B - h * vw)) / (2 * h)
        assert abs(num - float((db.double() * vw).sum())) <= TERM * float((dy.double().abs().sum(0) * vw.abs()).sum())


@pytest.mark.parametrize("ln", [False, True])
def test_bwd_rows_past_2_31_elements(ln):
    T, H = 140001, 16384
    g = torch.Generator("cuda").manual_seed(9)
    r = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dy = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = _inputs(1, H, False)[1]
    rows = torch.tensor([0, 1, 65535, 65536, 131071, 131072, 131073, T - 2, T - 1])
    rs, ds = r[rows].clone(), dy[rows].clone()
    wd = torch.zeros(H, dtype=torch.float64, device="cuda")
    wmag = torch.zeros_like(wd)
    for i in range(0, T, 8192):
        o = ref.norm_bwd(dy[i:i + 8192], r[i:i + 8192], w, EPS, None, ln)
        wd, wmag = wd + o[2], wmag + o[3]
    dw = torch.empty(H, device="cuda")
    _bwd(ln, dy, r, w, None, None, dy, dw, None, _ws(H))
    want, mag = ref.norm_bwd(ds, rs, w, EPS, None, ln)[:2]
    ref.inside(dy[rows], want, TERM * mag + ref.BF * (want.abs() + TERM * mag), "dx")
    ref.inside(dw, wd, (TERM + (T / 128 + 128) * ref.U) * wmag, "dweight")


@pytest.mark.parametrize("ln", [False, True])
def test_bwd_empty_batch(ln):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    n = moe.moe_get_launch_count()
    _bwd(ln, x, x, w, None, x, None, dw, db, None)
    assert moe.moe_get_launch_count() == n
    assert not dw.any() and (not ln or not db.any())


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("H", [512, 7168])
def test_bwd_on_another_stream_and_in_graphs(ln, H):
    r, w, _, dy = _inputs(640, H, False, seed=10)
    want = _run(ln, dy, r, w, None)
    got = [torch.zeros_like(t) if t is not None else None for t in want]
    ws = _ws(H)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    _bwd(ln, dy, r, w, None, *got, ws, stream=s)
    s.synchronize()
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))
    # two graphs with the same workspace, replayed one behind the other
    other = [torch.zeros_like(t) if t is not None else None for t in want]
    graphs = []
    for out in (got, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _bwd(ln, dy, r, w, None, *out, ws)
        graphs.append(g)
    for _ in range(3):
        for out in (got, other):
            for t in out:
                if t is not None:
                    t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in (got, other):
            assert all(a is None or torch.equal(a, b) for a, b in zip(out, want))


def _on_16_bytes(t):
    """A copy of t that starts 16 bytes behind a 32-byte boundary."""
    buf = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
    at = (-buf.data_ptr() % 32 + 16) // t.element_size()
    out = buf[at:at + t.numel()].view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


@pytest.mark.parametrize("H", [264, 2048, 7176])
@pytest.mark.parametrize("f32", [False, True])
def test_operands_on_16_bytes(H, f32):
    r, w, b, dy = _inputs(37, H, f32, seed=14)
    x, ds = ref.rnd(37, H, seed=25), ref.rnd(37, H, seed=26, std=0.01, dtype=r.dtype)
    want = _ln(x, r, w, b, True)
    ro, y = _on_16_bytes(torch.zeros_like(r)), _on_16_bytes(torch.zeros_like(x))
    moe.moe_add_layernorm(_on_16_bytes(x), _on_16_bytes(r), _on_16_bytes(w), _on_16_bytes(b), EPS, ro, y)
    assert torch.equal(ro, want[0]) and torch.equal(y, want[1])
    for ln in (False, True):
        want = _run(ln, dy, r, w, ds)
        got = [_on_16_bytes(torch.zeros_like(t)) if t is not None else None for t in want]
        _bwd(ln, _on_16_bytes(dy), _on_16_bytes(r), _on_16_bytes(w), _on_16_bytes(ds), *got, _ws(H))
        assert all(g is None or torch.equal(g, t) for g, t in zip(got, want))


@pytest.mark.parametrize("ln", [False, True])
def test_bwd_two_calls_at_once_beside_other_work(ln):
    """Two streams with a workspace each, and a third that keeps the GPU busy: the CTAs' sums are added whoever gets to
    run, and always in one order."""
    shapes = [(1700, 2048), (300, 512), (3000, 1024), (20, 7168)]
    data, want = [], []
    for i, (T, H) in enumerate(shapes):
        r, w, _, dy = _inputs(T, H, False, seed=30 + i)
        data.append((dy, r, w))
        want.append(_run(ln, dy, r, w, None))
    outs = [[[torch.zeros_like(t) if t is not None else None for t in w] for w in want] for _ in range(2)]
    spaces = [_ws(7168), _ws(7168)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    a = ref.rnd(2048, 2048, seed=1)
    torch.cuda.synchronize()
    for _ in range(25):
        with torch.cuda.stream(streams[2]):
            a @ a
        for i, d in enumerate(data):
            for s in range(2):
                _bwd(ln, *d, None, *outs[s][i], spaces[s], stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        for got, w in zip(outs[s], want):
            assert all(g is None or torch.equal(g, x) for g, x in zip(got, w))
        assert moe.moe_get_device_status(spaces[s]) == 0 and not spaces[s][:moe.MOE_WS_HEADER_BYTES].any()


def test_bwd_binding_refuses_what_it_would_misread():
    r, w, _, dy = _inputs(4, 64, False)
    dr, dx, dw, ws = torch.empty_like(r), torch.empty_like(dy), torch.empty(64, device="cuda"), _ws(64)
    good = dict(dy=dy, r=r, w=w, ds=None, dr=dr, dx=dx, dw=dw, ws=ws)
    for bad in (dict(dy=dy.float()), dict(dy=dy.t().contiguous().t()), dict(r=r.half()), dict(r=r[:3]), dict(w=w[:32]),
                dict(ds=r.float()), dict(dr=r.float()), dict(dx=dx.float()), dict(dw=dw.double()), dict(dw=dw[:32]),
                dict(ws=ws.view(torch.int32))):
        a = {**good, **bad}
        with pytest.raises(ValueError):
            moe.moe_add_rmsnorm_bwd(a["dy"], a["r"], a["w"], EPS, a["ds"], a["dr"], a["dx"], a["dw"], a["ws"])
    for bad_ws in (None, ws[:4096]):
        with pytest.raises(moe.MoEError) as e:
            moe.moe_add_rmsnorm_bwd(dy, r, w, EPS, None, dr, dx, dw, bad_ws)
        assert e.value.status == moe.MOE_ERR_WORKSPACE


# ------------------------------------------------------------------------------------------------ the layer norm forward

def _ln(x, r, w, b, q8, eps=EPS):
    T, H = x.shape
    ro = None if r is None else torch.empty_like(r)
    y = torch.empty_like(x)
    q = torch.full((T, H), 0xAB, dtype=torch.uint8, device="cuda") if q8 else None
    sc = torch.full((T,), -1.0, device="cuda") if q8 else None
    moe.moe_add_layernorm(x, r, w, b, eps, ro, y, q, sc)
    return ro, y, q, sc


def _check_ln(x, r, w, b, got, eps=EPS):
    ro, y, q, sc = got
    s = x.float() if r is None else r.float() + x.float()
    if r is not None:
        assert torch.equal(ro, s.to(r.dtype)), "residual_out"
    want, mag = ref.norm(s.double(), w.double(), None if b is None else b.double(), eps, True)
    tol = TERM * mag
    ref.inside(y, want, tol + ref.BF * (want.abs() + tol) + 1e-37, "y")
    if q is None:
        return
    amax, slack = want.abs().amax(1), tol.amax(1)
    lo, hi = act_exponent((amax - slack).clamp(min=0)), act_exponent(amax + slack)
    e = torch.round(torch.log2(sc.double())).to(lo.dtype)
    assert torch.equal(torch.exp2(e.double()).float(), sc) and ((e >= lo) & (e <= hi)).all()
    val = q.view(torch.float8_e4m3fn).double() * sc.double()[:, None]
    ref.inside(val, want, 2.0 ** -4 * (want.abs() + tol) + 2.0 ** -10 * sc.double()[:, None] + tol, "E4M3 values")


@pytest.mark.parametrize("H", [8, 64, 72, 520, 1408, 2040, 2048, 2056, 4096, 5000, 7168, 8200, 16384])
@pytest.mark.parametrize("f32", [False, True])
def test_layernorm_widths(H, f32):
    r, w, b, _ = _inputs(5, H, f32)
    x = ref.rnd(5, H, seed=20)
    _check_ln(x, r, w, b, _ln(x, r, w, b, True))


@pytest.mark.parametrize("T", [1, 2, 9, 153, 1217, 4999])
@pytest.mark.parametrize("H", [256, 2048, 7168])
def test_layernorm_row_counts(T, H):
    r, w, b, _ = _inputs(T, H, False, seed=1)
    x = ref.rnd(T, H, seed=21)
    _check_ln(x, r, w, b, _ln(x, r, w, b, T % 2 == 0))


def test_layernorm_without_residual_or_bias_and_in_place():
    r, w, b, _ = _inputs(77, 640, False, seed=2)
    x = ref.rnd(77, 640, seed=22)
    _check_ln(x, None, w, b, _ln(x, None, w, b, True))
    _check_ln(x, r, w, None, _ln(x, r, w, None, False))
    want = _ln(x, r, w, b, False)
    moe.moe_add_layernorm(x, r, w, b, EPS, r, x)
    assert torch.equal(r, want[0]) and torch.equal(x, want[1])


def test_layernorm_special_rows():
    H = 264
    r, w, b, _ = _inputs(6, H, True, seed=3, mean=2e4)   # far from zero
    x = ref.rnd(6, H, seed=23)
    x[0], r[0] = 0.0, 0.0
    x[1], r[1] = 1.0, 4.0                                # equal values
    ro, y, q, sc = _ln(x, r, w, b, True)
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    _check_ln(x, r, w, b, (ro, y, q, sc))
    clean = y.clone()
    x[4, 3], x[5, 7] = float("inf"), float("nan")
    ro, y, q, sc = _ln(x, r, w, b, True)
    assert torch.equal(y[:4], clean[:4]) and torch.isnan(y[4:]).all() and ((q[4:] & 0x7F) == 0x7F).all()


def test_layernorm_rows_do_not_depend_on_the_batch():
    r, w, b, _ = _inputs(4000, 2048, False, seed=6)
    x = ref.rnd(4000, 2048, seed=24)
    big = _ln(x, r, w, b, True)
    for t in (0, 1, 1999, 3999):
        for a, c in zip(_ln(x[t:t + 1], r[t:t + 1], w, b, True), big):
            assert torch.equal(a[0], c[t])


def test_layernorm_binding_refuses_what_it_would_misread():
    r, w, b, _ = _inputs(4, 64, False)
    x = ref.rnd(4, 64)
    for bad in (b.float(), b[:32], b.cpu()):
        with pytest.raises(ValueError):
            moe.moe_add_layernorm(x, r, w, bad, EPS, r, x)
