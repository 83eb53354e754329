"""moe_add_rmsnorm against the 64-bit formulas of tests/block_ops_ref.py, and the E4M3 rows' way into the experts.

Tolerances (derived from the definition):
  * residual_out is one binary32 addition (and one rounding to bf16): bitwise;
  * y: one bf16 rounding (2^-8 relative, the half spacing at a binade's bottom) of a binary32 value whose own relative
    error is at most (H / 8 + 20) 2^-24 (any order of the sum of squares, halved by the root, plus the products):
    below 2^-12 for H <= 16384;
  * scale: exact unless max|y| lies within that error of 448 2^e; q: the E4M3 rounding (2^-4 relative, 2^-10 of the
    scale below the smallest normal) plus the same 2^-12.
"""
import pytest
import torch

import moe_inputs as mi
import serving_router_gate_gb300 as moe
from serving_router_gate_gb300.layer import layer_from_inputs

from block_ops_ref import act_exponent, e4m3_round, rmsnorm

pytestmark = pytest.mark.gpu

EPS = 1e-6
F32_ERR = 2.0 ** -12


def _run(x, residual, w, eps=EPS, q8=True, in_place=False):
    T, H = x.shape
    x, w = x.cuda(), w.cuda()
    residual = None if residual is None else residual.cuda()
    ro = None if residual is None else (residual if in_place else torch.empty_like(residual))
    y = x if in_place else torch.empty_like(x)
    q = torch.full((T, H), 0xAB, dtype=torch.uint8, device="cuda") if q8 else None
    sc = torch.full((T,), -1.0, device="cuda") if q8 else None
    moe.moe_add_rmsnorm(x, residual, w, eps, ro, y, q, sc)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in (ro, y, q, sc)]


def _check(x, residual, w, got, eps=EPS):
    ro, y, q, sc = got
    r, ref = rmsnorm(x, residual, w, eps)
    if residual is not None:
        want = r.float().to(residual.dtype)
        assert torch.equal(ro, want), "residual_out differs"
    err = (y.double() - ref).abs()
    assert (err <= (2.0 ** -8 + F32_ERR) * ref.abs() + 1e-37).all(), float((err / ref.abs().clamp(min=1e-30)).max())
    if q is None:
        return
    amax = ref.abs().amax(dim=1)
    lo, hi = act_exponent(amax * (1 - F32_ERR)), act_exponent(amax * (1 + F32_ERR))
    e = torch.round(torch.log2(sc.double())).to(lo.dtype)
    assert torch.equal(torch.exp2(e.double()).float(), sc)
    assert ((e == lo) | (e == hi)).all(), "scale"
    val = q.view(torch.float8_e4m3fn).double() * sc.double()[:, None]
    tol = (2.0 ** -4 + 2 * F32_ERR) * ref.abs() + 2.0 ** -10 * sc.double()[:, None]
    assert ((val - ref).abs() <= tol).all(), "E4M3 values"
    # all but the values next to a rounding boundary are the E4M3 values of the exact norm
    same = (val == e4m3_round(ref / sc.double()[:, None]) * sc.double()[:, None])
    assert same.double().mean() > 0.995


def _inputs(T, H, f32, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + H)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    r = torch.randn(T, H, generator=g) * 3.0
    r[:, H // 2] *= 50.0
    w = (1.0 + 0.3 * torch.randn(H, generator=g)).to(torch.bfloat16)
    return x, (r if f32 else r.to(torch.bfloat16)), w


@pytest.mark.parametrize("H", [8, 64, 72, 1408, 2040, 2048, 2056, 4096, 5000, 7168, 8192, 8200, 16384])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_widths(H, f32):
    x, r, w = _inputs(5, H, f32)
    _check(x, r, w, _run(x, r, w))


@pytest.mark.parametrize("T", [1, 2, 3, 7, 151, 153, 1217, 4999])
@pytest.mark.parametrize("H", [256, 2048, 7168])
def test_norm_row_counts(T, H):
    x, r, w = _inputs(T, H, False, seed=1)
    _check(x, r, w, _run(x, r, w))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_norm_in_place(f32, q8):
    x, r, w = _inputs(333, 1024, f32, seed=2)
    _check(x, r, w, _run(x, r, w, q8=q8, in_place=True))


def test_norm_without_residual():
    x, _, w = _inputs(9, 640, False, seed=3)
    _check(x, None, w, _run(x, None, w))


@pytest.mark.parametrize("which", ["residual", "y", "q"])
def test_norm_single_outputs(which):
    x, r, w = (t.cuda() for t in _inputs(40, 512, False, seed=4))
    full = [torch.empty_like(r), torch.empty_like(x), torch.empty(40, 512, dtype=torch.uint8, device="cuda"),
            torch.empty(40, device="cuda")]
    moe.moe_add_rmsnorm(x, r, w, EPS, *full)
    one = [torch.empty_like(t) for t in full]
    pick = {"residual": [one[0], None, None, None], "y": [None, one[1], None, None],
            "q": [None, None, one[2], one[3]]}[which]
    moe.moe_add_rmsnorm(x, r, w, EPS, *pick)
    torch.cuda.synchronize()
    for a, b in zip(pick, full):
        if a is not None:
            assert torch.equal(a, b)


def test_norm_special_rows():
    H = 264
    x, r, w = _inputs(8, H, True, seed=5)
    x[0], r[0] = 0.0, 0.0                       # zeros: y = 0, the smallest scale
    r[1] = -x[1].float()                        # a sum of exact zeros
    x[2], r[2] = 0.0, 1e-30                     # far below eps: y = r / sqrt(eps)
    x[3], r[3] = 0.0, 1e15                      # large, its squares still finite
    ro, y, q, sc = _run(x, r, w)
    for t in (0, 1):
        assert not y[t].any() and not q[t].any() and sc[t] == 2.0 ** -126
    _check(x[2:], r[2:], w, [ro[2:], y[2:], q[2:], sc[2:]])
    x[4, 3] = float("inf")
    x[5, 7] = float("nan")
    ro, y, q, sc = _run(x, r, w)
    # an infinity: rstd = 0, the row's finite values become 0 and the infinity 0 * inf = NaN
    assert torch.isnan(y[4, 3]) and not y[4, :3].any() and not y[4, 4:].any()
    assert (q[4, 3] & 0x7F) == 0x7F and not (q[4, 4:] & 0x7F).any()
    assert torch.isnan(y[5].float()).all() and ((q[5] & 0x7F) == 0x7F).all()
    ok = [t for t in range(8) if t not in (0, 1, 4, 5)]
    _check(x[ok], r[ok], w, [ro[ok], y[ok], q[ok], sc[ok]])


def test_norm_rows_do_not_depend_on_the_batch():
    x, r, w = _inputs(4000, 2048, False, seed=6)
    big = _run(x, r, w)
    for t in (0, 1, 1999, 3999):
        one = _run(x[t:t + 1], r[t:t + 1], w)
        for a, b in zip(one, big):
            assert torch.equal(a[0], b[t])


def test_norm_rows_past_2_31_elements():
    T, H = 140001, 16384
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(9))
    r = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(10))
    w = _inputs(1, H, False)[2].cuda()
    rows = torch.tensor([0, 1, 65535, 65536, 131071, 131072, 131073, T - 2, T - 1])
    xs, rs = x[rows].cpu(), r[rows].cpu()
    q, sc = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_add_rmsnorm(x, r, w, EPS, r, x, q, sc)
    _check(xs, rs, w.cpu(), [t[rows].cpu() for t in (r, x, q, sc)])


def test_norm_binding_refuses_what_it_would_misread():
    x, r, w = (t.cuda() for t in _inputs(4, 64, False))
    y, q, sc = torch.empty_like(x), torch.empty(4, 64, dtype=torch.uint8, device="cuda"), torch.empty(4, device="cuda")
    good = dict(x=x, r=r, w=w, ro=r, y=y, q=q, sc=sc)
    for bad in (dict(x=x.t().contiguous().t()), dict(x=x.float()), dict(r=r.half()), dict(r=r[:3]), dict(w=w[:32]),
                dict(w=w.float()), dict(ro=r.float()), dict(y=y.t().contiguous().t()), dict(q=q.view(torch.int8)),
                dict(sc=sc[:3])):
        a = {**good, **bad}
        with pytest.raises(ValueError):
            moe.moe_add_rmsnorm(a["x"], a["r"], a["w"], EPS, a["ro"], a["y"], a["q"], a["sc"])


def test_norm_empty_batch():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    n = moe.moe_get_launch_count()
    moe.moe_add_rmsnorm(x, x, w, EPS, x, x)
    assert moe.moe_get_launch_count() == n


def test_norm_on_another_stream_and_in_a_graph():
    x, r, w = (t.cuda() for t in _inputs(64, 512, False, seed=7))
    want = [torch.empty_like(r), torch.empty_like(x)]
    moe.moe_add_rmsnorm(x, r, w, EPS, *want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [torch.empty_like(r), torch.empty_like(x)]
    moe.moe_add_rmsnorm(x, r, w, EPS, *got, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_add_rmsnorm(x, r, w, EPS, *got)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [3, 100])
@pytest.mark.parametrize("shared", [False, True])
def test_w8a8_rows_equal_the_call_that_quantises(T, shared):
    cfg = mi.MoEConfig("rows", T=T, H=512, I=256, E=8, k=3, renorm=True, fp8=True, act8=True,
                       n_shared=1 if shared else 0, I_shared=256, shared_gate=shared)
    inp = mi.make_inputs(cfg)
    layer = layer_from_inputs(inp, "cuda")
    x = inp["x"].cuda()
    want = layer.forward(x).clone()
    xq = torch.empty(T, cfg.H, dtype=torch.uint8, device="cuda")
    xs = torch.empty(T, device="cuda")
    moe.moe_quantize_act_rows(x, xq, xs)
    layer.ws[moe.MOE_WS_HEADER_BYTES:].fill_(0xFF)
    v = layer.expert_forward(x, None, None, xq, xs)
    torch.cuda.synchronize()
    assert torch.equal(v["out"], want)
    assert moe.moe_get_device_status(layer.ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "w8a8", "nvfp4"])
def test_block_is_the_norm_then_the_layer(fmt):
    cfg = mi.MoEConfig("block", T=37, H=512, I=256, E=8, k=3, renorm=True, fp8=fmt == "w8a8", act8=fmt == "w8a8",
                       fp4=fmt == "nvfp4", n_shared=1, I_shared=256, shared_gate=True)
    inp = mi.make_inputs(cfg)
    layer = layer_from_inputs(inp, "cuda")
    x, r, w = (t.cuda() for t in _inputs(37, 512, False, seed=8))
    with pytest.raises(ValueError):
        layer.block(x, r)
    from serving_router_gate_gb300.layer import MoELayer
    block = MoELayer(layer.Wg, layer.W1, layer.W2, cfg.k, cfg.renorm, cfg.T, W1s=layer.W1s, W2s=layer.W2s,
                     shared_gate_w=layer.gate, fp8=cfg.fp8, act8=cfg.act8, fp4=cfg.fp4, norm_w=w, norm_eps=EPS)
    r0 = r.clone()
    out = block.block(x, r).clone()
    ro, y = torch.empty_like(r), torch.empty_like(x)
    moe.moe_add_rmsnorm(x, r0, w, EPS, ro, y)
    want = layer.forward(y)
    torch.cuda.synchronize()
    assert torch.equal(r, ro)
    if fmt == "w8a8":  # the experts' rows are rounded once instead of twice: E4M3 codes differ at some boundaries
        rel = (out.double() - want.double()).norm() / want.double().norm()
        assert rel < 2.0 ** -4
    else:
        assert torch.equal(out, want)
    assert moe.moe_get_device_status(block.ws) == 0
