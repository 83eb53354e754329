"""The gradients of the combine, the sorted rows and the routing weights against 64-bit derivatives of the forward
formulas in tests/bwd_ref.py.

Tolerances: a dot product over H in binary32, in chains of at most H / 32 + 64 additions, is off by that many times 2^-24
of the absolute values summed; a product that is stored is rounded once more (2^-8 in bf16); a gate's logit z is off by
its dot's error e, the gate by at most e and a few roundings."""
import pytest
import torch

import serving_router_gate_gb300 as moe

import bwd_ref as ref

pytestmark = pytest.mark.gpu


def _ws(H=64):
    ws = torch.full((moe.moe_workspace_size_bwd(H),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    return ws


def _status(ws):
    return moe.moe_get_device_status(ws)


def _chain(H):
    return (H / 32 + 64) * ref.U


# ------------------------------------------------------------------------------------------------ combine

def _fin_inputs(T, H, E, k, S=None, gated=False, seed=0, pad=0):
    pr, w, rows = ref.routing(T, E, k, S, seed, pad)
    d = dict(dout=ref.rnd(T, H, seed=seed + 1, std=0.1), y=ref.rnd(rows, H, seed=seed + 2), pr=pr, w=w, ysh=None, x=None,
             gw=None)
    if gated:
        d.update(ysh=ref.rnd(T, H, seed=seed + 3), x=ref.rnd(T, H, seed=seed + 4), gw=ref.rnd(H, seed=seed + 5, std=0.05))
    return d


def _fin(d, ws, dy=None, dw=True, dgw=True, stream=None):
    T, k = d["pr"].shape
    H = d["dout"].shape[1]
    f32 = dict(dtype=torch.float32, device="cuda")
    gated = d["gw"] is not None
    o = dict(dy=torch.full_like(d["y"], 5.0) if dy is None else dy,
             dw=torch.full((T, k), 9.0, **f32) if dw else None,
             dysh=torch.empty_like(d["dout"]) if gated else None, dz=torch.empty(T, **f32) if gated else None,
             dgw=torch.empty(H, **f32) if gated and dgw else None)
    moe.moe_finalize_bwd(d["dout"], d["y"] if dw else None, d["pr"], d["w"], d["ysh"], d["x"], d["gw"], o["dy"], o["dw"],
                         o["dysh"], o["dz"], o["dgw"], ws, stream)
    return o


def _fin_check(d, o, untouched=5.0):
    T, k = d["pr"].shape
    H = d["dout"].shape[1]
    pr, dout = d["pr"].long(), d["dout"]
    live = pr >= 0
    # dy: one binary32 product, rounded once; other rows as they were
    want = torch.full_like(d["y"], untouched)
    w = torch.ones_like(live, dtype=torch.float32) if d["w"] is None else d["w"]
    for j in range(k):
        want[pr[live[:, j], j]] = (w[live[:, j], j, None] * dout[live[:, j]].float()).to(torch.bfloat16)
    assert torch.equal(o["dy"], want), "dy"
    if o["dw"] is not None:
        rows = d["y"][pr.clamp(min=0)].double()
        prod = rows * dout.double().unsqueeze(1)
        dot = prod.sum(-1) * live
        ref.inside(o["dw"], dot, _chain(H) * prod.abs().sum(-1) * live, "dtopk_w")
    if d["gw"] is None:
        return
    x, ysh, gw = d["x"].double(), d["ysh"].double(), d["gw"].double()
    g = torch.sigmoid(x @ gw)
    ez = (x * gw).abs().sum(1) * _chain(H)
    eg = g * (1 - g) * ez * 1.01 + 8 * ref.U * g
    want = g[:, None] * dout.double()
    tol = eg[:, None] * dout.double().abs()
    ref.inside(o["dysh"], want, tol + ref.BF * (want.abs() + tol), "dy_shared")
    dot, mag = (dout.double() * ysh).sum(1), (dout.double() * ysh).abs().sum(1)
    s = g * (1 - g)
    dz = s * dot
    tz = s * _chain(H) * mag + (s * ez * 1.01 + 16 * ref.U * s) * dot.abs() + 1e-30
    ref.inside(o["dz"], dz, tz, "dgate")
    if o["dgw"] is not None:
        chain = (T / 128 + 128) * ref.U
        ref.inside(o["dgw"], dz @ x, (tz[:, None] * x.abs()).sum(0) + chain * (dz[:, None] * x).abs().sum(0),
                   "dshared_gate_w")


@pytest.mark.parametrize("T,H,E,k,S", [(1, 64, 4, 1, None), (1, 2048, 64, 6, None), (2, 128, 8, 8, 4), (3, 7168, 16, 8, None),
                                       (77, 1408, 60, 4, None), (333, 64, 32, 32, 16), (1000, 2048, 64, 6, 20),
                                       (257, 192, 40, 17, 33), (64, 320, 12, 9, None), (5, 24640, 8, 3, None),
                                       (4099, 512, 60, 4, None), (130, 256, 16, 2, 0)])
@pytest.mark.parametrize("gated", [False, True])
def test_finalize_bwd(T, H, E, k, S, gated):
    d = _fin_inputs(T, H, E, k, S, gated, seed=1, pad=3)
    ws = _ws(H)
    _fin_check(d, _fin(d, ws))
    assert _status(ws) == 0


def test_finalize_bwd_options():
    d = _fin_inputs(90, 640, 16, 4, 10, True, seed=2)
    ws = _ws(640)
    full = _fin(d, ws)
    part = _fin(d, ws, dw=False, dgw=False)      # y is not read
    for n in ("dy", "dysh", "dz"):
        assert torch.equal(part[n], full[n])
    one = dict(d, w=None)                         # weight 1 for every kept pair
    _fin_check(one, _fin(one, ws, dw=False))
    y = d["y"].clone()
    got = _fin(dict(d, y=y), ws, dy=y)            # dy over y
    live = d["pr"][d["pr"] >= 0].long()
    assert torch.equal(got["dw"], full["dw"]) and torch.equal(y[live], full["dy"][live])
    dead = torch.ones(y.shape[0], dtype=torch.bool, device="cuda")
    dead[live] = False
    assert torch.equal(y[dead], d["y"][dead])
    # a small workspace serves where no weight gradient is asked for
    small = torch.zeros(moe.MOE_WS_HEADER_BYTES, dtype=torch.uint8, device="cuda")
    got = _fin(d, small, dgw=False)
    assert torch.equal(got["dz"], full["dz"])


def test_finalize_bwd_bad_rows_are_dropped_and_flagged():
    d = _fin_inputs(40, 256, 8, 4, seed=3)
    ws = _ws(256)
    want = _fin(d, ws)
    pr = d["pr"].clone()
    for t, j, bad in ((0, 0, -2), (7, 3, pr.numel()), (39, 1, 2 ** 31 - 1), (20, 2, -2 ** 31)):
        r = int(pr[t, j])
        pr[t, j] = bad
        want["dy"][r] = 5.0
        want["dw"][t, j] = 0.0
    got = _fin(dict(d, pr=pr), ws)
    assert torch.equal(got["dy"], want["dy"]) and torch.equal(got["dw"], want["dw"])
    assert _status(ws) == moe.MOE_ERR_DEVICE_BOUNDS


def test_finalize_bwd_bad_values_stay_in_their_rows():
    d = _fin_inputs(40, 256, 8, 4, gated=True, seed=4)
    ws = _ws(256)
    want = _fin(d, ws)
    d["dout"][3, 5] = float("nan")
    d["y"][int(d["pr"][9, 1]), 0] = float("inf")
    d["x"][12] = 1e4                              # a gate at its end: its logit's gradient vanishes
    got = _fin(d, ws)
    keep = [t for t in range(40) if t not in (3, 9, 12)]
    for n in ("dw", "dysh", "dz"):
        assert torch.equal(got[n][keep], want[n][keep])
    assert torch.isnan(got["dw"][3]).all() and torch.isnan(got["dz"][3]) and not torch.isfinite(got["dw"][9, 1])
    assert float(got["dz"][12]) == 0.0 or abs(float(got["dz"][12])) < 1e-30


def test_finalize_bwd_rows_past_2_31_elements():
    T, k, H = 37000, 9, 7168
    pr, w, rows = ref.routing(T, 16, k, None, 5)
    g = torch.Generator("cuda").manual_seed(3)
    y = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dout = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ws = _ws(64)
    pick = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    keep_rows = pr[pick].long()
    ysub = y[keep_rows].clone()
    dw = torch.empty(T, k, device="cuda")
    moe.moe_finalize_bwd(dout, y, pr, w, None, None, None, y, dw, None, None, None, ws)
    prod = ysub.double() * dout[pick].double().unsqueeze(1)
    ref.inside(dw[pick], prod.sum(-1), _chain(H) * prod.abs().sum(-1), "dtopk_w")
    assert torch.equal(y[keep_rows], (w[pick].unsqueeze(-1) * dout[pick].float().unsqueeze(1)).to(torch.bfloat16))
    # and the way back over the same rows
    dx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_permute_bwd(y, pr, None, None, None, None, None, dx, None, ws)
    rows = y[keep_rows].double()
    want, mag = rows.sum(1), rows.abs().sum(1)
    ref.inside(dx[pick], want, (k + 3) * ref.U * mag + ref.BF * want.abs() * 1.001, "dx")
    assert _status(ws) == 0


# ------------------------------------------------------------------------------------------------ sorted rows

def _perm_inputs(T, H, E, k, S=None, on_input=False, add=None, gated=False, seed=0, pad=0):
    pr, w, rows = ref.routing(T, E, k, S, seed, pad)
    return dict(dxp=ref.rnd(rows, H, seed=seed + 1, std=0.1), pr=pr, w=w if on_input else None,
                x=ref.rnd(T, H, seed=seed + 2) if on_input else None,
                add=None if add is None else ref.rnd(T, H, seed=seed + 3, std=0.1, dtype=add),
                dz=ref.rnd(T, seed=seed + 4, dtype=torch.float32) if gated else None,
                gw=ref.rnd(H, seed=seed + 5, std=0.05) if gated else None)


def _perm(d, ws, dx=None, dw=True, stream=None):
    T, k = d["pr"].shape
    dx = torch.empty(T, d["dxp"].shape[1], dtype=torch.bfloat16, device="cuda") if dx is None else dx
    dw = torch.full((T, k), 9.0, device="cuda") if dw and d["x"] is not None else None
    moe.moe_permute_bwd(d["dxp"], d["pr"], d["w"], d["x"], d["add"], d["dz"], d["gw"], dx, dw, ws, stream)
    return dx, dw


def _perm_check(d, got):
    dx, dw = got
    T, k = d["pr"].shape
    H = dx.shape[1]
    live = (d["pr"] >= 0).double()
    rows = d["dxp"][d["pr"].clamp(min=0).long()].double()
    w = live if d["w"] is None else d["w"].double() * live
    terms = rows * w.unsqueeze(-1)
    want, mag = terms.sum(1), terms.abs().sum(1)
    if d["add"] is not None:
        want, mag = want + d["add"].double(), mag + d["add"].double().abs()
    if d["dz"] is not None:
        z = d["dz"].double()[:, None] * d["gw"].double()
        want, mag = want + z, mag + z.abs()
    tol = (k + 4) * ref.U * mag
    ref.inside(dx, want, tol + ref.BF * (want.abs() + tol), "dx")
    if dw is not None:
        prod = rows * d["x"].double().unsqueeze(1)
        ref.inside(dw, prod.sum(-1) * live, _chain(H) * prod.abs().sum(-1) * live, "dtopk_w")


@pytest.mark.parametrize("T,H,E,k,S", [(1, 64, 4, 1, None), (1, 2048, 64, 6, None), (2, 128, 8, 8, 4), (3, 7168, 16, 8, None),
                                       (77, 1408, 60, 4, None), (333, 64, 32, 32, 16), (1000, 2048, 64, 6, 20),
                                       (257, 192, 40, 17, 33), (64, 320, 12, 9, None), (5, 24640, 8, 3, None),
                                       (4099, 512, 60, 4, None), (130, 256, 16, 2, 0), (2500, 7168, 16, 5, 12)])
@pytest.mark.parametrize("on_input", [False, True])
@pytest.mark.parametrize("add,gated", [(None, False), (torch.bfloat16, True), (torch.float32, False)])
def test_permute_bwd(T, H, E, k, S, on_input, add, gated):
    d = _perm_inputs(T, H, E, k, S, on_input, add, gated, seed=1, pad=2)
    ws = _ws()
    _perm_check(d, _perm(d, ws))
    assert _status(ws) == 0


def test_permute_bwd_options():
    ws = _ws()
    d = _perm_inputs(90, 640, 16, 4, 10, True, torch.bfloat16, True, seed=2)
    want = _perm(d, ws)
    assert torch.equal(_perm(d, ws, dw=False)[0], want[0])
    add = d["add"].clone()
    got = _perm(dict(d, add=add), ws, dx=add)         # dx over dx_add
    assert torch.equal(add, want[0]) and torch.equal(got[1], want[1])
    x = d["x"].clone()
    got = _perm(dict(d, x=x), ws, dx=x)               # dx over x
    assert torch.equal(x, want[0]) and torch.equal(got[1], want[1])


def test_permute_bwd_bad_rows_are_dropped_and_flagged():
    d = _perm_inputs(40, 256, 8, 4, None, True, seed=3)
    ws = _ws()
    pr = d["pr"].clone()
    pr[0, 0], pr[7, 3], pr[39, 1], pr[20, 2] = -2, pr.numel(), 2 ** 31 - 1, -2 ** 31
    clean = torch.where((pr >= 0) & (pr < pr.numel()), pr, -1)
    want = _perm(dict(d, pr=clean), ws)
    assert _status(ws) == 0
    got = _perm(dict(d, pr=pr), ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert _status(ws) == moe.MOE_ERR_DEVICE_BOUNDS


def test_permute_bwd_dropped_pairs_do_not_spread_bad_values():
    """A pair without a row, or the rows behind the last pair, may hold anything."""
    d = _perm_inputs(60, 256, 16, 4, 8, True, seed=4)
    ws = _ws()
    want = _perm(d, ws)
    rows = int(d["pr"].max()) + 1
    d["dxp"][rows:] = float("nan")
    d["w"] = torch.where(d["pr"] >= 0, d["w"], torch.full_like(d["w"], float("nan")))
    got = _perm(d, ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------------------------ routing weights

def _route_inputs(T, E, k, renorm, seed=0, std=1.5):
    logits = ref.rnd(T, E, seed=seed, std=std, dtype=torch.float32)
    ids = logits.topk(k, dim=1).indices.to(torch.int32).contiguous()
    w = ref.weights(logits.double(), ids, renorm).float()
    return logits, ids, w, ref.rnd(T, k, seed=seed + 1, dtype=torch.float32)


def _route(logits, ids, w, dw, renorm, ws, out=None, stream=None):
    out = torch.full_like(logits, 7.0) if out is None else out
    moe.moe_route_bwd(ids, w, dw, None if renorm else logits, renorm, out, ws, stream)
    return out


def _route_check(logits, ids, w, dw, renorm, got):
    lg = logits.double().requires_grad_()
    ref.weights(lg, ids, renorm).backward(dw.double())
    # w is binary32 (2^-24), the softmax's exponentials are off by |l - max| 2^-24 (here below 2^-19) and their few
    # roundings, each term of c by as much
    p = torch.softmax(logits.double(), 1)
    chosen = torch.zeros_like(p).scatter_add_(1, ids.long(), w.double())
    c = (w * dw).double().abs().sum(1, keepdim=True)
    own = torch.zeros_like(p).scatter_add_(1, ids.long(), (w * dw).double().abs())
    tol = 2.0 ** -18 * (own + c * (chosen if renorm else p)) + 1e-37
    ref.inside(got, lg.grad, tol, "dlogits")
    if renorm:
        assert not got[chosen == 0].any()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (3, 2, 2), (9, 60, 4), (16, 31, 5), (17, 33, 8), (100, 65, 8),
                                   (1000, 128, 32), (333, 130, 8), (2000, 256, 8), (77, 257, 9), (64, 511, 32), (5000, 512, 8)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd(T, E, k, renorm):
    logits, ids, w, dw = _route_inputs(T, E, k, renorm, seed=1)
    ws = _ws()
    got = _route(logits, ids, w, dw, renorm, ws)
    _route_check(logits, ids, w, dw, renorm, got)
    assert _status(ws) == 0
    over = logits.clone()
    if not renorm:
        moe.moe_route_bwd(ids, w, dw, over, renorm, over, ws)     # dlogits over logits
        assert torch.equal(over, got)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd_masked_and_far_logits(renorm):
    logits, ids, w, dw = _route_inputs(40, 60, 4, renorm, seed=2)
    logits[:, 50:] = -float("inf")                    # experts shut off by the bias
    logits[:20] += 500.0
    logits[7, 3] = 600.0                              # one weight is all of it
    logits[9, 40:50] = torch.finfo(torch.float32).min
    ids = logits.topk(4, dim=1).indices.to(torch.int32).contiguous()
    w = ref.weights(logits.double(), ids, renorm).float()
    ws = _ws()
    got = _route(logits, ids, w, dw, renorm, ws)
    assert torch.isfinite(got).all() and not got[:, 50:].any()
    _route_check(logits, ids, w, dw, renorm, got)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd_bad_ids_are_left_out_and_flagged(renorm):
    logits, ids, w, dw = _route_inputs(40, 60, 4, renorm, seed=3)
    ws = _ws()
    bad = ids.clone()
    w2 = w.clone()
    for t, j, v in ((0, 0, -1), (7, 3, 60), (39, 1, 2 ** 31 - 1), (20, 2, -2 ** 31)):
        bad[t, j] = v
        w2[t, j] = 0.0
    want = _route(logits, ids, w2, dw, renorm, ws)
    assert _status(ws) == 0
    got = _route(logits, bad, w, dw, renorm, ws)
    assert torch.equal(got, want) and _status(ws) == moe.MOE_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd_an_expert_named_twice_gets_the_sum(renorm):
    logits, ids, w, dw = _route_inputs(40, 60, 6, renorm, seed=5)
    twice = ids.clone()
    twice[::2, 4] = twice[::2, 1]
    twice[::3, 5] = twice[::3, 1]
    got = _route(logits, twice, w, dw, renorm, _ws())
    wd = (w * dw).double()
    c, mag = wd.sum(1, keepdim=True), wd.abs().sum(1, keepdim=True)
    p = torch.softmax(logits.double(), 1)
    if renorm:
        p = torch.zeros_like(p).scatter_add_(1, twice.long(), w.double())
    want = (-c * p).scatter_add_(1, twice.long(), wd)
    own = torch.zeros_like(p).scatter_add_(1, twice.long(), wd.abs())
    ref.inside(got, want, 2.0 ** -18 * (own + mag * p) + 1e-37, "dlogits")
    again = _route(logits, twice, w, dw, renorm, _ws())
    assert torch.equal(got, again)


def test_route_bwd_of_the_routers_own_weights():
    T, H, E, k = 50, 256, 60, 4
    x, Wg = ref.rnd(T, H, seed=1), ref.rnd(E, H, seed=2, std=0.05, dtype=torch.float32)
    bias = ref.rnd(E, seed=3, dtype=torch.float32)
    n = moe.moe_workspace_size(T, H, 64, E, E, k)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    dw = ref.rnd(T, k, seed=4, dtype=torch.float32)
    logits = (x.double() @ Wg.double().t() + bias.double()).float()
    for renorm in (False, True):
        ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        moe.moe_route(x, Wg, bias, k, renorm, ids, w, ws)
        got = _route(logits, ids, w, dw, renorm, ws)
        _route_check(logits, ids, ref.weights(logits.double(), ids, renorm).float(), dw, renorm, got)
    assert _status(ws) == 0


# ------------------------------------------------------------------------------------------------ all of them

def test_differences():
    """Directional derivatives of the 64-bit forward formulas, at a step of 1e-4, against the kernels' gradients (the
    formulas are of low degree: the step's error is below 1e-7 of them)."""
    T, H, E, k = 6, 128, 8, 3
    ws, h = _ws(H), 1e-4
    d = _fin_inputs(T, H, E, k, 5, True, seed=7)
    o = _fin(d, ws)
    pr, dout = d["pr"], d["dout"].double()
    args = [t.double() for t in (d["y"], d["w"], d["ysh"], d["gw"])]
    f = lambda y, w, s, gw: float((ref.finalize(y, pr, w, s, d["x"].double(), gw) * dout).sum())  # noqa: E731
    for i, (g, rel) in enumerate(((o["dy"], ref.BF), (o["dw"], 2.0 ** -16), (o["dysh"], ref.BF), (o["dgw"], 2.0 ** -14))):
        v = torch.randn(args[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64).cuda()
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * v, args[i] - h * v
        g = g.double()
        if i == 0:  # rows without a pair keep their filling
            v[torch.tensor([r for r in range(v.shape[0]) if r not in set(pr.flatten().tolist())], device="cuda")] = 0.0
            up[0], dn[0] = args[0] + h * v, args[0] - h * v
        num = (f(*up) - f(*dn)) / (2 * h)
        assert abs(num - float((g * v).sum())) <= rel * float((g * v).abs().sum()) + 1e-6, i
    p = _perm_inputs(T, H, E, k, 5, True, seed=8)
    dx, dw = _perm(p, ws)
    x, w, dxp = p["x"].double(), p["w"].double(), p["dxp"].double()
    f = lambda x, w: float((ref.permuted(x, p["pr"], w, dxp.shape[0]) * dxp).sum())  # noqa: E731
    for i, g in enumerate((dx, dw)):
        v = torch.randn(g.shape, generator=torch.Generator().manual_seed(9 + i), dtype=torch.float64).cuda()
        a, b = [x, w], [x, w]
        a[i], b[i] = a[i] + h * v, b[i] - h * v
        num = (f(*a) - f(*b)) / (2 * h)
        assert abs(num - float((g.double() * v).sum())) <= ref.BF * float((g.double() * v).abs().sum()) + 1e-6
    for renorm in (False, True):
        logits, ids, w, dw = _route_inputs(T, 20, k, renorm, seed=9)
        g = _route(logits, ids, w, dw, renorm, ws).double()
        v = torch.randn(g.shape, generator=torch.Generator().manual_seed(12), dtype=torch.float64).cuda()
        f = lambda l: float((ref.weights(l, ids, renorm) * dw.double()).sum())  # noqa: E731
        num = (f(logits.double() + h * v) - f(logits.double() - h * v)) / (2 * h)
        assert abs(num - float((g * v).sum())) <= 1e-6 * (1 + float((g * v).abs().sum()))


def test_empty_batch():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, y, w = torch.empty(0, 64, **bf), torch.ones(5, 64, **bf), torch.empty(0, 2, device="cuda")
    pr = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    gw, dgw, dz = torch.ones(64, **bf), torch.ones(64, device="cuda"), torch.empty(0, device="cuda")
    ws = _ws()
    n = moe.moe_get_launch_count()
    moe.moe_finalize_bwd(x, y, pr, w, x, x, gw, y, w, x, dz, dgw, ws)
    moe.moe_permute_bwd(y, pr, None, None, None, None, None, x, None, ws)
    moe.moe_route_bwd(pr, w, w, None, True, torch.empty(0, 8, device="cuda"), ws)
    assert moe.moe_get_launch_count() == n and not dgw.any() and (y == 1).all()


def test_on_another_stream_and_in_graphs():
    d = _fin_inputs(300, 512, 16, 4, 12, True, seed=10)
    p = _perm_inputs(300, 512, 16, 4, 12, True, torch.float32, True, seed=11)
    logits, ids, w, dw = _route_inputs(300, 60, 4, False, seed=12)
    ws, ws2 = _ws(512), _ws(512)
    want = _fin(d, ws), _perm(p, ws), _route(logits, ids, w, dw, False, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = _fin(d, ws2, stream=s), _perm(p, ws2, stream=s), _route(logits, ids, w, dw, False, ws2, stream=s)

    def same(got):
        torch.cuda.synchronize()
        assert all(torch.equal(got[0][n], want[0][n]) for n in want[0])
        assert all(torch.equal(a, b) for a, b in zip(got[1], want[1])) and torch.equal(got[2], want[2])
    # _fin fills dy on the current stream: wait for both before comparing the rows the calls write
    torch.cuda.synchronize()
    live = d["pr"][d["pr"] >= 0].long()
    assert torch.equal(got[0]["dw"], want[0]["dw"]) and torch.equal(got[0]["dgw"], want[0]["dgw"])
    assert torch.equal(got[1][0], want[1][0]) and torch.equal(got[2], want[2]) and live.numel() > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _fin(d, ws2), _perm(p, ws2), _route(logits, ids, w, dw, False, ws2)
    for _ in range(3):
        graph.replay()
        same(got)
    assert _status(ws2) == 0


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Before anything is launched: the current device is made to look like another one than the tensors'."""
    x, w, ws = ref.rnd(2, 64), ref.rnd(64), _ws()
    i, f = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, device="cuda")
    n = moe.moe_get_launch_count()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in (lambda: moe.moe_add_layernorm(x, x, w, w, 1e-5, x, x),
                 lambda: moe.moe_add_rmsnorm_bwd(x, x, w, 1e-5, None, x, None, None, None),
                 lambda: moe.moe_add_layernorm_bwd(x, x, w, 1e-5, None, x, None, None, None, None),
                 lambda: moe.moe_finalize_bwd(x, x, i, f, None, None, None, x, f, None, None, None, ws),
                 lambda: moe.moe_permute_bwd(x, i, None, None, None, None, None, x, None, ws),
                 lambda: moe.moe_route_bwd(i, f, f, None, True, torch.empty_like(f), ws),
                 lambda: moe.moe_route_bwd(i, f, f, None, True, torch.empty_like(f), ws, torch.cuda.default_stream(0))):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert moe.moe_get_launch_count() == n


def test_no_rows_at_all():
    """A rank that holds no expert of the batch: no rows, every pair -1."""
    bf = dict(dtype=torch.bfloat16, device="cuda")
    T, k, H = 9, 3, 192
    ws = _ws(H)
    pr = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    none, w = torch.empty(0, H, **bf), torch.zeros(T, k, device="cuda")
    dw = torch.full((T, k), 4.0, device="cuda")
    moe.moe_finalize_bwd(ref.rnd(T, H), none, pr, w, None, None, None, none, dw, None, None, None, ws)
    assert not dw.any()
    add, dx, dw = ref.rnd(T, H, seed=1), torch.empty(T, H, **bf), torch.full((T, k), 4.0, device="cuda")
    moe.moe_permute_bwd(none, pr, w, ref.rnd(T, H, seed=2), add, None, None, dx, dw, ws)
    assert torch.equal(dx, add) and not dw.any() and _status(ws) == 0


@pytest.mark.parametrize("H", [256, 2048, 8320])
def test_calls_that_overlap_their_neighbours_wait_for_them(H):
    """Each call reads what the one before it wrote; with programmatic launches their kernels overlap, and the results are
    those of launches one behind the other."""
    T, k = 1500, 4
    d = _fin_inputs(T, H, 16, k, 12, True, seed=40)
    r, w, b = ref.rnd(T, H, seed=41), ref.rnd(H, seed=42), ref.rnd(H, seed=43)
    f32 = dict(dtype=torch.float32, device="cuda")

    def run(n):
        outs, ws = [], _ws(H)
        for i in range(n):
            x, stream = torch.empty_like(r), torch.empty_like(r)
            dy, dysh, dx, dr = torch.zeros_like(d["y"]), torch.empty_like(r), torch.empty_like(r), torch.empty_like(r)
            dw, dz, dgw = torch.empty(T, k, **f32), torch.empty(T, **f32), torch.empty(H, **f32)
            nw, nb = torch.empty(H, **f32), torch.empty(H, **f32)
            res = r * (i + 1)
            moe.moe_add_layernorm(d["x"], res, w, b, 1e-5, stream, x)
            moe.moe_finalize_bwd(x, d["y"], d["pr"], d["w"], d["ysh"], x, d["gw"], dy, dw, dysh, dz, dgw, ws)
            moe.moe_permute_bwd(dy, d["pr"], None, None, dysh, dz, d["gw"], dx, None, ws)
            moe.moe_add_layernorm_bwd(dx, stream, w, 1e-5, dysh, dr, None, nw, nb, ws)
            outs.append((dy, dw, dysh, dz, dgw, dx, dr, nw, nb))
        torch.cuda.synchronize()
        assert _status(ws) == 0
        return outs

    moe.moe_set_pdl(False)
    try:
        want = run(6)
    finally:
        moe.moe_set_pdl(True)
    for _ in range(4):
        for got, exp in zip(run(6), want):
            assert all(torch.equal(g, e) for g, e in zip(got, exp))


def test_binding_refuses_what_it_would_misread():
    d = _fin_inputs(4, 64, 8, 2, gated=True)
    ws = _ws()
    o = _fin(d, ws)
    order = ["dout", "y", "pr", "w", "ysh", "x", "gw", "dy", "dw", "dysh", "dz", "dgw"]
    good = {**d, **o}
    for n, bad in (("dout", d["dout"].float()), ("y", d["y"][:7]), ("pr", d["pr"].long()), ("w", d["w"].double()),
                   ("ysh", d["ysh"][:3]), ("gw", d["gw"][:32]), ("dy", o["dy"].t().contiguous().t()), ("dw", o["dw"][:3]),
                   ("dysh", o["dysh"].float()), ("dz", o["dz"][:3]), ("dgw", o["dgw"].half())):
        a = {**good, n: bad}
        with pytest.raises(ValueError):
            moe.moe_finalize_bwd(*[a[m] for m in order], ws)
    for n in ("ysh", "x", "gw", "dysh", "dz"):     # the shared expert's tensors come together
        a = {**good, n: None}
        with pytest.raises(moe.MoEError) as e:
            moe.moe_finalize_bwd(*[a[m] for m in order], ws)
        assert e.value.status == moe.MOE_ERR_INVALID_ARG
    p = _perm_inputs(4, 64, 8, 2, None, True, torch.float32, True)
    dx, dw = _perm(p, ws)
    good = dict(p, dx=dx, dw=dw)
    order = ["dxp", "pr", "w", "x", "add", "dz", "gw", "dx", "dw"]
    for n, bad in (("dxp", p["dxp"].float()), ("pr", p["pr"][:3]), ("w", p["w"][:, :1]), ("x", p["x"][:3]),
                   ("add", p["add"].half()), ("dz", p["dz"][:3]), ("gw", p["gw"].float()), ("dx", dx.float()),
                   ("dw", dw[:3])):
        with pytest.raises(ValueError):
            moe.moe_permute_bwd(*[{**good, n: bad}[m] for m in order], ws)
    for n in ("w", "x", "dz", "gw"):
        with pytest.raises(moe.MoEError):
            moe.moe_permute_bwd(*[{**good, n: None}[m] for m in order], ws)
    logits, ids, w, dw = _route_inputs(4, 8, 2, False)
    good = [ids, w, dw, logits, False, torch.empty_like(logits)]
    for i, bad in ((0, ids.long()), (1, w[:3]), (2, dw.double()), (3, logits[:, :7]), (5, logits.double())):
        a = list(good)
        a[i] = bad
        with pytest.raises(ValueError):
            moe.moe_route_bwd(*a, ws)
    with pytest.raises(moe.MoEError):
        moe.moe_route_bwd(ids, w, dw, None, False, torch.empty_like(logits), ws)
